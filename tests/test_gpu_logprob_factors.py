"""The gradient of the logits with large factors: what has probability 0 gets a gradient of 0, whatever the factors and
however far below the mask lies; the rest against 64 bits with bounds counted from the roundings."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import token as K
from tests.gpu_util import DEV
from tests.test_gpu_embed import HALF, TYPES, U, _f64
from tests.test_gpu_logprob import _bounds

pytestmark = pytest.mark.gpu
NINF = float("-inf")

FACTORS = [
    # mask (a number of times the type's lowest where below 2), scale, dlogprob, dentropy
    ("number", -2e38, 1.0, 1.0, 2.0), ("number", -1e37, 0.5, 1.0, 1000.0), ("number", -1e37, 1.0, -1.0, 655.0), ("lowest", 0.5, 1.0, 1.0, 3.0),
    ("lowest", 1.0, 0.5, 1.0, 5.0), ("lowest", 1.0, 1.0, -3.0, -1000.0), ("number", -1e30, 1.0, 1.0, 1e9), ("number", NINF, 1.0, 1.0, 1e9),
    ("number", NINF, 1.0, 1e30, 1e30), ("number", NINF, 2.0 ** 40, 1.0, 1.0), ("number", NINF, 2.0 ** 64, 2.0 ** -10, 2.0 ** 30),
    ("number", -300.0, 1.0, 1.0, 1e30), ("number", -1e4, 1.0, 1e30, -1e31), ("number", NINF, 1.0, 1.0, 0.01),
    # so large that a limit on the exponent does not keep the product with the factor finite
    ("number", NINF, 1.0, 1e35, 1e33), ("lowest", 0.5, 1.0, -1e35, 1e36), ("number", NINF, 2.0 ** 64, 2.0 ** -10, 2.0 ** 60),
    ("number", -200.0, 1.0, 1e33, 1e36),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,pad", [(9, 0), (1003, 5), (4096, 0), (33000, 0), (140001, 0)])
@pytest.mark.parametrize("kind,mask,scale,da,db", FACTORS)
def test_what_is_masked_takes_no_gradient(V, pad, dtype, kind, mask, scale, da, db):
    rng = np.random.default_rng(V)
    M = torch.finfo(TYPES[dtype]).min * mask if kind == "lowest" else mask
    n = 5
    x = rng.normal(size=(n, V)) * 2
    masked = np.zeros((n, V), dtype=bool)
    masked[1] = rng.random(V) < 0.5
    masked[2] = True
    masked[2, rng.permutation(V)[:3]] = False
    masked[3, 1:] = True
    masked[4, V - 1] = True
    masked[1, 0] = False
    x[masked] = M
    xt = torch.zeros(n, V + pad).to(TYPES[dtype])
    xt[:, :V] = torch.from_numpy(x).to(TYPES[dtype])
    xt = xt.to(DEV)
    x64 = _f64(xt[:, :V])
    targets = np.array([rng.choice(np.nonzero(~m)[0]) for m in masked], dtype=np.int32)
    tg = torch.from_numpy(targets).to(DEV)
    a, b = torch.full((n,), da, device=DEV), torch.full((n,), db, device=DEV)
    lp, h, lse = (torch.empty(n, device=DEV) for _ in range(3))
    both, later = torch.empty_like(xt), torch.empty_like(xt)
    scratch = torch.empty(gc.gc_token_logprob_scratch_bytes([n], V), dtype=torch.uint8, device=DEV)
    common = dict(stride=V + pad, scale=scale)
    gc.gc_token_logprob([xt], [n], V, scratch, targets=[tg], logprob=[lp], entropy=[h], lse=[lse], dlogprob=[a], dentropy=[b],
                        dlogits=[both], **common)
    gc.gc_token_logprob_backward([xt], [n], V, [lse], [tg], [a], [later], entropy=[h], dentropy=[b], **common)
    none = masked & (np.arange(V) != targets[:, None])
    for g in (_f64(both), _f64(later)):
        assert (g[:, :V][none] == 0).all() and (g[:, V:] == 0).all()
    # the joint pass against the formula: bounds as for factors of 1, times the factors
    want = K.log_softmax(x64, scale)[0]
    want_h = K.entropy(want)
    rel_s, abs_h = _bounds(x64, want, scale, V)
    big = np.abs(x64.max(1) * scale)
    big = np.where(big < 2 ** 24, big, 0.0)
    lg = np.log(V)
    p, ok = np.exp(want), want > -1e3
    d = np.where(ok, np.abs(want), 0.0)
    hit = (np.arange(V) == targets[:, None]) * 1.0
    with np.errstate(invalid="ignore"):
        dz = scale * (da * (hit - p) - db * np.where(ok, p * (want + want_h[:, None]), 0.0))
    tol_h = abs_h + 8 * U * (1 + want_h + lg + big)
    rel_p = rel_s[:, None] + U * (8 + 4 * d + 4 * (lg + big)[:, None])
    hh = d + want_h[:, None]
    # the bracket's sum, its factors' products and the target's addition: each a rounding of the terms' magnitudes; below
    # 2^-126 a probability counts as 0
    err = abs(da) * (p * rel_p + 4 * U * (hit + p)) + abs(db) * p * (hh * (rel_p + 8 * U) + rel_p + (tol_h + abs_h)[:, None])
    err = err + 2.0 ** -125 * (abs(da) + abs(db) * hh)
    tol = scale * err + (HALF[dtype] + 4 * U) * np.abs(dz) * (1 + 2 ** -8) + 1e-37
    top = torch.finfo(TYPES[dtype]).max                       # beyond it a gradient may be infinite
    got = _f64(both)[:, :V]
    with np.errstate(invalid="ignore"):
        assert ((np.abs(got - dz) <= tol) | (np.abs(dz) + tol > top)).all()


def test_factors_that_are_no_numbers():
    """A NaN or infinity among the factors of a row reaches all of that row, and no other."""
    V, n = 1000, 4
    x = torch.randn(n, V, generator=torch.Generator().manual_seed(1)).to(DEV)
    x[:, 7::3] = NINF
    tg, a, b = torch.zeros(n, dtype=torch.int32, device=DEV), torch.ones(n, device=DEV), torch.ones(n, device=DEV)
    a[1], b[2] = float("nan"), float("nan")
    lp, h, lse = (torch.empty(n, device=DEV) for _ in range(3))
    both, later = torch.empty_like(x), torch.empty_like(x)
    scratch = torch.empty(gc.gc_token_logprob_scratch_bytes([n], V), dtype=torch.uint8, device=DEV)
    gc.gc_token_logprob([x], [n], V, scratch, targets=[tg], logprob=[lp], entropy=[h], lse=[lse], dlogprob=[a], dentropy=[b], dlogits=[both])
    gc.gc_token_logprob_backward([x], [n], V, [lse], [tg], [a], [later], entropy=[h], dentropy=[b])
    for g in (both, later):
        assert g[1:3].isnan().all() and g[[0, 3]].isfinite().all() and (g[[0, 3], 7::3] == 0).all()
