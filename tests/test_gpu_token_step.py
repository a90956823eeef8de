"""Embedding, dropout and log probabilities together: a data-parallel training step against autograd in 64 bits, a
serving step, both replayed from graphs, two streams at once, rows past 4 GiB."""

import numpy as np
import pytest
import torch

import collective_communication_reduction_amd as gc
from oracle import token as K
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu

N, T, V, H = 4, [70, 33, 64, 1], 257, 64
SEED, P = 77, 0.25


def _f32(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(DEV)


class Step:
    """Tied embedding -> dropout -> residual RMS norm -> logits -> loss, every rank on tokens of its own, then one
    all-reduce of the gradients where the backward left them."""

    def __init__(self, rng):
        e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        self.tokens = [torch.zeros(t, dtype=torch.int32, device=DEV) for t in T]
        self.targets = [torch.zeros(t, dtype=torch.int32, device=DEV) for t in T]
        w, g = _f32(rng, V, H), 1 + _f32(rng, H, scale=0.1)
        self.weight, self.norm_w = [w.clone() for _ in T], [g.clone() for _ in T]
        rows = lambda: [e(t, H) for t in T]  # noqa: E731
        self.emb, self.s, self.h, self.dh, self.ds, self.demb = (rows() for _ in range(6))
        self.rstd, self.lp, self.ent, self.lse = ([e(t) for t in T] for _ in range(4))
        self.logits = [e(t, V) for t in T]
        n = sum(T)
        self.dlp = [torch.full((t,), -1.0 / n, device=DEV) for t in T]
        self.dent = [torch.full((t,), -0.1 / n, device=DEV) for t in T]
        self.dw, self.dg = [e(V, H) for _ in T], [e(H) for _ in T]
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        u8 = lambda k: torch.empty(k, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.s1 = u8(gc.gc_token_logprob_scratch_bytes(T, V))
        self.s2 = u8(gc.gc_rms_norm_backward_scratch_bytes(T, H))
        self.s3 = u8(gc.gc_embedding_backward_scratch_bytes(T, V, H))
        self.plan = gc.BucketPlan([V * H, H], "fp32", 1 << 30)

    def feed(self, rng):
        for t, dst in zip(T + T, self.tokens + self.targets):
            dst.copy_(torch.from_numpy(rng.integers(-1, V, t).astype(np.int32)))

    def run(self):
        gc.gc_embedding(self.weight, self.tokens, T, V, H, self.emb, scale=0.5)
        n = [t * H for t in T]
        gc.gc_dropout(self.emb, n, P, SEED, self.s, offset=2, step=self.step, residual=self.emb)
        gc.gc_rms_norm(self.s, self.norm_w, T, H, self.h, rstd=self.rstd, eps=1e-5)
        for x, h, w in zip(self.logits, self.h, self.weight):
            torch.mm(h, w.t(), out=x)
        gc.gc_token_logprob(self.logits, T, V, self.s1, targets=self.targets, logprob=self.lp, entropy=self.ent, lse=self.lse,
                            dlogprob=self.dlp, dentropy=self.dent, dlogits=self.logits)      # over the logits
        for x, h, w, dh, dw in zip(self.logits, self.h, self.weight, self.dh, self.dw):
            torch.mm(x, w, out=dh)
            torch.mm(x.t(), h, out=dw)                                                      # the tied weight's use in the head
        gc.gc_rms_norm_backward(self.dh, self.s, self.norm_w, self.rstd, T, H, self.ds, self.dg, self.s2)
        gc.gc_dropout(self.ds, n, P, SEED, self.demb, offset=2, step=self.step, residual=self.ds)
        gc.gc_embedding_backward(self.demb, self.tokens, T, V, H, self.dw, self.s3, scale=0.5, accumulate=True)
        self.plan.all_reduce(0, [t for r in range(N) for t in (self.dw[r], self.dg[r])], N, op="sum")
        self.step.add_(1)

    def results(self):
        return [t.clone() for a in (self.dw, self.dg, self.lp, self.ent) for t in a]


def _reference(st, step):
    """The same step in 64 bits with autograd: summed gradients, log probabilities and entropies."""
    d = lambda t: t.detach().cpu().double()  # noqa: E731
    w, g = d(st.weight[0]).requires_grad_(), d(st.norm_w[0]).requires_grad_()
    lps, ents, loss = [], [], 0.0
    n = sum(T)
    for r, t in enumerate(T):
        ids, tg = st.tokens[r].cpu().long(), st.targets[r].cpu().long()
        ok, used = ids >= 0, tg >= 0
        emb = torch.where(ok[:, None], w[ids.clamp(min=0)] * 0.5, 0.0)
        keep = torch.from_numpy(K.keep(t * H, r, P, SEED, 2 + step).reshape(t, H))
        s = emb + torch.where(keep, emb * (65536 / (65536 - K.drop_steps(P))), 0.0)
        h = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(np.float32(1e-5))) * g
        lp = torch.log_softmax(h @ w.t(), 1)
        e = -(lp.exp() * lp).sum(1)
        chosen = torch.where(used, lp[torch.arange(t), tg.clamp(min=0)], 0.0)
        loss = loss - (chosen.sum() + 0.1 * e.sum()) / n
        lps.append(chosen.detach())
        ents.append(e.detach())
    loss.backward()
    return w.grad, g.grad, lps, ents


# Six operators in a row, each with sums of at most V terms and a few operations more: 6 (V + 40) roundings of 2^-24,
# of each result's norm (the rows are normed, so nothing grows by more than the 2-norm of the weights, 20 here, once forth
# and once back; the terms' signs are mixed, so that the norms stay well below the sums of magnitudes that they bound).
TOL = 6 * (V + 40) * 2.0 ** -24 * 20


def _close(got, want):
    got = got.detach().cpu().double()
    return float((got - want).norm()) <= TOL * max(float(want.norm()), 1e-3)


def test_training_step():
    rng = np.random.default_rng(0)
    st = Step(rng)
    for step in range(2):
        st.feed(rng)
        st.run()
        dw, dg, lps, ents = _reference(st, step)
        for r in range(N):
            assert _close(st.dw[r], dw) and _close(st.dg[r], dg), r
            assert _close(st.lp[r], lps[r]) and _close(st.ent[r], ents[r]), r
            assert torch.equal(st.dw[r], st.dw[0])


def test_training_step_replayed():
    """One graph of the whole step, replayed on new tokens: bit for bit the eager step."""
    rng = np.random.default_rng(1)
    st, eager = Step(np.random.default_rng(2)), Step(np.random.default_rng(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st.feed(rng)
        st.run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.run()
    st.step.zero_()
    for k in range(4):
        state = rng.bit_generator.state
        st.feed(rng)
        rng.bit_generator.state = state
        eager.feed(rng)
        g.replay()
        eager.run()
        torch.cuda.synchronize()
        for a, b in zip(st.results(), eager.results()):
            assert torch.equal(a, b), k


def test_serving_step_replayed():
    """One token: lookup and the alternatives of its logits (a long row, in parts, and a short one), from one graph."""
    rng = np.random.default_rng(3)
    for vocab in (70000, 1000):
        w, big = _f32(rng, 50, H).bfloat16(), _f32(rng, vocab, H, scale=0.3).bfloat16()
        ids = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = torch.empty(1, H, dtype=torch.bfloat16, device=DEV)
        logits = torch.empty(1, vocab, dtype=torch.bfloat16, device=DEV)
        top, lp, lse = torch.empty(1, 8, dtype=torch.int32, device=DEV), torch.empty(1, 8, device=DEV), torch.empty(1, device=DEV)
        scratch = torch.empty(gc.gc_token_logprob_scratch_bytes([1], vocab, 8), dtype=torch.uint8, device=DEV)

        def step():
            gc.gc_embedding([w], [ids], [1], 50, H, [out], scale=8.0)
            torch.mm(out, big.t(), out=logits)
            gc.gc_token_logprob([logits], [1], vocab, scratch, lse=[lse], top=8, top_ids=[top], top_logprob=[lp])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for k in range(4):
            ids.fill_(7 * k + 1)
            g.replay()
            got = [t.clone() for t in (top, lp, lse)]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (top, lp, lse)))
            x = logits.cpu().double().numpy()
            want, _ = K.alternatives(x, K.log_softmax(x)[0], 8)
            assert np.array_equal(top.cpu().numpy(), want)


def test_two_streams_at_once():
    """Calls on two streams, each with scratch of its own, give what they give alone."""
    rng = np.random.default_rng(4)
    steps = [Step(np.random.default_rng(10 + i)) for i in range(2)]
    for st in steps:
        st.feed(rng)
        st.run()
    torch.cuda.synchronize()
    alone = [st.results() for st in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for st in steps:
        st.step.zero_()
    torch.cuda.synchronize()
    for st, s in zip(steps, streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                st.step.zero_()
                st.run()
    torch.cuda.synchronize()
    for st, want in zip(steps, alone):
        assert all(torch.equal(a, b) for a, b in zip(st.results(), want))


@pytest.fixture
def room():
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_rows_past_4_gib(room):
    """Rows behind 4 GiB of logits, weights and gradients: those of a small call on the same data."""
    g = torch.Generator(device=DEV).manual_seed(5)
    R, W = 70001, 33000                                          # 4.6 GB of bf16
    x = torch.zeros(R, W, dtype=torch.bfloat16, device=DEV)
    some = [0, 1, 40000, R - 2, R - 1]
    x[some] = torch.empty(len(some), W, dtype=torch.bfloat16, device=DEV).normal_(0, 3, generator=g)
    tg = torch.full((R,), 5, dtype=torch.int32, device=DEV)
    w = torch.full((R,), -1.0, device=DEV)
    lp, dx = torch.empty(R, device=DEV), torch.empty_like(x)
    scratch = torch.empty(gc.gc_token_logprob_scratch_bytes([R], W, 4), dtype=torch.uint8, device=DEV)
    ids, tl = torch.empty(R, 4, dtype=torch.int32, device=DEV), torch.empty(R, 4, device=DEV)
    gc.gc_token_logprob([x], [R], W, scratch, targets=[tg], logprob=[lp], dlogprob=[w], dlogits=[dx])
    gc.gc_token_logprob([x], [R], W, scratch, top=4, top_ids=[ids], top_logprob=[tl])
    n = len(some)
    xs, lps, dxs = x[some].contiguous(), torch.empty(n, device=DEV), torch.empty(n, W, dtype=torch.bfloat16, device=DEV)
    gc.gc_token_logprob([xs], [n], W, scratch, targets=[tg[:n]], logprob=[lps], dlogprob=[w[:n]], dlogits=[dxs])
    assert torch.equal(lp[some], lps) and torch.equal(dx[some], dxs)
    assert float((lp[[2, R - 3]] + np.log(W)).abs().max()) < 1e-5          # the rows of zeros between
    want, _ = K.alternatives(xs.cpu().double().numpy(), np.zeros((n, W)), 4)
    assert np.array_equal(ids[some].cpu().numpy(), want)
    # the same buffer as a weight of 70001 rows, and its gradient
    tok = torch.tensor([R - 1, 0, 40000, R, R - 1, -1], dtype=torch.int32, device=DEV)
    out = torch.empty(6, W, dtype=torch.bfloat16, device=DEV)
    gc.gc_embedding([x], [tok], [6], R, W, [out])
    zero = torch.zeros(W, dtype=torch.bfloat16, device=DEV)
    assert all(torch.equal(a, b) for a, b in zip(out, (x[R - 1], x[0], x[40000], zero, x[R - 1], zero)))
    dx.fill_(7)
    scratch = torch.empty(gc.gc_embedding_backward_scratch_bytes([6], R, W), dtype=torch.uint8, device=DEV)
    gc.gc_embedding_backward([out], [tok], [6], R, W, [dx], scratch)
    twice = (x[R - 1].float() * 2).bfloat16()
    assert torch.equal(dx[R - 1], twice) and torch.equal(dx[0], x[0]) and torch.equal(dx[40000], x[40000])
    assert float(dx.view(-1, 33).sum(1, dtype=torch.float32).abs().count_nonzero()) <= 3 * W // 33


def test_dropout_past_2_32_elements(room):
    n = (1 << 32) + 19
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    gc.gc_dropout([x], [n], 0.5, SEED, [x], offset=1)
    for first in (0, (1 << 32) - 64, n - 11 - (n - 11) % 8):
        count = min(64, n - first)
        b = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
        counter = np.stack([b & K.M32, b >> np.uint64(32), np.full_like(b, 1), np.zeros_like(b)], axis=-1)
        words = K.philox4x32(counter, (SEED, 0))
        keep = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=-1).reshape(-1)[:count] >= 32768
        assert np.array_equal(x[first:first + count].float().cpu().numpy() != 0, keep), first
