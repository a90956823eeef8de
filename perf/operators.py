"""Cases of the MoE layer's operators: norm, experts, combine gradient, 8-bit rows.

Every case is one call sequence a training or serving step makes on the N rank
buffers of one GPU.  With `own` false, run() computes the operators from
elementary torch operations in 32 bits; with `own` true, it calls the library.

  norm       s = x + residual; y = s / rms(s) * w, in the row type or as 8-bit rows
  norm_bwd   gradients of x (= residual) and w
  pack       activation rows to 8-bit rows with a scale per 32 values, and back
  combine_bwd  gradients of the weighted un-permute: expert rows and gate weights
  ffn        the experts' gated feed-forward on the receive layout
  ffn_bwd    its gradients, from 16-bit or 8-bit checkpoints

8-bit rows ("mx8"): n e4m3 values, one scale byte per 32 values (a power of two,
biased by 127), zero bytes up to a multiple of 16.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a serving step, hidden size of the repository's transformer layer
        {"name": "norm_one_token", "op": "norm", "ranks": 1, "tokens": 1, "hidden": 4096, "dtype": "bf16", "out": "bf16"},
        # the expert-parallel workload's 8 x 16384 tokens, sent on in 8 bits
        {"name": "norm_8bit_8x16384", "op": "norm", "ranks": 8, "tokens": 16384, "hidden": 4096, "dtype": "bf16", "out": "mx8"},
        # fp32 rows of an odd length, ragged ranks
        {"name": "norm_bwd_fp32_odd", "op": "norm_bwd", "ranks": 3, "tokens": 1021, "hidden": 4099, "dtype": "fp32", "out": "fp32"},
        # the same layer's backward at the expert-parallel workload's size
        {"name": "norm_bwd_8x16384", "op": "norm_bwd", "ranks": 8, "tokens": 16384, "hidden": 4096, "dtype": "bf16", "out": "bf16"},
        # a short sequence's activations of a small fp32 layer
        {"name": "pack_fp32_odd", "op": "pack", "ranks": 2, "tokens": 257, "hidden": 1000, "dtype": "fp32", "out": "mx8"},
        # activations of the transformer layer's MLP kept for the backward pass
        {"name": "pack_4x8192_mlp", "op": "pack", "ranks": 4, "tokens": 8192, "hidden": 11008, "dtype": "bf16", "out": "mx8"},
        # a short batch of a few tokens per rank
        {"name": "combine_bwd_fp32_small", "op": "combine_bwd", "ranks": 4, "tokens": 37, "hidden": 1000, "dtype": "fp32",
         "experts": 3, "topk": 2},
        # the expert-parallel workload: 8 ranks, 64 experts, top-2
        {"name": "combine_bwd_8x16384", "op": "combine_bwd", "ranks": 8, "tokens": 16384, "hidden": 4096, "dtype": "bf16",
         "experts": 8, "topk": 2},
        # one decoded token, top-2 of eight experts of the transformer layer's MLP size: weights streamed once
        {"name": "ffn_one_token", "op": "ffn", "ranks": 1, "experts": 8, "rows": 2, "hidden": 4096, "inter": 11008,
         "x": "bf16", "saved": "none", "skew": 1.1},
        # training forward, checkpoints in 8 bits, ragged experts
        {"name": "ffn_32768_saved8", "op": "ffn", "ranks": 8, "experts": 2, "rows": 32768, "hidden": 4096, "inter": 2048,
         "x": "bf16", "saved": "mx8", "skew": 0.4},
        # backward of many small ragged experts (64 experts of the expert-parallel workload), 16-bit checkpoints
        {"name": "ffn_bwd_64_experts", "op": "ffn_bwd", "ranks": 8, "experts": 8, "rows": 8111, "hidden": 2048, "inter": 1024,
         "x": "bf16", "saved": "bf16", "skew": 1.1},
        # the training forward's backward, every checkpoint in 8 bits
        {"name": "ffn_bwd_32768_saved8", "op": "ffn_bwd", "ranks": 8, "experts": 2, "rows": 32768, "hidden": 4096,
         "inter": 2048, "x": "mx8", "saved": "mx8", "skew": 0.4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "pack", "combine_bwd", "ffn", "ffn", "ffn_bwd", "ffn_bwd"])
    if op in ("ffn", "ffn_bwd"):
        return {"op": op, "ranks": rng.randint(1, 8), "experts": rng.randint(1, 8), "rows": _log(rng, 1, 16384),
                "hidden": 8 * _log(rng, 8, 512), "inter": 32 * _log(rng, 2, 128), "x": rng.choice(["bf16", "mx8"]),
                "saved": rng.choice(["bf16", "mx8"] if op == "ffn_bwd" else ["none", "bf16", "mx8"]),
                "skew": rng.choice([0.0, 0.4, 1.1])}
    hidden = _log(rng, 32, 8192)
    if rng.random() < 0.6:
        hidden = max(32, hidden // 32 * 32)
    t = rng.choice(["bf16", "bf16", "fp32"])
    c = {"op": op, "ranks": rng.randint(1, 8), "tokens": _log(rng, 1, 4096), "hidden": hidden, "dtype": t}
    if op == "combine_bwd":
        c.update(experts=rng.randint(1, 8), topk=rng.randint(1, 4))
        c["topk"] = min(c["topk"], c["ranks"] * c["experts"])
    else:
        c["out"] = "mx8" if op == "pack" else rng.choice([t, "mx8"]) if op == "norm" else t
    return c


def _sizes(n, ranks):
    """Tokens of each rank: full on the first, a few fewer on each later one."""
    return [max(0, n - 3 * r if n < 4096 else n) for r in range(ranks)]


def _row8(n):
    return (n + -(-n // 32) + 15) // 16 * 16


def _split_rows(case, seed):
    """Rows of every (destination rank, expert) and source: the table of the routing plan, on the host."""
    N, E, R = case["ranks"], case["experts"], case["rows"]
    g = torch.Generator().manual_seed(seed * 7 + 3)
    w = (torch.arange(N * E, dtype=torch.float64) + 1) ** -case["skew"]
    w = w[torch.randperm(N * E, generator=g)]
    e = torch.multinomial(w, R, replacement=True, generator=g)
    s = torch.randint(0, N, (R,), generator=g)
    return torch.bincount(s * (N * E) + e, minlength=N * N * E).view(N, N, E)


# ------------------------------------------------------------------ 8-bit rows, plain

def _quantise(v):
    """fp32 rows [T, n] to (e4m3 codes as bytes [T, n], exponents [T, ceil(n/32)])."""
    T, n = v.shape
    nb = -(-n // 32)
    p = torch.nn.functional.pad(v, (0, nb * 32 - n)).view(T, nb, 32)
    a = torch.where(p.isfinite(), p.abs(), torch.zeros_like(p)).amax(2)
    m, e = torch.frexp(a)                                   # a = m * 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)                # smallest e with a <= 448 * 2^e
    e = torch.where(a > 0, e, torch.full_like(e, -117)).clamp(-117, 120)
    q = torch.where(p.isfinite(), torch.ldexp(p, -e.unsqueeze(2)), torch.full_like(p, float("nan")))
    return q.to(torch.float8_e4m3fn).view(T, nb * 32)[:, :n], e


def _dequantise(q, e):
    T, n = q.shape
    s = e.repeat_interleave(32, dim=1)[:, :n]
    return torch.ldexp(q.float(), s)


def _rows8(v):
    """fp32 rows as 8-bit rows [T, row bytes] uint8."""
    q, e = _quantise(v)
    T, n = v.shape
    out = torch.zeros(T, _row8(n), dtype=torch.uint8, device=v.device)
    out[:, :n] = q.view(torch.uint8)
    out[:, n:n + e.shape[1]] = (e + 127).to(torch.uint8)
    return out


def _values8(rows, n):
    q = rows[:, :n].contiguous().view(torch.float8_e4m3fn)
    return _dequantise(q, rows[:, n:n + -(-n // 32)].int() - 127)


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    N = case["ranks"]
    c = dict(case)
    if case["op"] in ("ffn", "ffn_bwd"):
        E, H, F = case["experts"], case["hidden"], case["inter"]
        table = _split_rows(case, seed)
        counts = table.sum(0)                                         # [rank][expert]
        rows = counts.sum(1).tolist()
        R = sum(rows)
        x = torch.empty(R, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        st = {"case": c, "rows": rows, "counts": counts.view(-1).tolist(), "splits": table.reshape(-1).to(DEV)}
        st["x"] = _rows8(x.float()) if case["x"] == "mx8" else x
        for k, (o, i) in {"w_gate": (F, H), "w_up": (F, H), "w_down": (H, F)}.items():
            st[k] = torch.empty(N, E, o, i, dtype=torch.bfloat16, device=DEV).normal_(0, i ** -0.5, generator=g)
        if case["saved"] != "none":
            # gate and up projections of unit variance, as the forward leaves them
            st["saved"] = torch.empty(R, 2 * F, dtype=torch.bfloat16, device=DEV)
            if case["op"] == "ffn_bwd":
                st["saved"].normal_(generator=g)
            if case["saved"] == "mx8":
                st["saved"] = _rows8(st["saved"].float()) if case["op"] == "ffn_bwd" else \
                    torch.empty(R, _row8(2 * F), dtype=torch.uint8, device=DEV)
        if case["op"] == "ffn":
            st["y"] = torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
            if case["saved"] == "mx8":
                st["values"] = torch.empty(R, 2 * F, dtype=torch.bfloat16, device=DEV)
        else:
            st["dy"] = torch.empty(R, H, dtype=torch.bfloat16, device=DEV).normal_(0, 1e-3, generator=g)
            st["dx"] = torch.empty(R, H, dtype=torch.bfloat16, device=DEV)
            for k in ("w_gate", "w_up", "w_down"):
                st["d" + k] = torch.empty_like(st[k])
        return st
    T, H, t = _sizes(case["tokens"], N), case["hidden"], TYPES[case["dtype"]]
    A = sum(T)
    st = {"case": c, "tokens": T}
    if case["op"] == "norm":
        st["x"], st["residual"] = _randn(g, A, H, dtype=t, scale=0.5), _randn(g, A, H, dtype=t, scale=2.0)
        st["weight"] = _randn(g, N, H, dtype=t, scale=0.1) + 1
        st["sum"] = torch.empty(A, H, dtype=t, device=DEV)
        st["rstd"] = torch.empty(A, dtype=torch.float32, device=DEV)
        st["y"] = torch.empty(A, _row8(H), dtype=torch.uint8, device=DEV) if case["out"] == "mx8" else torch.empty_like(st["sum"])
        if case["out"] == "mx8":
            st["values"] = torch.empty(A, H, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "norm_bwd":
        st["sum"] = _randn(g, A, H, dtype=t, scale=2.0)
        st["rstd"] = torch.rsqrt(st["sum"].float().square().mean(1) + EPS)
        st["weight"] = _randn(g, N, H, dtype=t, scale=0.1) + 1
        st["dy"], st["dsum"] = _randn(g, A, H, dtype=t, scale=1e-3), _randn(g, A, H, dtype=t, scale=1e-3)
        st["dx"] = torch.empty(A, H, dtype=t, device=DEV)
        st["dweight"] = torch.empty(N, H, dtype=torch.float32, device=DEV)
    elif case["op"] == "pack":
        st["x"] = _randn(g, A, H, dtype=t)
        st["packed"] = torch.empty(A, _row8(H), dtype=torch.uint8, device=DEV)
        st["values"] = torch.empty(A, H, dtype=torch.bfloat16, device=DEV)
    else:                                                              # combine_bwd
        K, E = case["topk"], case["experts"]
        p = (torch.arange(N * E, dtype=torch.float32, device=DEV) + 1) ** -1.1
        expert = torch.multinomial(p.expand(max(1, A), -1), K, generator=g)[:A]
        src = torch.repeat_interleave(torch.arange(N, device=DEV), torch.tensor(T, device=DEV))
        key = ((expert * N + src[:, None]) * (A * K + 1) + torch.arange(A * K, device=DEV).view(A, K)).view(-1)
        order = torch.argsort(key)                                     # receive layout: expert, source, route
        pos = torch.empty_like(order)
        pos[order] = torch.arange(A * K, device=DEV)
        rank = expert.view(-1) // E
        per = torch.bincount(rank, minlength=N)
        base = torch.cumsum(per, 0) - per
        st["dest"] = torch.stack([rank, pos - base[rank]], 1).to(torch.int32).contiguous()
        st["rows"] = per.tolist()
        st["expert_out"] = _randn(g, A * K, H, dtype=t)
        st["weights"] = torch.rand(A, K, generator=g, device=DEV)
        st["dout"] = _randn(g, A, H, dtype=t, scale=1e-3)
        st["dexpert"] = torch.empty(A * K, H, dtype=t, device=DEV)
        st["dweights"] = torch.empty(A, K, dtype=torch.float32, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _per_row(weight, T):
    """A rank's weight for each of its rows."""
    return weight.float().repeat_interleave(torch.tensor(T, device=DEV), dim=0, output_size=sum(T))


def _norm_plain(st):
    c = st["case"]
    t = TYPES[c["dtype"]]
    s = (st["x"].float() + st["residual"].float()).to(t)
    v = s.float()
    r = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * r[:, None] * _per_row(st["weight"], st["tokens"])
    return [_dequantise(*_quantise(y)).bfloat16() if c["out"] == "mx8" else y.to(t), s, r]


def _norm_bwd_plain(st):
    T = st["tokens"]
    n = st["sum"].float() * st["rstd"][:, None]
    dy = st["dy"].float()
    d = dy * _per_row(st["weight"], T)
    dx = st["rstd"][:, None] * (d - n * (d * n).mean(1, keepdim=True)) + st["dsum"].float()
    dw = torch.stack([p.sum(0) for p in (dy * n).split(T)])
    return [dx.to(st["sum"].dtype), dw]


def _pack_plain(st):
    return _dequantise(*_quantise(st["x"].float())).bfloat16()


def _combine_bwd_plain(st):
    K = st["case"]["topk"]
    base = torch.tensor(st["rows"], device=DEV).cumsum(0) - torch.tensor(st["rows"], device=DEV)
    row = base[st["dest"][:, 0].long()] + st["dest"][:, 1].long()
    dout = st["dout"].float()
    w = st["weights"].view(-1)
    de = torch.empty_like(st["expert_out"])
    de[row] = (dout.repeat_interleave(K, dim=0) * w[:, None]).to(de.dtype)
    dw = (dout.repeat_interleave(K, dim=0) * st["expert_out"].float()[row]).sum(1)
    return [de, dw.view_as(st["weights"])]


def _padded(st):
    """Experts with rows, and the rows of each padded to the longest: index [S, C] and its mask."""
    counts = torch.tensor(st["counts"], device=DEV)
    seg = torch.tensor([i for i, n in enumerate(st["counts"]) if n], device=DEV)
    n = counts[seg]
    start = (counts.cumsum(0) - counts)[seg]
    c = torch.arange(max(st["counts"]), device=DEV)
    mask = c[None, :] < n[:, None]
    return seg, torch.where(mask, start[:, None] + c, 0), mask


def _ffn_plain(st):
    c = st["case"]
    H, F = c["hidden"], c["inter"]
    seg, idx, mask = _padded(st)
    x = _values8(st["x"], H) if c["x"] == "mx8" else st["x"].float()
    xp = x[idx]
    gate = torch.bmm(xp, st["w_gate"].view(-1, F, H)[seg].float().transpose(1, 2))
    up = torch.bmm(xp, st["w_up"].view(-1, F, H)[seg].float().transpose(1, 2))
    y = torch.bmm(gate * torch.sigmoid(gate) * up, st["w_down"].view(-1, H, F)[seg].float().transpose(1, 2))
    out = [y[mask].bfloat16()]
    if c["saved"] != "none":
        saved = torch.cat([gate, up], 2)[mask]
        out.append((_dequantise(*_quantise(saved)) if c["saved"] == "mx8" else saved).bfloat16())
    return out


def _ffn_bwd_plain(st):
    c = st["case"]
    H, F = c["hidden"], c["inter"]
    seg, idx, mask = _padded(st)
    m = mask[:, :, None].float()
    x = (_values8(st["x"], H) if c["x"] == "mx8" else st["x"].float())[idx]
    saved = (_values8(st["saved"], 2 * F) if c["saved"] == "mx8" else st["saved"].float())[idx]
    dy = st["dy"].float()[idx] * m
    gate, up = saved[:, :, :F], saved[:, :, F:]
    sig = torch.sigmoid(gate)
    act = gate * sig
    dh = torch.bmm(dy, st["w_down"].view(-1, H, F)[seg].float())
    dg = dh * up * (sig * (1 + gate * (1 - sig)))
    du = dh * act
    dx = torch.bmm(dg, st["w_gate"].view(-1, F, H)[seg].float()) + torch.bmm(du, st["w_up"].view(-1, F, H)[seg].float())
    grads = []
    for a, b, k in ((dg, x, "w_gate"), (du, x, "w_up"), (dy, act * up, "w_down")):
        w = torch.zeros_like(st[k]).view(-1, a.shape[2], b.shape[2])
        w[seg] = torch.bmm(a.transpose(1, 2), b).bfloat16()
        grads.append(w.view_as(st[k]))
    return [dx[mask].bfloat16()] + grads


# ------------------------------------------------------------------ the library's calls

def _run_own(st):
    import collective_communication_reduction_amd as gc

    c = st["case"]
    op, N, H = c["op"], c["ranks"], c["hidden"]
    if op in ("ffn", "ffn_bwd"):
        E, F, rows = c["experts"], c["inter"], st["rows"]
        kw = dict(x_dtype=c["x"], saved_dtype=None if c["saved"] == "none" else c["saved"])
        need = gc.gc_moe_ffn_scratch_bytes(rows, E, H, F, x_dtype=c["x"], backward=op == "ffn_bwd")
        scratch = torch.empty(need, dtype=torch.uint8, device=DEV)
        w = [st[k].unbind(0) for k in ("w_gate", "w_up", "w_down")]
        x = st["x"].split(rows)
        saved = None if c["saved"] == "none" else st["saved"].split(rows)
        if op == "ffn":
            gc.gc_moe_ffn(x, rows, st["splits"], E, H, F, *w, st["y"].split(rows), scratch, saved=saved, **kw)
            if c["saved"] == "mx8":
                gc.gc_mx8_unpack(saved, rows, 2 * F, st["values"].split(rows))
                return [st["y"], st["values"]]
            return [st["y"]] if saved is None else [st["y"], st["saved"]]
        gc.gc_moe_ffn_backward(st["dy"].split(rows), x, saved, rows, st["splits"], E, H, F, *w, st["dx"].split(rows),
                               st["dw_gate"].unbind(0), st["dw_up"].unbind(0), st["dw_down"].unbind(0), scratch, **kw)
        return [st["dx"], st["dw_gate"], st["dw_up"], st["dw_down"]]
    T = st["tokens"]
    if op == "norm":
        y = st["y"].split(T)
        gc.gc_rms_norm(st["x"].split(T), st["weight"].unbind(0), T, H, y, residual=st["residual"].split(T),
                       sum_out=st["sum"].split(T), rstd=st["rstd"].split(T), eps=EPS)
        if c["out"] == "mx8":
            gc.gc_mx8_unpack(y, T, H, st["values"].split(T))
            return [st["values"], st["sum"], st["rstd"]]
        return [st["y"], st["sum"], st["rstd"]]
    if op == "norm_bwd":
        scratch = torch.empty(gc.gc_rms_norm_backward_scratch_bytes(T, H), dtype=torch.uint8, device=DEV)
        gc.gc_rms_norm_backward(st["dy"].split(T), st["sum"].split(T), st["weight"].unbind(0), st["rstd"].split(T), T, H,
                                st["dx"].split(T), st["dweight"].unbind(0), scratch, dsum=st["dsum"].split(T))
        return [st["dx"], st["dweight"]]
    if op == "pack":
        packed = st["packed"].split(T)
        gc.gc_mx8_pack(st["x"].split(T), T, H, packed)
        gc.gc_mx8_unpack(packed, T, H, st["values"].split(T))
        return st["values"]
    K, rows = c["topk"], st["rows"]
    per = [n * K for n in T]
    gc.gc_moe_combine_backward(st["dout"].split(T), st["expert_out"].split(rows), rows, st["dest"].split(per),
                               st["weights"].split(T), T, K, H, c["dtype"], st["dexpert"].split(rows), st["dweights"].split(T))
    return [st["dexpert"], st["dweights"]]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "pack": _pack_plain, "combine_bwd": _combine_bwd_plain,
            "ffn": _ffn_plain, "ffn_bwd": _ffn_bwd_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, H = case["op"], case["hidden"]
    if op in ("ffn", "ffn_bwd"):
        R, F = case["rows"], case["inter"]
        experts = min(R, case["ranks"] * case["experts"])
        w = 3 * experts * H * F * 2
        x = R * (_row8(H) if case["x"] == "mx8" else 2 * H)
        saved = {"none": 0, "bf16": R * 4 * F, "mx8": R * _row8(2 * F)}[case["saved"]]
        if op == "ffn":
            values = R * (_row8(2 * F) + 4 * F) if case["saved"] == "mx8" else 0   # read back as values
            return {"bytes": x + w + saved + R * 2 * H + values, "flops": 6 * R * H * F}
        return {"bytes": x + saved + w + R * 4 * H + 3 * case["ranks"] * case["experts"] * H * F * 2, "flops": 12 * R * H * F}
    A, e = sum(_sizes(case["tokens"], case["ranks"])), SIZE[case["dtype"]]
    N = case["ranks"]
    if op == "norm":
        y = 2 * _row8(H) + 2 * H if case["out"] == "mx8" else e * H
        return {"bytes": A * (3 * e * H + y + 4) + N * H * e, "flops": 6 * A * H}
    if op == "norm_bwd":
        return {"bytes": A * (4 * e * H + 4) + N * H * (e + 4), "flops": 10 * A * H}
    if op == "pack":
        return {"bytes": A * (e * H + 2 * _row8(H) + 2 * H), "flops": 3 * A * H}
    K = case["topk"]
    return {"bytes": A * (e * H * (1 + 2 * K) + K * 16), "flops": 3 * A * K * H}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact8(v):
    """What 8-bit rows stand for, from the definition: nearest multiple of the e4m3 spacing, ties to even."""
    T, n = v.shape
    out = torch.empty_like(v)
    for b in range(0, n, 32):
        p = v[:, b:b + 32]
        a = p.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / 448.0))
        e = e - (a <= 448.0 * torch.exp2(e - 1)).to(e.dtype) + (a > 448.0 * torch.exp2(e)).to(e.dtype)
        s = torch.exp2(torch.where(a > 0, e, torch.full_like(e, -117)).clamp(-117, 120))
        z = p / s
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, b:b + 32] = torch.round(z / step) * step * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, H, N = case["op"], case["hidden"], case["ranks"]
    if op in ("ffn", "ffn_bwd"):
        F = case["inter"]
        value = lambda v, n: _values8(v, n).double() if v.dtype == torch.uint8 else v.double()  # noqa: E731
        x = value(st["x"], H)
        flat = {k: st[k].view(-1, *st[k].shape[2:]) for k in ("w_gate", "w_up", "w_down")}
        grads = {k: torch.zeros(v.shape, dtype=torch.float64, device=DEV) for k, v in flat.items()} if op == "ffn_bwd" else {}
        outs, saves, at = [], [], 0
        for i, n in enumerate(st["counts"]):
            if not n:
                continue
            xs, rows = x[at:at + n], slice(at, at + n)
            at += n
            wg, wu, wd = (flat[k][i].double() for k in ("w_gate", "w_up", "w_down"))
            if op == "ffn":
                g, u = xs @ wg.T, xs @ wu.T
                outs.append((g / (1 + torch.exp(-g)) * u) @ wd.T)
                saves.append(torch.cat([g, u], 1))
                continue
            sv = value(st["saved"][rows], 2 * F)
            g, u, dy = sv[:, :F], sv[:, F:], st["dy"][rows].double()
            sg = 1 / (1 + torch.exp(-g))
            dh = dy @ wd
            dg, du = dh * u * (sg + g * sg * (1 - sg)), dh * g * sg
            outs.append(dg @ wg + du @ wu)
            grads["w_gate"][i], grads["w_up"][i], grads["w_down"][i] = dg.T @ xs, du.T @ xs, dy.T @ (g * sg * u)
        y = torch.cat(outs)
        if op == "ffn_bwd":
            return [y] + [grads[k].view(st[k].shape) for k in ("w_gate", "w_up", "w_down")]
        if case["saved"] == "none":
            return [y]
        saved = torch.cat(saves)
        return [y, _exact8(saved) if case["saved"] == "mx8" else saved]
    T = st["tokens"]
    parts = [slice(sum(T[:r]), sum(T[:r + 1])) for r in range(N)]
    if op == "norm":
        s = (st["x"].double() + st["residual"].double()).to(st["sum"].dtype)
        v = s.double()
        r = 1 / torch.sqrt((v * v).sum(1) / H + EPS)
        for k, p in enumerate(parts):
            v[p] *= r[p, None] * st["weight"][k].double()
        return [_exact8(v) if case["out"] == "mx8" else v, s.double(), r]
    if op == "norm_bwd":
        dx = torch.empty(sum(T), H, dtype=torch.float64, device=DEV)
        dw = torch.zeros(N, H, dtype=torch.float64, device=DEV)
        for k, p in enumerate(parts):
            s, r, dy = st["sum"][p].double(), st["rstd"][p].double()[:, None], st["dy"][p].double()
            d = dy * st["weight"][k].double()
            dx[p] = r * d - s * r ** 3 * (d * s).sum(1, keepdim=True) / H + st["dsum"][p].double()
            dw[k] = (dy * s * r).sum(0)
        return [dx, dw]
    if op == "pack":
        return _exact8(st["x"].double())
    K = case["topk"]
    start = [sum(st["rows"][:r]) for r in range(N)]
    row = torch.tensor(start, device=DEV)[st["dest"][:, 0].long()] + st["dest"][:, 1]
    de = torch.zeros(st["expert_out"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(st["weights"].shape, dtype=torch.float64, device=DEV)
    dout = st["dout"].double()
    for k in range(K):
        at = row.view(-1, K)[:, k]
        de[at] = st["weights"][:, k:k + 1].double() * dout
        dw[:, k] = (dout * st["expert_out"][at].double()).sum(1)
    return [de, dw]
