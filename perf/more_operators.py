"""Cases of the two ends of a training step: embedding, dropout, token log probabilities.

Every case is one call a training or serving step makes on the N rank buffers
of one GPU.  With `own` false, run() computes the operators from elementary
torch operations in 32 bits; with `own` true, it calls the library.

  embed        out[t] = scale * weight[token t]
  embed_bwd    the weight's gradient: rows of dout summed by token
  dropout      y = residual + x * keep / (1 - p), keep from a counter-based generator
  logprob      log probability of a given token, entropy, the largest alternatives
  loss         logprob without alternatives, and the gradient of the logits from
               those of log probability and entropy: in the same call where they are
               known before it, in a second one where they depend on its results
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a serving step, vocabulary and hidden size of the repository's transformer
        {"name": "embed_one_token", "op": "embed", "ranks": 1, "tokens": 1, "hidden": 4096, "vocab": 32000, "dtype": "bf16",
         "scale": 1.0, "skew": 1.1},
        # the expert-parallel workload's 8 x 16384 tokens through the transformer's embedding, scaled by sqrt(hidden)
        {"name": "embed_8x16384", "op": "embed", "ranks": 8, "tokens": 16384, "hidden": 4096, "vocab": 32000,
         "dtype": "bf16", "scale": 64.0, "skew": 1.1},
        # a short fp32 batch with an odd row length
        {"name": "embed_bwd_fp32_odd", "op": "embed_bwd", "ranks": 3, "tokens": 517, "hidden": 999, "vocab": 1013,
         "dtype": "fp32", "grad": "fp32", "scale": 1.0, "skew": 1.1},
        # the gradient of the first tensor of the 7B set, on each of its 8 ranks
        {"name": "embed_bwd_8x16384", "op": "embed_bwd", "ranks": 8, "tokens": 16384, "hidden": 4096, "vocab": 32000,
         "dtype": "bf16", "grad": "bf16", "scale": 64.0, "skew": 1.1},
        # a short fp32 batch whose length is no multiple of anything
        {"name": "dropout_fp32_odd", "op": "dropout", "ranks": 2, "tokens": 257, "hidden": 1001, "dtype": "fp32", "p": 0.25,
         "residual": True},
        # the residual stream of the expert-parallel workload's tokens
        {"name": "dropout_8x16384", "op": "dropout", "ranks": 8, "tokens": 16384, "hidden": 4096, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # one sampled token with its alternatives, at a temperature
        {"name": "logprob_one_token", "op": "logprob", "ranks": 1, "tokens": 1, "vocab": 131072, "pad": 0, "dtype": "bf16",
         "scale": 1.25, "top": 20, "banned": 0.0},
        # a serving batch, fp32 logits, an odd vocabulary in padded rows, part of it banned
        {"name": "logprob_64_padded", "op": "logprob", "ranks": 1, "tokens": 64, "vocab": 32003, "pad": 61, "dtype": "fp32",
         "scale": 1.0, "top": 5, "banned": 0.3},
        # sequences scored with their alternatives, kept to train another model on
        {"name": "logprob_4x2048_top5", "op": "logprob", "ranks": 4, "tokens": 2048, "vocab": 32000, "pad": 0, "dtype": "bf16",
         "scale": 1.0, "top": 5, "banned": 0.0},
        # a small fp32 model's loss and gradient, odd rows
        {"name": "loss_fp32_odd", "op": "loss", "ranks": 2, "tokens": 37, "vocab": 1003, "pad": 0, "dtype": "fp32",
         "scale": 1.0, "entropy": False, "known": True, "banned": 0.0},
        # the loss of a training step with an entropy term, and its gradient, on 8 ranks
        {"name": "loss_8x4096", "op": "loss", "ranks": 8, "tokens": 4096, "vocab": 32000, "pad": 0, "dtype": "bf16",
         "scale": 1.0, "entropy": True, "known": True, "banned": 0.0},
        # a policy's update at a temperature: the weights follow from the log probabilities; a large vocabulary
        {"name": "policy_2x1024", "op": "loss", "ranks": 2, "tokens": 1024, "vocab": 131072, "pad": 0, "dtype": "bf16",
         "scale": 1.25, "entropy": True, "known": False, "banned": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "embed_bwd", "dropout", "logprob", "logprob", "loss"])
    ranks = rng.randint(1, 8)
    c = {"op": op, "ranks": ranks, "tokens": _log(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    if op in ("embed", "embed_bwd", "dropout"):
        c["hidden"] = _log(rng, 8, 8192)
        if rng.random() < 0.6:
            c["hidden"] = max(8, c["hidden"] // 8 * 8)
    if op == "dropout":
        c.update(p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5)
        c["tokens"] = max(1, min(c["tokens"], (1 << 28) // (ranks * c["hidden"])))
        return c
    c["vocab"] = _log(rng, 64, 131072)
    if op in ("embed", "embed_bwd"):
        c["vocab"] = max(64, min(c["vocab"], (1 << 29) // (ranks * c["hidden"])))
        c["tokens"] = max(1, min(c["tokens"], (1 << 28) // (ranks * c["hidden"])))
        c.update(scale=rng.choice([1.0, 1.0, round(c["hidden"] ** 0.5, 3)]), skew=rng.choice([0.0, 0.7, 1.1]))
        if op == "embed_bwd":
            c["grad"] = rng.choice(["bf16", "fp32"])
        return c
    c["tokens"] = max(1, min(c["tokens"], (1 << 28) // (ranks * c["vocab"])))
    c.update(pad=rng.choice([0, 0, 8, rng.randint(1, 63)]), scale=rng.choice([1.0, 1.0, 0.7, 1.25]),
             banned=rng.choice([0.0, 0.0, 0.3]))
    if op == "logprob":
        c["top"] = rng.choice([0, 1, 5, 20, 64])
    else:
        c.update(entropy=rng.random() < 0.5, known=rng.random() < 0.5)
    return c


def _sizes(n, ranks):
    """Tokens of each rank: full on the first, a few fewer on each later one of short batches."""
    return [max(0, n - 3 * r if n < 4096 else n) for r in range(ranks)]


def _elements(case):
    return [t * case["hidden"] for t in _sizes(case["tokens"], case["ranks"])]


# ------------------------------------------------------------------ inputs

def _normal(g, *shape, dtype, scale=1.0):
    return torch.empty(*shape, dtype=dtype, device=DEV).normal_(0, scale, generator=g)


def _zipf_tokens(g, n, vocab, skew):
    """n tokens, P(k-th most frequent) ~ k^-skew, the most frequent ones spread over the vocabulary; one in 64 is padding (-1)."""
    w = torch.arange(1, vocab + 1, dtype=torch.float64, device=DEV).pow(-skew).cumsum(0)
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64) * w[-1]
    k = torch.searchsorted(w, u).clamp(max=vocab - 1)
    ids = torch.randperm(vocab, generator=g, device=DEV)[k].to(torch.int32)
    return torch.where(torch.rand(n, generator=g, device=DEV) < 1 / 64, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    N, T, t = case["ranks"], _sizes(case["tokens"], case["ranks"]), TYPES[case["dtype"]]
    A = sum(T)
    st = {"case": dict(case), "tokens": T}
    if case["op"] in ("embed", "embed_bwd"):
        V, H = case["vocab"], case["hidden"]
        st["ids"] = _zipf_tokens(g, A, V, case["skew"])
        if case["op"] == "embed":
            st["weight"] = _normal(g, N, V, H, dtype=t, scale=0.02)
            st["out"] = torch.empty(A, H, dtype=t, device=DEV)
        else:
            st["dout"] = _normal(g, A, H, dtype=t, scale=1e-3)
            st["dweight"] = torch.empty(N, V, H, dtype=TYPES[case["grad"]], device=DEV)
        return st
    if case["op"] == "dropout":
        n = A * case["hidden"]
        st["x"] = _normal(g, n, dtype=t)
        st["residual"] = _normal(g, n, dtype=t, scale=2.0) if case["residual"] else None
        st["y"] = torch.empty(n, dtype=t, device=DEV)
        st["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64)
        st["offset"] = seed % 7                                        # which of the step's dropouts
        st["step"] = torch.tensor([seed * 3 + 5], dtype=torch.int64, device=DEV)
        return st
    V, S = case["vocab"], case["vocab"] + case["pad"]
    # logits of a trained model: a few likely tokens far above the rest
    st["logits"] = _normal(g, A, S, dtype=t, scale=2.0)
    hot = torch.randint(0, V // 4, (A, 4), generator=g, device=DEV) + torch.arange(4, device=DEV) * (V // 4)
    st["logits"].scatter_add_(1, hot, _normal(g, A, 4, dtype=t, scale=3.0) + 9)
    if case["banned"]:
        for p in st["logits"].split(4096):
            p.masked_fill_(torch.rand(p.shape, generator=g, device=DEV) < case["banned"], float("-inf"))
    at = torch.randint(0, V, (A,), generator=g, device=DEV)
    at = torch.where(torch.rand(A, generator=g, device=DEV) < 0.5, hot[:, 0], at)
    skip = torch.rand(A, generator=g, device=DEV) < 1 / 16
    st["targets"] = torch.where(skip, torch.full_like(at, -1), at).to(torch.int32)
    f = dict(dtype=torch.float32, device=DEV)
    st["logprob"], st["entropy"], st["lse"] = (torch.empty(A, **f) for _ in range(3))
    if case["op"] == "logprob":
        K = st["case"]["top"] = min(case["top"], V)
        st["top_ids"], st["top_logprob"] = torch.empty(A, K, dtype=torch.int32, device=DEV), torch.empty(A, K, **f)
        return st
    n = max(1, int((~skip).sum()))
    st["dlogprob"] = torch.rand(A, generator=g, device=DEV) * (-2.0 / n)
    st["dentropy"] = torch.full((A,), -0.01 / n, **f) if case["entropy"] else None
    st["dlogits"] = torch.empty(A, S, dtype=t, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _rank_of_rows(T):
    return torch.repeat_interleave(torch.arange(len(T), device=DEV), torch.tensor(T, device=DEV), output_size=sum(T))


def _embed_plain(st):
    c = st["case"]
    ids = st["ids"].long()
    ok = (ids >= 0) & (ids < c["vocab"])
    rows = st["weight"].view(-1, c["hidden"])[_rank_of_rows(st["tokens"]) * c["vocab"] + torch.where(ok, ids, 0)]
    return torch.where(ok[:, None], rows.float() * c["scale"], 0.0).to(rows.dtype)


def _embed_bwd_plain(st):
    c = st["case"]
    N, V, H = c["ranks"], c["vocab"], c["hidden"]
    out = []
    for r, (ids, dout) in enumerate(zip(st["ids"].split(st["tokens"]), st["dout"].split(st["tokens"]))):
        i = ids.long()
        row = torch.where((i >= 0) & (i < V), i, V)                   # padding adds to a row that is dropped
        dw = torch.zeros(V + 1, H, dtype=torch.float32, device=DEV)
        dw.index_add_(0, row, dout.float())
        out.append((dw[:V] * c["scale"]).to(st["dweight"].dtype))
    return torch.stack(out)


def _philox(seed, c0, c1, c2, c3):
    """Philox4x32-10: counter words (int64 tensors of 32-bit values) to four random words."""
    M = 0xFFFFFFFF
    k0, k1 = seed & M, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57                        # 64-bit products, wrapped: every bit is right
        c0, c1, c2, c3 = (b >> 32 & M) ^ c1 ^ k0, b & M, (a >> 32 & M) ^ c3 ^ k1, a & M
        k0, k1 = (k0 + 0x9E3779B9) & M, (k1 + 0xBB67AE85) & M
    return c0, c1, c2, c3


def _drop_at(p):
    return int(math.floor(p * 65536 + 0.5))


def _dropout_plain(st):
    c = st["case"]
    drop = _drop_at(c["p"])
    at = st["offset"] + st["step"]                                     # stays on the device, as a captured step needs it
    keeps = []
    for r, n in enumerate(_elements(c)):
        b = torch.arange(-(-n // 8), dtype=torch.int64, device=DEV)    # a block of 8 values
        words = _philox(st["seed"], b & 0xFFFFFFFF, (b >> 32) | r << 8, (at & 0xFFFFFFFF).expand_as(b),
                        (at >> 32 & 0xFFFFFFFF).expand_as(b))
        u = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 1)
        keeps.append((u >= drop).view(-1)[:n])
    scale = 65536.0 / (65536 - drop) if drop < 65536 else 0.0
    v = torch.where(torch.cat(keeps), st["x"].float() * scale, 0.0)
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(st["x"].dtype)


def _logprob_plain(st):
    c = st["case"]
    V, K = c["vocab"], c.get("top", 0)
    out = []
    for x, targets in zip(st["logits"].split(8192), st["targets"].split(8192)):
        x = x[:, :V].float()
        z = x * c["scale"]
        m = z.amax(1, keepdim=True)
        m = torch.where(m == float("-inf"), 0.0, m)
        e = torch.exp(z - m)
        s = e.sum(1)
        log_s = torch.log(s)
        lse = m[:, 0] + log_s
        u = torch.where(e > 0, e * (z - m), 0.0).sum(1)
        entropy = torch.where(s > 0, log_s - u / s, 0.0)
        i = targets.long()
        ok = (i >= 0) & (i < V)
        zt = z.gather(1, torch.where(ok, i, 0)[:, None])[:, 0]
        lp = torch.where(ok, torch.where(s > 0, zt - m[:, 0] - log_s, float("-inf")), 0.0)
        row = [lp, entropy, lse]
        if K:
            bits = (x + 0.0).view(torch.int32).long()                  # an order of 64-bit keys: value, then lowest token
            key = torch.where(bits < 0, ~bits, bits | 0x80000000)
            key = (key << 20) | (V - 1 - torch.arange(V, device=DEV))
            ids = V - 1 - (key.topk(K, dim=1).values & 0xFFFFF)
            zt = z.gather(1, ids)
            tl = torch.where((s > 0)[:, None], zt - m - log_s[:, None], float("-inf"))
            row += [ids.to(torch.int32), tl]
        out.append(row)
    return [torch.cat(p) for p in zip(*out)]


def _loss_plain(st):
    c = st["case"]
    V = c["vocab"]
    logprob, entropy, lse = _logprob_plain(st)
    out = torch.zeros_like(st["logits"])
    for k in range(0, out.shape[0], 8192):
        r = slice(k, k + 8192)
        z = st["logits"][r, :V].float() * c["scale"]
        some = lse[r, None] > float("-inf")
        d = torch.where(some, z - lse[r, None], float("-inf"))
        p = torch.exp(d)
        i = st["targets"][r].long()
        ok = (i >= 0) & (i < V) & some[:, 0]
        dlp = torch.where(ok, st["dlogprob"][r], 0.0)[:, None]
        dz = -dlp * p
        if st["dentropy"] is not None:
            dz = dz - torch.where(p > 0, st["dentropy"][r, None] * p * (d + entropy[r, None]), 0.0)
        dz.scatter_add_(1, torch.where(ok, i, 0)[:, None], dlp)
        out[r, :V] = (dz * c["scale"]).to(out.dtype)
    return [logprob, entropy, lse, out]


# ------------------------------------------------------------------ the library's calls

def _run_own(st):
    import collective_communication_reduction_amd as gc

    c, T = st["case"], st["tokens"]
    op, N = c["op"], c["ranks"]
    if op == "embed":
        gc.gc_embedding(st["weight"].unbind(0), st["ids"].split(T), T, c["vocab"], c["hidden"], st["out"].split(T),
                        scale=c["scale"])
        return st["out"]
    if op == "embed_bwd":
        scratch = torch.empty(gc.gc_embedding_backward_scratch_bytes(T, c["vocab"], c["hidden"]), dtype=torch.uint8, device=DEV)
        gc.gc_embedding_backward(st["dout"].split(T), st["ids"].split(T), T, c["vocab"], c["hidden"],
                                 st["dweight"].unbind(0), scratch, scale=c["scale"])
        return st["dweight"]
    if op == "dropout":
        n = _elements(c)
        res = None if st["residual"] is None else st["residual"].split(n)
        gc.gc_dropout(st["x"].split(n), n, c["p"], st["seed"], st["y"].split(n), offset=st["offset"], step=st["step"],
                      residual=res)
        return st["y"]
    kw = dict(stride=c["vocab"] + c["pad"], scale=c["scale"])
    kw.update(targets=st["targets"].split(T))
    top = c.get("top", 0)
    scratch = torch.empty(gc.gc_token_logprob_scratch_bytes(T, c["vocab"], top), dtype=torch.uint8, device=DEV)
    logits, entropy, lse = st["logits"].split(T), st["entropy"].split(T), st["lse"].split(T)
    more = dict(top=top, top_ids=st["top_ids"].split(T), top_logprob=st["top_logprob"].split(T)) if top else {}
    if op == "loss":
        grads = dict(dlogprob=st["dlogprob"].split(T), dlogits=st["dlogits"].split(T))
        if c["entropy"]:
            grads.update(dentropy=st["dentropy"].split(T))
        if c["known"]:
            more = grads
    gc.gc_token_logprob(logits, T, c["vocab"], scratch, logprob=st["logprob"].split(T), entropy=entropy, lse=lse, **kw, **more)
    if op == "logprob":
        return [st[k] for k in ("logprob", "entropy", "lse") + (("top_ids", "top_logprob") if top else ())]
    if not c["known"]:
        gc.gc_token_logprob_backward(logits, T, c["vocab"], lse, entropy=entropy, **kw, **grads)
    return [st["logprob"], st["entropy"], st["lse"], st["dlogits"]]


def run(state):
    if own:
        return _run_own(state)
    return {"embed": _embed_plain, "embed_bwd": _embed_bwd_plain, "dropout": _dropout_plain, "logprob": _logprob_plain,
            "loss": _loss_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def _distinct(n, vocab, skew):
    """Expected number of distinct tokens among n of the inputs' distribution."""
    w = torch.arange(1, vocab + 1, dtype=torch.float64).pow(-skew)
    return int((1 - (1 - w / w.sum()).pow(n)).sum())


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    T = _sizes(case["tokens"], case["ranks"])
    A = sum(T)
    if op == "embed":
        H = case["hidden"]
        rows = sum(_distinct(n, case["vocab"], case["skew"]) for n in T)
        return {"bytes": A * (4 + e * H) + rows * e * H, "flops": A * H}
    if op == "embed_bwd":
        H = case["hidden"]
        return {"bytes": A * (4 + e * H) + case["ranks"] * case["vocab"] * H * SIZE[case["grad"]], "flops": A * H}
    if op == "dropout":
        n = A * case["hidden"]
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": n * 10}
    V = case["vocab"]
    if op == "logprob":
        K = min(case["top"], V)
        return {"bytes": A * (V * e + 16 + 8 * K), "flops": A * V * 8}
    # a gradient that has to wait for the results reads the logits again
    return {"bytes": A * (((2 if case["known"] else 3) * V + case["pad"]) * e + 28), "flops": A * V * 18}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_keep(n, rank, seed, at, drop):
    """keep of n values, from the generator's definition with products in 16-bit limbs."""
    M = (1 << 32) - 1
    def mul(a, k):                                                     # (high, low) words of a * k
        lo, hi = (a & 0xFFFF) * k, (a >> 16) * k                       # below 2^48
        mid = hi + (lo >> 16)
        return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)
    out = torch.empty((n + 7) // 8, 8, dtype=torch.bool, device=DEV)
    for first in range(0, out.shape[0], 1 << 24):
        b = torch.arange(first, min(out.shape[0], first + (1 << 24)), device=DEV)
        x = [b % (1 << 32), torch.div(b, 1 << 32, rounding_mode="floor") + 256 * rank,
             torch.full_like(b, at % (1 << 32)), torch.full_like(b, (at >> 32) % (1 << 32))]
        key = [seed % (1 << 32), seed >> 32]
        for _ in range(10):
            h0, l0 = mul(x[0], 0xD2511F53)
            h1, l1 = mul(x[2], 0xCD9E8D57)
            x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) & M, (key[1] + 0xBB67AE85) & M]
        for i in range(8):
            out[first:first + b.numel(), i] = torch.div(x[i // 2], 65536 ** (i % 2), rounding_mode="floor") % 65536 >= drop
    return out.view(-1)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    T, N, op = st["tokens"], case["ranks"], case["op"]
    parts = [slice(sum(T[:r]), sum(T[:r + 1])) for r in range(N)]
    if op == "embed":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
        for r, p in enumerate(parts):
            ids = st["ids"][p].long()
            ok = ids >= 0
            out[p][ok] = st["weight"][r][ids[ok]].double() * case["scale"]
        return out
    if op == "embed_bwd":
        out = torch.zeros(st["dweight"].shape, dtype=torch.float64, device=DEV)
        for r, p in enumerate(parts):
            ids, order = torch.sort(st["ids"][p])
            order = order[ids >= 0]
            ids = ids[ids >= 0]
            for k in range(0, case["hidden"], 512):                    # differences of running sums would lose digits
                out[r][:, k:k + 512].index_add_(0, ids.long(), st["dout"][p][order, k:k + 512].double() * case["scale"])
        return out
    if op == "dropout":
        n = _elements(case)
        drop = _drop_at(case["p"])
        at = st["offset"] + int(st["step"])
        out = []
        for r in range(N):
            p = slice(sum(n[:r]), sum(n[:r + 1]))
            v = st["x"][p].double() * (65536 / (65536 - drop))
            v[~_exact_keep(n[r], r, st["seed"], at, drop)] = 0
            out.append(v if st["residual"] is None else v + st["residual"][p].double())
        return torch.cat(out)
    V, c, outs = case["vocab"], case["scale"], []
    for k in range(0, sum(T), 2048):
        r = slice(k, k + 2048)
        x = st["logits"][r, :V].double()
        i = st["targets"][r].long()
        rows = torch.arange(len(i), device=DEV)
        lse = torch.logsumexp(x * c, 1)
        empty = lse == float("-inf")
        lp = torch.where(empty[:, None], float("-inf"), torch.log_softmax(x * c, 1))
        p = lp.exp()
        plp = torch.where(p > 0, p * lp, 0.0)
        entropy = -plp.sum(1)
        row = [torch.where(i >= 0, lp[rows, i.clamp(min=0)], 0.0), entropy, lse]
        if op == "logprob" and st["case"]["top"]:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :st["case"]["top"]]
            row += [ids, lp.gather(1, ids)]
        if op == "loss":
            g = torch.where((i >= 0) & ~empty, st["dlogprob"][r].double(), 0.0)
            dz = -g[:, None] * p
            dz[rows, i.clamp(min=0)] += g
            if case["entropy"]:
                dz -= st["dentropy"][r].double()[:, None] * (plp + p * entropy[:, None])
            row.append(torch.nn.functional.pad(dz * c, (0, case["pad"])))
        outs.append(row)
    return [torch.cat(p) for p in zip(*outs)]
