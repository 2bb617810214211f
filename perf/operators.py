"""Layer norm, low-rank adapters beside an N:M projection, and cross entropy
over a large vocabulary: the cases they are timed on, their plain forms and
their values in 64 bits.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where `own` is true, with the calls that
a user of structured_sparse_gemm_nm_amd makes.  `exact` gives the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
PATTERNS = {"2:4": (2, 4), "1:4": (1, 4), "1:8": (1, 8)}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the norm in front of a projection for one generated token
        dict(name="norm_token", op="norm", train=False, T=1, H=4096, dtype="bf16"),
        # a batch of 64 images' tokens before the first MLP product of a vision transformer
        dict(name="norm_images", op="norm", train=False, T=12608, H=768, dtype="f16"),
        # an odd width whose rows are not aligned, forward and backward
        dict(name="norm_train_odd", op="norm", train=True, T=1999, H=1543, dtype="f16"),
        # a training batch through the norm and back
        dict(name="norm_train", op="norm", train=True, T=8192, H=4096, dtype="bf16"),
        # one request generating one token with its adapter on a square projection
        dict(name="adapter_token", op="adapter", train=False, T=1, R=4096, K=4096, pattern="2:4", rank=16,
             adapters=8, requests=1, dtype="bf16", out="bf16"),
        # sixteen requests generating together, each with its own adapter, on an up projection
        dict(name="adapter_decode", op="adapter", train=False, T=16, R=11008, K=4096, pattern="2:4", rank=16,
             adapters=24, requests=16, dtype="bf16", out="bf16"),
        # prompts of several requests in one batch, ragged, some without an adapter
        dict(name="adapter_prefill", op="adapter", train=False, T=1999, R=4096, K=4096, pattern="2:4", rank=24,
             adapters=8, requests=7, dtype="bf16", out="bf16"),
        # four adapters trained in one batch over the frozen packed weight
        dict(name="adapter_train", op="adapter", train=True, T=2048, R=4096, K=4096, pattern="2:4", rank=32,
             adapters=4, requests=8, dtype="bf16", out="bf16"),
        # the log-probabilities of a few tokens
        dict(name="xent_score_few", op="xent", train=False, T=7, V=32000, H=4096, dtype="bf16"),
        # the perplexity of a text, a vocabulary of odd size
        dict(name="xent_score", op="xent", train=False, T=2048, V=32003, H=4096, dtype="f16"),
        # a training step's head and loss
        dict(name="xent_train", op="xent", train=True, T=2048, V=32000, H=4096, dtype="bf16"),
        # the same over a large vocabulary and a larger batch
        dict(name="xent_train_large", op="xent", train=True, T=4096, V=128000, H=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "adapter", "adapter", "xent"])
    if op == "norm":
        while True:
            T, H = _log(rng, 1, 16384), _log(rng, 64, 16384)
            if T * H <= 8192 * 4096:
                break
        return dict(op=op, train=rng.random() < 0.5, T=T, H=H, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "adapter":
        train = rng.random() < 0.4
        T = _log(rng, 1, 2048)
        R = _log(rng, 256, 11008)
        K = 32 * _log(rng, 8, 344)
        if train:
            R = (R + 7) // 8 * 8
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, train=train, T=T, R=R, K=K, pattern=rng.choice(["2:4", "2:4", "1:4", "1:8"]),
                    rank=_log(rng, 4, 64), adapters=_log(rng, 1, 32), requests=min(T, _log(rng, 1, 32)),
                    dtype=dtype, out=rng.choice([dtype, "f32"]))
    return dict(op=op, train=rng.random() < 0.5, T=_log(rng, 1, 4096), V=_log(rng, 1000, 128000),
                H=16 * _log(rng, 16, 256), dtype=rng.choice(["bf16", "f16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


def _pack(w, n, m):
    """Packed N:M form of w [R, K]: the n largest magnitudes of every m, ascending
    positions, and the positions as a little-endian bit stream a row."""
    R, K = w.shape
    g = w.view(R, K // m, m)
    pos = g.abs().float().topk(n, dim=2).indices.sort(dim=2).values
    values = g.gather(2, pos).reshape(R, K // m * n)
    pos = pos.reshape(R, -1)
    bits = 3 if m == 8 else 2
    stream = ((pos.unsqueeze(2) >> torch.arange(bits, device=w.device)) & 1).reshape(R, -1).to(torch.uint8)
    words = (stream.shape[1] + 31) // 32
    stream = torch.nn.functional.pad(stream, (0, words * 32 - stream.shape[1])).view(R, words, 32)
    idx = torch.zeros((R, words), dtype=torch.int64, device=w.device)
    for i in range(32):
        idx |= stream[:, :, i].long() << i
    idx = torch.where(idx >= 2 ** 31, idx - 2 ** 32, idx)
    return values.contiguous(), idx.to(torch.int32)


def _request_lengths(gen, tokens, requests):
    """Ragged lengths, at least one token each, that add up to `tokens`."""
    share = torch.rand(requests, generator=gen, device="cuda").cpu().double() + 0.1
    length = (share / share.sum() * (tokens - requests)).long() + 1
    length[0] += tokens - int(length.sum())
    return length


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # activations with a per-token offset and a few outlying channels
        x = torch.randn((T, H), generator=gen, device="cuda") + torch.randn((T, 1), generator=gen, device="cuda")
        x[:, :: 97] *= 8
        s.update(x=x.to(dt), w=(1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dt),
                 b=_normal(gen, (H,), 0.1, dt))
        if case["train"]:
            s["dy"] = _normal(gen, (T, H), 1.0, dt)
        return s
    if case["op"] == "adapter":
        T, R, K, r, na = case["T"], case["R"], case["K"], case["rank"], case["adapters"]
        n, m = PATTERNS[case["pattern"]]
        values, idx = _pack(_normal(gen, (R, K), 0.02, dt), n, m)
        length = _request_lengths(gen, T, case["requests"])
        # every eighth request or so runs without an adapter (-1)
        which = torch.randint(0, na, (case["requests"],), generator=gen, device="cuda")
        bare = torch.rand(case["requests"], generator=gen, device="cuda") < 0.12
        which = torch.where(bare, torch.full_like(which, -1), which)
        adapter = torch.repeat_interleave(which, length.cuda()).to(torch.int32)
        s.update(values=values, idx=idx, adapter=adapter, act=_normal(gen, (T, K), 1.0, dt),
                 A=_normal(gen, (na, r, K), K ** -0.5, dt), B=_normal(gen, (na, R, r), 0.1, dt),
                 scale=(16.0 / r) * (0.5 + torch.rand(na, generator=gen, device="cuda")))
        if case["train"]:
            s["G"] = _normal(gen, (T, R), 0.05, dt)
        return s
    T, V, H = case["T"], case["V"], case["H"]
    s.update(x=_normal(gen, (T, H), 1.0, dt), w=_normal(gen, (V, H), 2 * H ** -0.5, dt))
    labels = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # prompts and padding carry no loss
    skip = torch.rand(T, generator=gen, device="cuda") < 0.1
    s["labels"] = torch.where(skip, torch.full_like(labels, IGNORE), labels).to(torch.int32)
    if case["train"]:
        valid = int((~skip).sum())
        s["dloss"] = torch.full((T,), 1.0 / max(valid, 1), device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _RUN_OWN[state["case"]["op"]](state)
    return _RUN_PLAIN[state["case"]["op"]](state)


def _norm_plain(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = ((d * d).mean(1, keepdim=True) + EPS).rsqrt()
    xh = d * rstd
    y = (xh * w + b).to(s["x"].dtype)
    if not s["case"]["train"]:
        return y
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return y, dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _unpack_plain(values, idx, K, n, m):
    R, S = values.shape
    bits = 3 if m == 8 else 2
    first = torch.arange(S, device=values.device) * bits
    word, off = first >> 5, first & 31
    stream = torch.nn.functional.pad(idx.long() & 0xFFFFFFFF, (0, 1))
    pos = ((stream[:, word] >> off) | (stream[:, word + 1] << (32 - off))) & (m - 1)
    dense = torch.zeros((R, K // m, m), device=values.device)
    dense.scatter_(2, pos.view(R, K // m, n), values.float().view(R, K // m, n))
    return dense.view(R, K)


def _adapter_plain(s):
    c = s["case"]
    na, r, K = s["A"].shape
    T, R = c["T"], c["R"]
    n, m = PATTERNS[c["pattern"]]
    W = _unpack_plain(s["values"], s["idx"], K, n, m)
    x = s["act"].float()
    A = s["A"].float().view(na * r, K)
    B = s["B"].float().permute(0, 2, 1).reshape(na * r, R)
    # every token against every adapter, and only its own kept
    mine = s["adapter"].view(T, 1) == torch.arange(na, device=x.device, dtype=torch.int32)
    mine = mine.repeat_interleave(r, 1)
    weight = s["scale"].repeat_interleave(r)
    zero = torch.zeros((), device=x.device)
    xa = torch.where(mine, x @ A.t(), zero)
    y = x @ W.t() + (xa * weight) @ B
    out = DTYPES[c["out"]]
    if not c["train"]:
        return y.to(out)
    g = s["G"].float()
    u = torch.where(mine, (g @ B.t()) * weight, zero)
    dx = g @ W + u @ A
    dA = (u.t() @ x).view(na, r, K)
    dB = (g.t() @ (xa * weight)).view(R, na, r).permute(1, 0, 2).contiguous()
    return y.to(out), dx.to(out), dA, dB


def _xent_plain(s):
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"].long()
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    e = (logits - top).exp()
    total = e.sum(1, keepdim=True)
    lse = (total.log() + top).squeeze(1)
    keep = (labels >= 0) & (labels < w.shape[0])
    at = labels.clamp(0, w.shape[0] - 1).unsqueeze(1)
    zero = torch.zeros((), device=x.device)
    loss = torch.where(keep, lse - logits.gather(1, at).squeeze(1), zero)
    if not s["case"]["train"]:
        return loss, lse
    d = e / total
    d.scatter_add_(1, at, torch.full_like(lse, -1.0).unsqueeze(1))
    d = torch.where(keep.unsqueeze(1), d * s["dloss"].unsqueeze(1), zero)
    return loss, lse, (d @ w).to(s["x"].dtype), (d.t() @ x).to(s["w"].dtype)


def _norm_own(s):
    import structured_sparse_gemm_nm_amd as nm
    if not s["case"]["train"]:
        return nm.nm_layernorm(s["x"], s["w"], s["b"], eps=EPS)
    y, mean, rstd = nm.nm_layernorm(s["x"], s["w"], s["b"], eps=EPS, stats=True)
    dx, dw, db = nm.nm_layernorm_bwd(s["dy"], s["x"], mean, rstd, s["w"])
    return y, dx, dw, db


def _adapter_own(s):
    import structured_sparse_gemm_nm_amd as nm
    c = s["case"]
    n, m = PATTERNS[c["pattern"]]
    out = DTYPES[c["out"]]
    y, xa = nm.nm_adapter_spmm(s["values"], s["idx"], s["act"], s["adapter"], s["A"], s["B"], s["scale"], c["K"],
                               n, m, out_dtype=out)
    if not c["train"]:
        return y
    dx, dA, dB = nm.nm_adapter_spmm_bwd(s["values"], s["idx"], s["G"], s["act"], xa, s["adapter"], s["A"], s["B"],
                                        s["scale"], c["K"], n, m, out_dtype=out)
    return y, dx, dA, dB


def _xent_own(s):
    import structured_sparse_gemm_nm_amd as nm
    loss, lse = nm.nm_xent(s["x"], s["w"], s["labels"], ignore_index=IGNORE)
    if not s["case"]["train"]:
        return loss, lse
    dx, dw = nm.nm_xent_bwd(s["x"], s["w"], s["labels"], lse, s["dloss"], ignore_index=IGNORE,
                            out_dtype=s["x"].dtype)
    return loss, lse, dx, dw


_RUN_PLAIN = {"norm": _norm_plain, "adapter": _adapter_plain, "xent": _xent_plain}
_RUN_OWN = {"norm": _norm_own, "adapter": _adapter_own, "xent": _xent_own}


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        fwd = dict(bytes=2 * T * H * e + 2 * H * e, flops=8 * T * H)
        if not case["train"]:
            return fwd
        # x and dy read, y and dx written, dw and db written
        return dict(bytes=4 * T * H * e + 2 * H * e + 8 * H, flops=22 * T * H)
    if case["op"] == "adapter":
        T, R, K, r = case["T"], case["R"], case["K"], case["rank"]
        n, m = PATTERNS[case["pattern"]]
        S = K // m * n
        packed = R * S * 2 + R * ((S * (3 if m == 8 else 2) + 31) // 32) * 4
        used = min(case["requests"], case["adapters"])
        o = 4 if case["out"] == "f32" else 2
        b = packed + used * r * (K + R) * 2 + T * K * 2 + T * R * o + 4 * T
        f = 2 * T * R * S + 2 * T * r * (K + R)
        if case["train"]:
            # G read, dX written, dA and dB written whole
            b += T * R * 2 + T * K * o + case["adapters"] * r * (K + R) * 4
            f += 2 * T * R * K + 4 * T * r * (K + R)
        return dict(bytes=b, flops=f)
    T, V, H = case["T"], case["V"], case["H"]
    b, f = (T + V) * H * 2 + 12 * T, 2 * T * V * H
    if case["train"]:
        b, f = b + (T + V) * H * 2 + 4 * T, 3 * f
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------------------
# the same outputs in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "adapter": _adapter_exact, "xent": _xent_exact}[case["op"]](s)


def _norm_exact(s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    H = x.shape[1]
    mu = x.sum(1) / H
    sd = ((x - mu[:, None]).square().sum(1) / H + EPS).sqrt()
    xh = (x - mu[:, None]) / sd[:, None]
    y = torch.addcmul(b, xh, w)
    if not s["case"]["train"]:
        return y
    dy = s["dy"].double()
    gw = dy * w
    # the projection of gw onto the complement of (1, xh), over the deviation
    dx = (gw - gw.sum(1, keepdim=True) / H - xh * ((gw * xh).sum(1, keepdim=True) / H)) / sd[:, None]
    return y, dx, torch.einsum("th,th->h", dy, xh), torch.einsum("th->h", dy)


def _adapter_exact(s):
    c = s["case"]
    n, m = PATTERNS[c["pattern"]]
    R, K, T = c["R"], c["K"], c["T"]
    bits = 3 if m == 8 else 2
    # the stream bit by bit: survivor j's position is bits [j*bits, j*bits + bits)
    words = s["idx"].long() & 0xFFFFFFFF
    W = torch.zeros((R, K), dtype=torch.float64, device="cuda")
    S = s["values"].shape[1]
    j = torch.arange(S, device="cuda")
    pos = torch.zeros((R, S), dtype=torch.int64, device="cuda")
    for i in range(bits):
        at = j * bits + i
        pos |= ((words[:, at // 32] >> (at % 32)) & 1) << i
    W.scatter_(1, pos + (j // n * m), s["values"].double())
    x = s["act"].double()
    y = x @ W.t()
    ids = s["adapter"].cpu().tolist()
    rows = {a: torch.tensor([t for t in range(T) if ids[t] == a], device="cuda") for a in sorted(set(ids)) if a >= 0}
    A, B, scale = s["A"].double(), s["B"].double(), s["scale"].double()
    for a, at in rows.items():
        y[at] += scale[a] * ((x[at] @ A[a].t()) @ B[a].t())
    if not c["train"]:
        return y
    g = s["G"].double()
    dx = g @ W
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a, at in rows.items():
        u = scale[a] * (g[at] @ B[a])
        dx[at] += u @ A[a]
        dA[a] = u.t() @ x[at]
        dB[a] = scale[a] * (g[at].t() @ (x[at] @ A[a].t()))
    return y, dx, dA, dB


def _xent_exact(s):
    x, w, labels = s["x"].double(), s["w"].double(), s["labels"].long()
    T, V = x.shape[0], w.shape[0]
    train = s["case"]["train"]
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dx, dw = (torch.zeros_like(x), torch.zeros_like(w)) if train else (None, None)
    for t0 in range(0, T, 512):
        at = slice(t0, min(t0 + 512, T))
        logits = x[at] @ w.t()
        lse[at] = torch.logsumexp(logits, 1)
        lab = labels[at]
        keep = (lab != IGNORE).double()
        hot = torch.zeros_like(logits)
        hot[torch.arange(lab.shape[0], device="cuda"), lab.clamp(min=0)] = keep
        loss[at] = lse[at] * keep - (hot * logits.nan_to_num()).sum(1)
        if train:
            d = torch.exp(logits - lse[at, None]) * keep[:, None] - hot
            d *= s["dloss"][at, None].double()
            dx[at] = d @ w
            dw += d.t() @ x[at]
    return (loss, lse, dx, dw) if train else (loss, lse)
