"""Products grouped by expert over packed N:M weights, microscaled 4-bit
quantisation and product, and the global norm and clipping of gradients: the
cases they are timed on, their plain forms and their values in 64 bits.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where `own` is true, with the calls that
a user of structured_sparse_gemm_nm_amd makes.  `exact` gives the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
PATTERNS = {"2:4": (2, 4), "1:4": (1, 4), "1:8": (1, 8)}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32                                     # values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token on its two experts of eight
        dict(name="experts_token", op="experts", train=False, T=2, E=8, used=2, R=4096, K=4096, pattern="2:4",
             dtype="bf16", out="bf16"),
        # sequences generating together, spread over many experts, few rows each
        dict(name="experts_decode", op="experts", train=False, T=96, E=64, used=41, R=2816, K=2048, pattern="1:4",
             dtype="f16", out="f16"),
        # prompts, ragged: every expert a different number of rows, one of them none
        dict(name="experts_prefill", op="experts", train=False, T=7999, E=8, used=7, R=4096, K=4096, pattern="2:4",
             dtype="bf16", out="bf16"),
        # a small layer of odd sizes, trained in fp16 with fp32 gradients
        dict(name="experts_train_odd", op="experts", train=True, T=1333, E=5, used=5, R=1000, K=1056, pattern="1:8",
             dtype="f16", out="f32"),
        # a training step of an expert layer with its pattern held
        dict(name="experts_train", op="experts", train=True, T=8192, E=16, used=16, R=4096, K=2048, pattern="2:4",
             dtype="bf16", out="bf16"),
        # one token's activations through four bits
        dict(name="mx_round_token", op="mx_round", T=1, K=4096, dtype="bf16"),
        # a weight through four bits, as training that looks ahead to them does
        dict(name="mx_round_weight", op="mx_round", T=11008, K=4096, dtype="f32"),
        # a few sequences generating on a 4-bit up projection
        dict(name="mx_decode", op="mx", T=7, E=0, used=0, R=11008, K=4096, dtype="bf16", out="bf16"),
        # a prompt on a 4-bit projection
        dict(name="mx_prefill", op="mx", T=4096, E=0, used=0, R=11008, K=4096, dtype="bf16", out="bf16"),
        # ragged rows of several experts held in four bits
        dict(name="mx_experts", op="mx", T=1999, E=8, used=7, R=2816, K=4096, dtype="f16", out="f16"),
        # the gradients of every layer's adapters, hundreds of small tensors
        dict(name="clip_adapters", op="clip", kind="adapters", layers=32, H=4096, F=0, rank=16, dtype="f32",
             max_norm=1.0),
        # the gradients of a model's packed weights and norms
        dict(name="clip_model", op="clip", kind="model", layers=8, H=4096, F=11008, rank=0, dtype="bf16",
             max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "experts", "mx_round", "mx", "mx", "clip"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "experts":
        train = rng.random() < 0.5
        while True:
            T, E = _log(rng, 1, 8192), _log(rng, 1, 64)
            R, K = _log(rng, 64, 4096), 32 * _log(rng, 4, 128)
            if E * R * K <= 8 * 4096 * 4096 and T * R * K * (2 if train else 1) <= 7999 * 4096 * 4096:
                break
        if train:
            R = (R + 7) // 8 * 8
        return dict(op=op, train=train, T=T, E=E, used=rng.randint(1, min(T, E)), R=R, K=K,
                    pattern=rng.choice(["2:4", "2:4", "1:4", "1:8"]), dtype=dtype, out=rng.choice([dtype, "f32"]))
    if op == "mx_round":
        while True:
            T, K = _log(rng, 1, 16384), 32 * _log(rng, 1, 352)
            if T * K <= 11008 * 4096:
                break
        return dict(op=op, T=T, K=K, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "mx":
        while True:
            T, R, K = _log(rng, 1, 4096), _log(rng, 64, 11008), 32 * _log(rng, 2, 352)
            E = rng.choice([0, 0, _log(rng, 1, 32)])
            if max(E, 1) * R * K <= 8 * 2816 * 4096 and T * R * K <= 4096 * 11008 * 4096:
                break
        return dict(op=op, T=T, E=E, used=rng.randint(1, min(T, E)) if E else 0, R=R, K=K, dtype=dtype,
                    out=rng.choice([dtype, "f32"]))
    kind = rng.choice(["adapters", "model", "ragged"])
    return dict(op=op, kind=kind, layers=_log(rng, 1, 16), H=8 * _log(rng, 8, 256), F=8 * _log(rng, 8, 700),
                rank=_log(rng, 1, 64), dtype=rng.choice(["bf16", "f16", "f32"]),
                max_norm=rng.choice([0.1, 1.0, 1e6]))


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


def _lengths(gen, T, E, used):
    """Rows of each of E experts, `used` of them with at least one, T in all."""
    share = torch.rand(used, generator=gen, device="cuda").cpu().double() + 0.05
    length = (share / share.sum() * (T - used)).long() + 1
    length[0] += T - int(length.sum())
    at = torch.randperm(E, generator=gen, device="cuda").cpu()[:used]
    out = torch.zeros(E, dtype=torch.int64)
    out[at] = length
    return out.tolist()


def _offsets(lengths):
    ends = [0]
    for n in lengths:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def _shapes(case):
    """(shape, type) of every gradient of a clip case."""
    dt, H, F, r = DTYPES[case["dtype"]], case["H"], case["F"], case["rank"]
    if case["kind"] == "adapters":      # A and B beside four projections
        layer = [((r, H), dt), ((H, r), dt)] * 4
    elif case["kind"] == "model":       # packed 2:4 weights, and norms in fp32
        layer = [((H, H // 2), dt)] * 4 + [((F, H // 2), dt)] * 2 + [((H, F // 2), dt)] + [((H,), torch.float32)] * 4
    else:                               # odd counts, single values and empty tensors among them
        layer = [((H * F // 7 + 1,), dt), ((1,), torch.float32), ((r, 3), dt), ((0,), dt), ((F + 1,), torch.float32)]
    return layer * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "experts":
        T, E, R, K = case["T"], case["E"], case["R"], case["K"]
        n, m = PATTERNS[case["pattern"]]
        values, idx = _pack(_normal(gen, (E * R, K), 0.02, dt), n, m)
        s.update(values=values.view(E, R, -1), idx=idx.view(E, R, -1), lengths=_lengths(gen, T, E, case["used"]),
                 act=_normal(gen, (T, K), 1.0, dt))
        s["offsets"] = _offsets(s["lengths"])
        if case["train"]:
            s["G"] = _normal(gen, (T, R), 0.05, dt)
        return s
    if case["op"] == "clip":
        # gradients of different layers differ in size; a few entries stand out
        s["grads"] = []
        for shape, t in _shapes(case):
            g = torch.randn(shape, generator=gen, device="cuda") * torch.rand((), generator=gen, device="cuda")
            s["grads"].append((g * (1 + 9 * (g.abs() > 3))).mul_(1e-2).to(t))
        # the clipped gradients go into one buffer a type, tensor after tensor
        s["flat"] = {t: torch.empty(sum(g.numel() for g in s["grads"] if g.dtype == t), dtype=t, device="cuda")
                     for t in dict.fromkeys(g.dtype for g in s["grads"])}
        at = dict.fromkeys(s["flat"], 0)
        s["out"] = []
        for g in s["grads"]:
            s["out"].append(s["flat"][g.dtype][at[g.dtype]: at[g.dtype] + g.numel()].view(g.shape))
            at[g.dtype] += g.numel()
        if own:     # a training loop's gradients keep their tensors, and it keeps their list
            import structured_sparse_gemm_nm_amd as nm
            s["list"] = nm.nm_grad_list(s["grads"], s["out"])
        return s
    T, K = case["T"], case["K"]
    # activations or weights of differing rows, with a few outlying columns
    x = torch.randn((T, K), generator=gen, device="cuda") * (0.1 + torch.rand((T, 1), generator=gen, device="cuda"))
    x[:, :: 97] *= 8
    s["x"] = x.to(dt)
    if case["op"] == "mx":
        E, R = case["E"], case["R"]
        packed = [_mx_pack(torch.randn((R, K), generator=gen, device="cuda") * 0.02) for _ in range(max(E, 1))]
        s["wq"], s["ws"] = (torch.stack([p[i] for p in packed]) if E else packed[0][i] for i in range(2))
        if E:
            s["lengths"] = _lengths(gen, T, E, case["used"])
            s["offsets"] = _offsets(s["lengths"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _RUN_OWN[state["case"]["op"]](state)
    return _RUN_PLAIN[state["case"]["op"]](state)


def _unpack_plain(values, idx, K, n, m):
    R, S = values.shape
    bits = 3 if m == 8 else 2
    first = torch.arange(S, device=values.device) * bits
    word, off = first >> 5, first & 31
    stream = torch.nn.functional.pad(idx.long() & 0xFFFFFFFF, (0, 1))
    pos = ((stream[:, word] >> off) | (stream[:, word + 1] << (32 - off))) & (m - 1)
    dense = torch.zeros((R, K // m, m), device=values.device)
    dense.scatter_(2, pos.view(R, K // m, n), values.float().view(R, K // m, n))
    return dense.view(R, K), pos


def _experts_plain(s):
    c = s["case"]
    n, m = PATTERNS[c["pattern"]]
    K, R, out = c["K"], c["R"], DTYPES[c["out"]]
    act = s["act"].float()
    y = torch.empty((c["T"], R), device="cuda", dtype=out)
    if c["train"]:
        g = s["G"].float()
        dx = torch.empty((c["T"], K), device="cuda", dtype=out)
        dw = torch.zeros(s["values"].shape, device="cuda", dtype=out)
    at = 0
    for e, length in enumerate(s["lengths"]):
        if length == 0:
            continue
        rows = slice(at, at + length)
        at += length
        W, pos = _unpack_plain(s["values"][e], s["idx"][e], K, n, m)
        y[rows] = (act[rows] @ W.t()).to(out)
        if c["train"]:
            dx[rows] = (g[rows] @ W).to(out)
            full = (g[rows].t() @ act[rows]).view(R, K // m, m)
            dw[e] = full.gather(2, pos.view(R, K // m, n)).view(R, -1).to(out)
    return (y, dx, dw) if c["train"] else y


def _pow2(e, dtype=torch.float32):
    """2^e for whole e in [-150, 150], from a table of exact powers."""
    table = torch.tensor([2.0 ** i for i in range(-150, 151)], dtype=torch.float64, device=e.device)
    return table.to(dtype)[(e + 150).long()]


def _mx_split(x):
    """x [T, K] in blocks of 32: each value's four bits (sign, 2 exponent, 1
    mantissa bits) and each block's exponent byte, 2^(byte - 127): the exponent
    of the block's largest magnitude less 2, so that it lies in [4, 8)."""
    b = x.float().view(x.shape[0], -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    byte = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)
    # 2^(127 - byte), and the value in two exact factors (2^127 is the largest power fp32 holds)
    half = (127 - byte) // 2
    v = b * _pow2(half) * _pow2(127 - byte - half)
    a = v.abs()
    # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (8 and above saturate), ties to the even mantissa
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = code + 8 * torch.signbit(v).int()
    return code, byte.squeeze(2)


def _mx_pack(x):
    """The codes two a byte, and the exponent bytes in panels of eight: block i of
    row r at [i // 8, r, i % 8], zeros behind the last."""
    code, byte = _mx_split(x)
    code = code.view(x.shape[0], -1, 2)
    byte = torch.nn.functional.pad(byte, (0, -byte.shape[1] % 8)).view(x.shape[0], -1, 8).transpose(0, 1)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).to(torch.uint8), byte.to(torch.uint8).contiguous()


def _mx_values(code, byte):
    """The values that codes [T, blocks, 32] and exponent bytes [T, blocks] stand for."""
    mag = torch.tensor(E2M1, device=code.device)[(code & 7).long()]
    mag = torch.where(code >= 8, -mag, mag)
    e = (byte.int() - 127).unsqueeze(2)
    half = e // 2
    return (mag * _pow2(half) * _pow2(e - half)).view(code.shape[0], -1)


def _mx_unpack(q, panels):
    code = torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1, BLOCK).int()
    byte = panels.transpose(0, 1).reshape(q.shape[0], -1)[:, : code.shape[1]]
    return _mx_values(code, byte)


def _mx_round_plain(s):
    x = s["x"]
    code, byte = _mx_split(x)
    return _mx_values(code, byte).to(x.dtype)


def _mx_plain(s):
    c = s["case"]
    out = DTYPES[c["out"]]
    x = _mx_values(*_mx_split(s["x"]))
    if not c["E"]:
        return (x @ _mx_unpack(s["wq"], s["ws"]).t()).to(out)
    y = torch.empty((c["T"], c["R"]), device="cuda", dtype=out)
    at = 0
    for e, length in enumerate(s["lengths"]):
        if length:
            y[at: at + length] = (x[at: at + length] @ _mx_unpack(s["wq"][e], s["ws"][e]).t()).to(out)
            at += length
    return y


def _clip_plain(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        f = g.float()
        total = total + (f * f).sum(dtype=torch.float64)
    norm = total.sqrt()
    coef = (s["case"]["max_norm"] / (norm + EPS)).clamp(max=1.0).float()
    for o, g in zip(s["out"], s["grads"]):
        o.copy_(g.float() * coef)
    return [norm.float(), *s["flat"].values()]


def _experts_own(s):
    import structured_sparse_gemm_nm_amd as nm
    c = s["case"]
    n, m = PATTERNS[c["pattern"]]
    out = DTYPES[c["out"]]
    y = nm.nm_group_spmm(s["values"], s["idx"], s["act"], s["offsets"], c["K"], n, m, out_dtype=out)
    if not c["train"]:
        return y
    dx = nm.nm_group_spmm_dx(s["values"], s["idx"], s["G"], s["offsets"], c["K"], n, m, out_dtype=out)
    dw = nm.nm_group_spmm_dw(s["idx"], s["G"], s["act"], s["offsets"], c["K"], n, m, out_dtype=out)
    return y, dx, dw


def _mx_round_own(s):
    import structured_sparse_gemm_nm_amd as nm
    q, scale = nm.nm_mx_quantize(s["x"])
    return nm.nm_mx_dequantize(q, scale, s["x"].dtype)


def _mx_own(s):
    import structured_sparse_gemm_nm_amd as nm
    xq, xs = nm.nm_mx_quantize(s["x"])
    return nm.nm_mx_gemm(s["wq"], s["ws"], xq, xs, s.get("offsets"), out_dtype=DTYPES[s["case"]["out"]])


def _clip_own(s):
    import structured_sparse_gemm_nm_amd as nm
    norm, _ = nm.nm_grad_clip(s["list"], s["case"]["max_norm"], eps=EPS)
    return [norm, *s["flat"].values()]


_RUN_PLAIN = {"experts": _experts_plain, "mx_round": _mx_round_plain, "mx": _mx_plain, "clip": _clip_plain}
_RUN_OWN = {"experts": _experts_own, "mx_round": _mx_round_own, "mx": _mx_own, "clip": _clip_own}


# ---------------------------------------------------------------------------
# what one pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "experts":
        T, R, K, E = case["T"], case["R"], case["K"], case["E"]
        n, m = PATTERNS[case["pattern"]]
        S = K // m * n
        idx = R * ((S * (3 if m == 8 else 2) + 31) // 32) * 4
        o = 4 if case["out"] == "f32" else 2
        b = case["used"] * (R * S * 2 + idx) + T * K * 2 + T * R * o + 4 * (E + 1)
        f = 2 * T * R * S
        if case["train"]:
            # G read, dX and the packed dW of every expert written
            b += T * R * 2 + T * K * o + E * R * S * o
            f += 2 * T * R * S + 2 * T * R * K
        return dict(bytes=b, flops=f)
    if case["op"] == "clip":
        b = f = 0
        for shape, t in _shapes(case):
            n = math.prod(shape)
            b += 2 * n * (4 if t == torch.float32 else 2)
            f += 3 * n
        return dict(bytes=b + 4, flops=f)
    T, K = case["T"], case["K"]
    e = 4 if case["dtype"] == "f32" else 2
    four = K // 2 + K // BLOCK
    if case["op"] == "mx_round":
        # x read, the four bits and scales written, the values they stand for written
        return dict(bytes=T * (2 * K * e + four), flops=4 * T * K)
    R, o = case["R"], 4 if case["out"] == "f32" else 2
    weights = max(case["used"], 1)
    return dict(bytes=T * K * e + T * four + weights * R * four + T * R * o, flops=2 * T * R * K)


# ---------------------------------------------------------------------------
# the same outputs in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"experts": _experts_exact, "mx_round": _mx_round_exact, "mx": _mx_exact, "clip": _clip_exact}[case["op"]](s)


def _experts_exact(s):
    c = s["case"]
    n, m = PATTERNS[c["pattern"]]
    R, K, T, E = c["R"], c["K"], c["T"], c["E"]
    S = K // m * n
    bits = 3 if m == 8 else 2
    ends = s["offsets"].cpu().tolist()
    x = s["act"].double()
    y = torch.zeros((T, R), dtype=torch.float64, device="cuda")
    dx = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    dw = torch.zeros((E, R, S), dtype=torch.float64, device="cuda")
    j = torch.arange(S, device="cuda")
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        # the stream bit by bit: survivor j's position is bits [j*bits, j*bits + bits)
        words = s["idx"][e].long() & 0xFFFFFFFF
        col = torch.zeros((R, S), dtype=torch.int64, device="cuda")
        for i in range(bits):
            at = j * bits + i
            col |= ((words[:, at // 32] >> (at % 32)) & 1) << i
        col += j // n * m
        W = torch.zeros((R, K), dtype=torch.float64, device="cuda").scatter_(1, col, s["values"][e].double())
        y[lo:hi] = x[lo:hi] @ W.t()
        if c["train"]:
            g = s["G"][lo:hi].double()
            dx[lo:hi] = g @ W
            dw[e] = torch.gather(g.t() @ x[lo:hi], 1, col)
    return (y, dx, dw) if c["train"] else y


def _mx_round_exact(s):
    """Each value's nearest of the sixteen in its block's scale, found by distance."""
    x = s["x"].double()
    out = torch.empty_like(x)
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for lo in range(0, x.shape[0], 1024):
        b = x[lo: lo + 1024].view(-1, BLOCK)
        mant, e = torch.frexp(b.abs().amax(1, keepdim=True))       # amax = mant 2^e, mant in [.5, 1)
        e = torch.where(mant > 0, e - 3, torch.full_like(e, -127)).clamp(min=-127)
        scale = _pow2(e, torch.float64)
        a = b.abs() / scale
        best = torch.zeros_like(a, dtype=torch.int64)
        for k in range(1, 8):
            near, far = (a - grid[k]).abs(), (a - grid[best]).abs()
            best = torch.where((near < far) | ((near == far) & (k % 2 == 0)), torch.full_like(best, k), best)
        out[lo: lo + 1024] = (grid[best] * scale * torch.sign(b)).view(-1, x.shape[1])
    return out


def _mx_exact(s):
    c = s["case"]
    x = _mx_round_exact(s)
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")

    def weight(q, panels):
        block = torch.arange(q.shape[1] * 2 // BLOCK, device="cuda")
        byte = panels[block // 8, :, block % 8].t()
        w = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = grid[(q % 16).long()], grid[(q // 16).long()]
        return w * _pow2(byte.int() - 127, torch.float64).repeat_interleave(BLOCK, 1)

    if not c["E"]:
        return x @ weight(s["wq"], s["ws"]).t()
    ends = s["offsets"].cpu().tolist()
    return torch.cat([x[ends[e]: ends[e + 1]] @ weight(s["wq"][e], s["ws"][e]).t() for e in range(c["E"])])


def _clip_exact(s):
    flat = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in s["grads"]:
        d = g.double().reshape(-1)
        flat = flat + torch.dot(d, d)
    norm = flat.sqrt()
    scale = min(1.0, s["case"]["max_norm"] / (float(norm) + EPS))
    return [norm, *(torch.cat([g.double().reshape(-1) for g in s["grads"] if g.dtype == t]) * scale for t in s["flat"])]
