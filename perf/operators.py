"""Workloads of the experts' MLP operators: the grouped products (one weight
matrix per expert, ragged groups of rows) and the SwiGLU activation that keeps
its input in 8 bits for the backward pass.

Operators (``op`` of a case):

  ckpt8_fwd   y = w[r] silu(g) u and the 8-bit checkpoint (codes, scales) of x = [g | u]
  ckpt8_bwd   from the checkpoint alone: dx = [dg | du], dw[r], and y once more
  fc1         per expert: y = probs[t] silu(x Wg^T) (x Wu^T), with what the
              backward keeps (nothing, fc1 in bf16, or fc1 in 8 bits)
  mm          per expert: y = x W^T
  mm_bwd      per expert: dx = dy W and dW = dy^T x

Rows are sorted by expert; ``ends[e]`` is the end of expert e's rows, and rows
past the last end belong to nobody (their outputs are zero).  The checkpoint
holds each half of a row in blocks of 32 columns: one power of two per block
(8 bits of exponent) and one e4m3 code per element.  ``own`` picks the
implementation: the package's kernels, or the formulas in 32 bits.
"""
import math

import torch

own = False

BLOCK = 32
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # training, the Llama-like MLP of 8192 tokens: the activation between two dense products
        dict(name="ckpt8_fwd_llama", op="ckpt8_fwd", rows=8192, n=14336, dtype="bf16", weighted=False, pad=0),
        # the odd-width fp32 stress shape, every row with its routing weight, rows in a wider buffer
        dict(name="ckpt8_fwd_odd_f32", op="ckpt8_fwd", rows=3000, n=5503, dtype="f32", weighted=True, pad=3),
        # training, the Megatron ffn-4096 shape as routed experts: weights' gradient, y made again
        dict(name="ckpt8_bwd_megatron", op="ckpt8_bwd", rows=8192, n=4096, dtype="bf16", weighted=True, again=True, pad=0),
        # the smallest configuration (16 x 2 rows, n = 256): launch latency
        dict(name="ckpt8_bwd_tiny", op="ckpt8_bwd", rows=32, n=256, dtype="f32", weighted=False, again=False, pad=0),
        # serving: one token of a sequence sent to two of eight small experts
        dict(name="fc1_one_token", op="fc1", rows=2, E=8, active=2, K=1024, n=1792, tail=0, probs=True, save="none"),
        # serving: sixteen sequences decode together, two experts each, Llama-like experts: weights stream
        dict(name="fc1_decode", op="fc1", rows=32, E=8, active=8, K=4096, n=14336, tail=0, probs=True, save="none"),
        # training: 8192 tokens, two of eight Llama-like experts each, 8-bit checkpoint
        dict(name="fc1_train", op="fc1", rows=16384, E=8, active=8, K=4096, n=14336, tail=0, probs=True, save="fp8"),
        # training: many small experts, some without a row, a buffer that is not full
        dict(name="fc1_fine", op="fc1", rows=8250, E=64, active=61, K=2048, n=1288, tail=37, probs=True, save="bf16"),
        # serving: the second product of the same decode step
        dict(name="mm_decode", op="mm", rows=32, E=8, active=8, K=14336, N=4096, tail=0),
        # prefill: many small experts
        dict(name="mm_fine", op="mm", rows=16500, E=64, active=64, K=1288, N=2048, tail=100),
        # training: both gradients of the Llama-like experts' second product
        dict(name="mm_bwd_train", op="mm_bwd", rows=16384, E=8, active=8, K=14336, N=4096, tail=0, dw="bf16"),
        # a small, ragged group: few rows per expert, fp32 weight gradients
        dict(name="mm_bwd_ragged", op="mm_bwd", rows=1333, E=12, active=10, K=520, N=1160, tail=5, dw="f32"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _count(rng, lo, hi):
    """A number of rows: any odd one, or a power of two."""
    v = _log(rng, lo, hi)
    return int(v) | 1 if rng.random() < 0.6 else 2 ** round(math.log2(v))


def _width(rng, lo, hi):
    """A width the tensor-core products take: 1, 1.25 or 1.75 times a power of
    two, or an odd multiple of 8."""
    v = _log(rng, lo, hi)
    if rng.random() < 0.5:
        p = 2 ** int(math.log2(v))
        w = max(f * p for f in (1, 1.25, 1.75) if f * p <= v)
        return max(8, int(w) // 8 * 8)
    return 8 * (int(v / 8) | 1)


def draw(rng):
    op = rng.choice(["ckpt8_fwd", "ckpt8_bwd", "fc1", "mm", "mm_bwd"])
    if op in ("ckpt8_fwd", "ckpt8_bwd"):
        rows, n = _count(rng, 1, 16384), rng.choice([_width(rng, 64, 32768), int(_log(rng, 1, 8000)) | 1])
        while rows * n > 8192 * 14336:
            rows = rows // 2 | 1
        c = dict(op=op, rows=rows, n=n, dtype=rng.choice(["f32", "bf16", "bf16"]), weighted=rng.random() < 0.5,
                 pad=rng.choice([0, 0, 16, 3]))
        if op == "ckpt8_bwd":
            c["again"] = rng.random() < 0.5
        return c
    E = rng.choice([1, 2, 8, 8, 16, 64])
    rows = _count(rng, 1, 32768)
    K, N = _width(rng, 64, 14336), _width(rng, 64, 7168 if op == "fc1" else 14336)
    while rows * K * N > 2 ** 39 or E * K * N > 2 ** 28:
        if rows > 4 * E:
            rows = rows // 2 | 1
        elif K > N:
            K = 8 * (K // 16 | 1)
        else:
            N = 8 * (N // 16 | 1)
    tail = rng.choice([0, 0, 1, min(rows - 1, 37)]) if rows > 1 else 0
    c = dict(op=op, rows=rows, E=E, active=min(rows - tail, rng.randint(max(1, E // 2), E)), K=K, tail=tail)
    if op == "fc1":
        return dict(c, n=N, probs=rng.random() < 0.7, save=rng.choice(["none", "bf16", "fp8"]))
    if op == "mm":
        return dict(c, N=N)
    return dict(c, N=N, dw=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------ inputs ---

def _groups(case, seed):
    """Rows per expert: `active` experts share the assigned rows unevenly (none of
    them without a row), the others have none."""
    g = torch.Generator().manual_seed(seed)
    E, active, rows = case["E"], case["active"], case["rows"] - case["tail"]
    who = torch.randperm(E, generator=g)[:active]
    share = torch.rand(active, generator=g) + 0.5
    counts = torch.ones(active, dtype=torch.int64)
    if rows > active:
        extra = torch.multinomial(share, rows - active, replacement=True, generator=g)
        counts += torch.bincount(extra, minlength=active)
    out = torch.zeros(E, dtype=torch.int64)
    out[who] = counts
    return out


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    """N(0, std^2), made in slices (no fp32 copy of a whole weight tensor)."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    flat = t.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(std))
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("ckpt8_fwd", "ckpt8_bwd"):
        rows, n, dt = case["rows"], case["n"], _DT[case["dtype"]]
        x = _randn(g, rows, 2 * n + case["pad"], dtype=dt)[:, :2 * n]
        # a few columns are far larger than the rest, as in trained models
        loud = torch.randperm(2 * n, generator=g, device="cuda")[:max(1, n // 128)]
        x[:, loud] *= 16
        s = {"x": x, "w": torch.rand(rows, generator=g, device="cuda") if case["weighted"] else None}
        if op == "ckpt8_bwd":
            s["q"], s["scales"] = _encode(x)
            s["dy"] = _randn(g, rows, n, dtype=dt)
            del s["x"]
        return dict(s, case=case)
    counts = _groups(case, seed)
    rows, E, K = case["rows"], case["E"], case["K"]
    s = {"case": case, "counts": counts.tolist() + [case["tail"]],
         "ends": counts.cumsum(0).to(torch.int32).cuda(), "x": _randn(g, rows, K)}
    N = 2 * case["n"] if op == "fc1" else case["N"]
    s["w"] = _randn(g, E, N, K, std=K ** -0.5)
    if op == "fc1":
        s["probs"] = torch.rand(rows, generator=g, device="cuda") if case["probs"] else None
    if op == "mm_bwd":
        s["dy"] = _randn(g, rows, N)
    return s


# ---------------------------------------------------------------- one pass ---

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gate_up_swiglu_gb300 as sw

    c = s["case"]
    op = c["op"]
    if op == "ckpt8_fwd":
        return sw.swiglu_ckpt8_fwd(s["x"], s["w"])
    if op == "ckpt8_bwd":
        dx, dw, y = sw.swiglu_ckpt8_bwd(s["dy"], s["q"], s["scales"], s["w"], return_y=c["again"])
        return {"dx": dx, "dw": dw, "y": y}
    if op == "fc1":
        save = None if c["save"] == "none" else c["save"]
        return sw.swiglu_grouped_fc1_fwd(s["x"], s["w"], s["ends"], s["probs"], save=save)
    if op == "mm":
        return sw.swiglu_grouped_mm_fwd(s["x"], s["w"], s["ends"])
    return {"dx": sw.swiglu_grouped_mm_dgrad(s["dy"], s["w"], s["ends"]),
            "dw": sw.swiglu_grouped_mm_wgrad(s["dy"], s["x"], s["ends"], dtype=_DT[c["dw"]])}


def _blocks(t):
    """[rows, n] -> [rows, blocks, 32], the last block filled up with zeros."""
    return torch.nn.functional.pad(t, (0, -t.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))


def _encode_half(x):
    b = _blocks(x.float())
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    # the smallest 2^e with amax <= 448 * 2^e, 448 = 1.75 * 2^8 the largest e4m3 value
    m, e = torch.frexp(amax)
    code = torch.where(amax > 0, e + (m > 0.875) + (127 - 9), 0).clamp(min=0)
    up = ((254 - code) << 23).view(torch.float32)  # 2^(127 - code)
    q = (b * up.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.flatten(1)[:, :x.shape[1]], code.to(torch.uint8)


def _encode(x):
    n = x.shape[1] // 2
    (qg, sg), (qu, su) = _encode_half(x[:, :n]), _encode_half(x[:, n:])
    q = torch.cat([qg.view(torch.uint8), qu.view(torch.uint8)], 1).view(torch.float8_e4m3fn)
    return q, torch.cat([sg, su], 1).view(torch.float8_e8m0fnu)


def _decode_half(q, scales):
    code = scales.view(torch.uint8).int()
    scale = torch.where(code > 0, code << 23, 1 << 22).view(torch.float32)
    return (_blocks(q.float()) * scale.unsqueeze(-1)).flatten(1)[:, :q.shape[1]]


def _swiglu(g, u, w):
    y = g / (1 + torch.exp(-g)) * u
    return y if w is None else y * w[:, None]


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "ckpt8_fwd":
        x, n = s["x"], c["n"]
        y = _swiglu(x[:, :n].float(), x[:, n:].float(), s["w"]).to(x.dtype)
        return (y, *_encode(x))
    if op == "ckpt8_bwd":
        n, dt = c["n"], s["dy"].dtype
        nb = s["scales"].shape[1] // 2
        g = _decode_half(s["q"][:, :n], s["scales"][:, :nb])
        u = _decode_half(s["q"][:, n:], s["scales"][:, nb:])
        dy, w = s["dy"].float(), s["w"]
        sig = 1 / (1 + torch.exp(-g))
        silu = g * sig
        dw = (dy * silu * u).sum(1) if w is not None else None
        d = dy if w is None else dy * w[:, None]
        dx = torch.cat([d * u * sig * (1 + g * (1 - sig)), d * silu], 1).to(dt)
        return {"dx": dx, "dw": dw, "y": _swiglu(g, u, w).to(dt) if c["again"] else None}
    x, w, counts = s["x"].float().split(s["counts"]), s["w"].float(), s["counts"]
    none = x[-1].new_zeros(counts[-1], w.shape[1])  # the rows that belong to nobody
    if op == "mm_bwd":
        dy = s["dy"].float().split(counts)
        dx = torch.cat([d @ m for d, m in zip(dy, w)] + [torch.zeros_like(x[-1])])
        dw = torch.stack([d.T @ r for d, r in zip(dy, x[:-1])])
        return {"dx": dx.to(torch.bfloat16), "dw": dw.to(_DT[c["dw"]])}
    out = torch.cat([r @ m.T for r, m in zip(x, w)] + [none])
    if op == "mm":
        return out.to(torch.bfloat16)
    n = c["n"]
    y = _swiglu(out[:, :n], out[:, n:], s["probs"]).to(torch.bfloat16)
    if c["save"] == "bf16":
        return y, out.to(torch.bfloat16)
    return (y, *_encode(out)) if c["save"] == "fp8" else y


# -------------------------------------------------------------------- cost ---

def work(case):
    op = case["op"]
    if op in ("ckpt8_fwd", "ckpt8_bwd"):
        rows, n, e = case["rows"], case["n"], 4 if case["dtype"] == "f32" else 2
        ckpt = 2 * n + 2 * -(-n // BLOCK)
        per_row = ckpt + (3 * n * e if op == "ckpt8_fwd" else 3 * n * e)
        if op == "ckpt8_bwd" and case["again"]:
            per_row += n * e
        if case["weighted"]:
            per_row += 4 if op == "ckpt8_fwd" else 8
        return {"bytes": rows * per_row, "flops": (30 if op == "ckpt8_fwd" else 25) * rows * n}
    rows, E, K = case["rows"], case["E"], case["K"]
    live = rows - case["tail"]
    if op == "fc1":
        n = case["n"]
        saved = {"none": 0, "bf16": 4 * n, "fp8": 2 * n + 2 * -(-n // BLOCK)}[case["save"]]
        out = rows * (2 * n + saved) + (4 * live if case["probs"] else 0)
        return {"bytes": live * K * 2 + case["active"] * 2 * n * K * 2 + 4 * E + out, "flops": 4 * live * n * K}
    N = case["N"]
    if op == "mm":
        return {"bytes": live * K * 2 + case["active"] * N * K * 2 + 4 * E + rows * N * 2, "flops": 2 * live * N * K}
    dw = E * N * K * (4 if case["dw"] == "f32" else 2)
    return {"bytes": live * (N + K) * 2 + case["active"] * N * K * 2 + 4 * E + rows * K * 2 + dw,
            "flops": 4 * live * N * K}


# ----------------------------------------------------------- in 64 bits -------

def _e4m3(v):
    """v rounded to e4m3 (4 significant bits down to 2^-6, steps of 2^-9 below), nearest even."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(v / step) * step


def _codes64(x):
    """The checkpoint's codes and scales for x, as the numbers they stand for."""
    qs, ss = [], []
    for half in x.double().chunk(2, 1):
        n = half.shape[1]
        nb = -(-n // BLOCK)
        b = torch.zeros(half.shape[0], nb * BLOCK, dtype=torch.float64, device=x.device)
        b[:, :n] = half
        b = b.view(-1, nb, BLOCK)
        amax = b.abs().max(-1).values
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        scale = torch.where(amax > 448.0 * scale, 2 * scale, scale)
        scale = torch.where(amax <= 224.0 * scale, scale / 2, scale).clamp(min=2.0 ** -127)
        qs.append(_e4m3(b / scale[..., None]).flatten(1)[:, :n])
        ss.append(scale)
    return torch.cat(qs, 1), torch.cat(ss, 1)


def _silu64(g):
    return torch.where(g >= 0, g / (1 + torch.exp(-g.abs())), g * torch.exp(-g.abs()) / (1 + torch.exp(-g.abs())))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ckpt8_fwd":
        n = case["n"]
        x = s["x"].double()
        y = _silu64(x[:, :n]) * x[:, n:]
        if s["w"] is not None:
            y *= s["w"].double()[:, None]
        return (y, *_codes64(s["x"]))
    if op == "ckpt8_bwd":
        n = case["n"]
        nb = -(-n // BLOCK)
        scale = torch.exp2(s["scales"].view(torch.uint8).double() - 127).view(-1, 2, nb)
        col = torch.arange(n, device="cuda") // BLOCK
        q = s["q"].double()
        g, u = q[:, :n] * scale[:, 0][:, col], q[:, n:] * scale[:, 1][:, col]
        dy = s["dy"].double()
        silu, sig = _silu64(g), torch.sigmoid(g)
        y, dw, d = silu * u, None, dy
        if s["w"] is not None:
            w = s["w"].double()[:, None]
            dw, d, y = (dy * y).sum(1), dy * w, y * w
        dx = torch.cat([d * u * sig * (1 + g * torch.sigmoid(-g)), d * silu], 1)
        return {"dx": dx, "dw": dw, "y": y if case["again"] else None}
    # rows and weights expert by expert, in place of one 64-bit copy of all of them
    rows, N = case["rows"], s["w"].shape[1]
    at = 0
    if op == "mm_bwd":
        dx = torch.zeros(rows, case["K"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["E"], N, case["K"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            k = s["counts"][e]
            if k:
                d = s["dy"][at:at + k].double()
                dx[at:at + k] = torch.matmul(d, s["w"][e].double())
                dw[e] = torch.matmul(d.t(), s["x"][at:at + k].double())
            at += k
        return {"dx": dx, "dw": dw}
    out = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        k = s["counts"][e]
        if k:
            out[at:at + k] = torch.matmul(s["x"][at:at + k].double(), s["w"][e].double().t())
        at += k
    if op == "mm":
        return out
    n = case["n"]
    y = _silu64(out[:, :n]) * out[:, n:]
    if s["probs"] is not None:
        y *= s["probs"].double()[:, None]
    if case["save"] == "bf16":
        return y, out
    # a product on the border between two codes may be rounded either way: no 64-bit value
    return (y, None, None) if case["save"] == "fp8" else y
