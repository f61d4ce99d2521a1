"""Workloads of the MLP sublayer's other operators: the layer norm in front of
linear_fc1, and the MLP with weights and activations in 4 bits.

Operators (``op`` of a case):

  norm_fwd   y = (x - mean) rstd w + b, and mean and rstd of each row
  norm_bwd   dx, dw and db from dy, x, mean and rstd
  quantize   x in microscaled 4-bit floating point and back: the values its codes stand for
  mm         y = x W^T, both in microscaled 4-bit floating point
  mlp        out = (silu(x W1g^T) (x W1u^T)) W2^T: x [rows, hidden] in bf16 is rounded to
             4 bits, and so is the activation in front of the second product

The 4-bit format: blocks of 32 consecutive values of a row, one power of two per
block (8 bits of exponent, 255 for NaN), one e2m1 code per value (0, 0.5, 1, 1.5,
2, 3, 4, 6 and a sign).  Codes lie two to a byte, the even column in the low half,
rows filled up with zeros to whole blocks.  Scales lie in tiles of 128 rows by 4
blocks, 512 bytes each: row i of the tile has its four bytes at 16 (i % 32) +
4 (i // 32).  ``own`` picks the implementation: the package's kernels, or the
formulas in 32 bits.
"""
import math

import torch

own = False

BLOCK, TILE, CHUNK = 32, 128, 4
EPS = 1e-5
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # training, 2048 x 4 tokens of the Megatron-like layer: the norm in front of linear_fc1
        dict(name="norm_fwd_megatron", op="norm_fwd", rows=8192, n=4096, dtype="bf16", w=True, b=True, pad=0),
        # the odd-width fp32 stress shape, rows in a wider buffer, no bias
        dict(name="norm_fwd_odd_f32", op="norm_fwd", rows=3000, n=5503, dtype="f32", w=True, b=False, pad=3),
        # the same layer's backward, with the gradients of weight and bias
        dict(name="norm_bwd_megatron", op="norm_bwd", rows=8192, n=4096, dtype="bf16", w=True, b=True, pad=0),
        # the smallest configuration (16 x 2 rows, n = 256): launch latency
        dict(name="norm_bwd_tiny", op="norm_bwd", rows=32, n=256, dtype="f32", w=True, b=True, pad=0),
        # loading a model: the first projection of a Llama-like MLP to 4 bits and back
        dict(name="quantize_weight", op="quantize", rows=28672, n=4096, dtype="bf16", pad=0),
        # activations of an odd width in fp32, rows in a wider buffer
        dict(name="quantize_odd_f32", op="quantize", rows=1000, n=5503, dtype="f32", pad=1),
        # serving: the second projection for sixteen sequences that decode together
        dict(name="mm_decode", op="mm", rows=16, N=4096, K=14336),
        # prompts: the second projection of 8192 tokens
        dict(name="mm_prompt", op="mm", rows=8192, N=4096, K=14336),
        # ragged sizes: a few hundred tokens, odd outputs, a contraction that ends inside a block
        dict(name="mm_ragged", op="mm", rows=333, N=5503, K=2000),
        # serving: one token through a small MLP
        dict(name="mlp_one_token", op="mlp", rows=1, H=1024, n=1792),
        # serving: sixteen sequences decode together, Llama-like MLP: weights stream
        dict(name="mlp_decode", op="mlp", rows=16, H=4096, n=14336),
        # prompts: 8192 tokens through the Llama-like MLP
        dict(name="mlp_prompt", op="mlp", rows=8192, H=4096, n=14336),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _size(rng, lo, hi):
    """An odd number, a multiple of 8, or 1, 1.25 or 1.75 times a power of two."""
    v = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.35:
        return max(lo, min(hi, int(v) | 1))
    if kind < 0.65:
        return max(lo, int(v) // 8 * 8)
    p = 2 ** int(math.log2(v))
    return max(lo, int(max(f * p for f in (1, 1.25, 1.75) if f * p <= v)))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "quantize", "mm", "mm", "mlp", "mlp"])
    rows = _size(rng, 1, 8192 if op in ("mm", "mlp") else 16384)
    if op in ("norm_fwd", "norm_bwd", "quantize"):
        n = _size(rng, 16, 32768)
        while rows * n > 2 ** 26:
            rows = rows // 2 | 1
        c = dict(op=op, rows=rows, n=n, dtype=rng.choice(["f32", "bf16", "bf16"]), pad=rng.choice([0, 0, 16, 3]))
        if op != "quantize":
            c["w"] = rng.random() < 0.8
            c["b"] = c["w"] and rng.random() < 0.7
        return c
    if op == "mm":
        c = dict(op=op, rows=rows, N=_size(rng, 1, 16384), K=_size(rng, 32, 14336))
        most, last = 8192 * 4096 * 14336, "N"
    else:
        c = dict(op=op, rows=rows, H=_size(rng, 64, 8192), n=_size(rng, 256, 14336))
        most, last = 8192 * 4096 * 14336, "n"
    while c["rows"] * c.get("K", c.get("H")) * c[last] > most:
        c["rows"] = c["rows"] // 2 | 1
    return c


# ------------------------------------------------------------------ inputs ---

def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def _loud(g, x):
    """A few columns far larger than the rest, as in trained models."""
    n = x.shape[1]
    x[:, torch.randperm(n, generator=g, device="cuda")[:max(1, n // 128)]] *= 16
    return x


def _weight(g, N, K, parts=1):
    return _quantize(_randn(g, N, K, std=K ** -0.5), parts)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, rows = case["op"], case["rows"]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd", "quantize"):
        n, dt = case["n"], _DT[case["dtype"]]
        s["x"] = _loud(g, _randn(g, rows, n + case["pad"], dtype=dt)[:, :n])
        if op == "quantize":
            return s
        s["x"].add_(0.5)  # a mean that is not zero
        s["w"] = (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dt) if case["w"] else None
        s["b"] = (0.2 * torch.randn(n, generator=g, device="cuda")).to(dt) if case["b"] else None
        if op == "norm_bwd":
            s["dy"] = _randn(g, rows, n, dtype=dt)
            _, s["mean"], s["rstd"] = _norm(s["x"].double(), None, None)
            s["mean"], s["rstd"] = s["mean"].float(), s["rstd"].float()
        return s
    if op == "mm":
        s["x"] = _quantize(_loud(g, _randn(g, rows, case["K"])))
        s["w"] = _weight(g, case["N"], case["K"])
        return s
    s["x"] = _loud(g, _randn(g, rows, case["H"]))
    s["w1"] = _weight(g, 2 * case["n"], case["H"], parts=2)
    s["w2"] = _weight(g, case["H"], case["n"])
    return s


# ---------------------------------------------------------------- one pass ---

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gate_up_swiglu_gb300 as sw

    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        return sw.swiglu_layer_norm_fwd(s["x"], s["w"], s["b"], EPS, return_stats=True)
    if op == "norm_bwd":
        dx, dw, db = sw.swiglu_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], bias_grad=c["b"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "quantize":
        q, scales = sw.swiglu_mx4_quantize(s["x"])
        return sw.swiglu_mx4_dequantize(q, scales, c["n"], dtype=s["x"].dtype)
    if op == "mm":
        return sw.swiglu_mx4_mm_fwd(*_as_bytes(*s["x"]), *_as_bytes(*s["w"]))
    return sw.swiglu_mx4_mlp_fwd(s["x"], *_as_bytes(*s["w1"]), *_as_bytes(*s["w2"]))


def _as_bytes(q, scales):
    """The package's operators take codes as bytes: prepare() keeps them in 64 bits, so
    this conversion is a part of the pass."""
    return q.to(torch.uint8), scales


def _norm(x, w, b):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w.to(y.dtype)
    return y if b is None else y + b.to(y.dtype), mean, rstd


def _codes(x):
    """(codes 0 .. 15, scale bytes) of x [rows, n]: [rows, blocks, 32] and [rows, blocks]."""
    v = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))
    amax = v.abs().amax(-1)
    # the smallest 2^e with amax <= 6 * 2^e, 6 = 0.75 * 2^3
    m, e = torch.frexp(amax)
    scale = torch.where(amax > 0, e + (m > 0.75) + (127 - 3), 0).clamp(min=0)
    bad = ~torch.isfinite(v).all(-1)
    scale = torch.where(bad, 255, scale)
    up = ((254 - scale).clamp(min=0) << 23).view(torch.float32)  # 2^(127 - scale)
    v = torch.where(bad[..., None], 0.0, v * up[..., None])
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
    return code + 8 * torch.signbit(v), scale.to(torch.uint8)


def _quantize(x, parts=1):
    """x [rows, n] as (q, scales) in the layout of the package's operators."""
    code, scale = _codes(x)
    code = code.flatten(1)
    q = code[:, ::2] | (code[:, 1::2] << 4)
    s = scale.unflatten(0, (parts, -1))
    s = torch.nn.functional.pad(s, (0, -s.shape[2] % CHUNK, 0, -s.shape[1] % TILE))
    p, r, b = s.shape
    s = s.view(p, r // TILE, 4, 32, b // CHUNK, CHUNK).permute(0, 1, 4, 3, 2, 5)
    s = s.reshape(p * r // TILE, b // CHUNK, TILE * CHUNK)
    return q.contiguous(), s.view(torch.float8_e8m0fnu)


def _values(code, scale):
    """The 32-bit values of codes [..., 32] and scale bytes [...]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=code.device)
    table = torch.cat([table, -table])
    s = scale.int()
    s = torch.where(s > 0, s << 23, 1 << 22).view(torch.float32)  # 2^(byte - 127); 255 is NaN
    s = torch.where(scale == 255, torch.nan, s)
    return table[code.int()] * s[..., None]


def _restore(q, scales, parts=1):
    """The values that (q, scales) stand for: [rows, 32 blocks]."""
    rows, nb = q.shape[0], q.shape[1] // 16
    code = torch.stack([q & 15, q >> 4], -1).view(rows, nb, BLOCK)
    t, ch, _ = scales.shape
    s = scales.view(torch.uint8).view(parts, t // parts, ch, 32, 4, CHUNK).permute(0, 1, 4, 3, 2, 5)
    s = s.reshape(parts, t // parts * TILE, ch * CHUNK)[:, :rows // parts, :nb].reshape(rows, nb)
    return _values(code, s).flatten(1)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_fwd":
        y, mean, rstd = _norm(s["x"].float(), s["w"], s["b"])
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_bwd":
        dt = s["dy"].dtype
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        h = dy if s["w"] is None else dy * s["w"].float()
        dx = rstd * (h - h.mean(1, keepdim=True) - xhat * (h * xhat).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dw": (dy * xhat).sum(0).to(dt) if c["w"] else None,
                "db": dy.sum(0).to(dt) if c["b"] else None}
    if op == "quantize":
        code, scale = _codes(s["x"])
        return _values(code, scale).flatten(1)[:, :c["n"]].to(s["x"].dtype)
    if op == "mm":
        return (_restore(*s["x"]) @ _restore(*s["w"]).T).to(torch.bfloat16)
    x = _values(*_codes(s["x"])).flatten(1)
    g, u = (x @ _restore(*s["w1"], parts=2).T).split(c["n"], 1)
    y = g / (1 + torch.exp(-g)) * u
    return (_values(*_codes(y)).flatten(1) @ _restore(*s["w2"]).T).to(torch.bfloat16)


# -------------------------------------------------------------------- cost ---

def _bytes4(rows, n):
    """Codes and scales of [rows, n] in 4 bits."""
    return rows * -(-n // BLOCK) * 17


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("norm_fwd", "norm_bwd", "quantize"):
        n, e = case["n"], 4 if case["dtype"] == "f32" else 2
        if op == "quantize":
            return {"bytes": 2 * rows * n * e + 2 * _bytes4(rows, n), "flops": 6 * rows * n}
        params = (case["w"] + case["b"]) * n * e
        if op == "norm_fwd":
            return {"bytes": 2 * rows * n * e + 8 * rows + params, "flops": 8 * rows * n}
        return {"bytes": 3 * rows * n * e + 8 * rows + case["w"] * n * e + params, "flops": 16 * rows * n}
    if op == "mm":
        N, K = case["N"], case["K"]
        return {"bytes": _bytes4(rows, K) + _bytes4(N, K) + 2 * rows * N, "flops": 2 * rows * N * K}
    H, n = case["H"], case["n"]
    return {"bytes": 4 * rows * H + _bytes4(2 * n, H) + _bytes4(H, n), "flops": 6 * rows * H * n}


# ----------------------------------------------------------- in 64 bits -------

def _round64(x):
    """x [rows, n] in 64 bits as its 4-bit codes and scales stand for it."""
    rows, n = x.shape
    nb = -(-n // BLOCK)
    v = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :n] = x
    v = v.view(rows, nb, BLOCK)
    top = v.abs().max(-1, keepdim=True).values
    scale = torch.exp2(torch.ceil(torch.log2(top / 6)).clamp(min=-127))
    scale = torch.where(top > 6 * scale, 2 * scale, scale)
    scale = torch.where((top <= 3 * scale) & (scale > 2.0 ** -127), scale / 2, scale)
    r = v / scale
    _, e = torch.frexp(r)
    step = torch.exp2((e - 2).clamp(min=-1).double())  # two significant bits, steps of 0.5 below 1
    out = torch.round(r / step) * step * scale
    return out.flatten(1)[:, :n]


def _decode64(q, scales, parts=1):
    """What (q, scales) stand for, from the definition of each byte's place."""
    rows, nb = q.shape[0], q.shape[1] // 16
    col = torch.arange(nb * BLOCK, device=q.device)
    code = (q[:, col // 2].int() >> (4 * (col % 2)).int()) & 15
    m, e = (code & 1).double(), (code >> 1) & 3
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    v = torch.where(code >= 8, -v, v)
    per = rows // parts
    r = torch.arange(rows, device=q.device)
    part, i = r // per, r % per
    tile, i = part * (-(-per // TILE)) + i // TILE, i % TILE
    b = torch.arange(nb, device=q.device)
    s = scales.view(torch.uint8)[tile[:, None], (b // CHUNK)[None], (16 * (i % 32) + 4 * (i // 32))[:, None] + b % CHUNK]
    return v * torch.exp2(s.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _round64(s["x"].double())
    if op == "norm_fwd":
        x = s["x"].double()
        mean = x.sum(1) / case["n"]
        rstd = (((x - mean[:, None]) ** 2).sum(1) / case["n"] + EPS) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None]
        if s["w"] is not None:
            y *= s["w"].double()
        return (y if s["b"] is None else y + s["b"].double(), mean, rstd)
    if op == "norm_bwd":
        n, dy, rstd = case["n"], s["dy"].double(), s["rstd"].double()[:, None]
        xhat = (s["x"].double() - s["mean"].double()[:, None]) * rstd
        h = dy if s["w"] is None else dy * s["w"].double()
        dx = rstd * (h - h.sum(1, keepdim=True) / n - xhat * (h * xhat).sum(1, keepdim=True) / n)
        return {"dx": dx, "dw": torch.einsum("rc,rc->c", dy, xhat) if case["w"] else None,
                "db": dy.sum(0) if case["b"] else None}
    if op == "mm":
        return torch.matmul(_decode64(*s["x"]), _decode64(*s["w"]).t())
    n = case["n"]
    x, w1 = _round64(s["x"].double()), _decode64(*s["w1"], parts=2)
    f = torch.matmul(x, w1[:, :case["H"]].t())
    y = f[:, :n] * torch.sigmoid(f[:, :n]) * f[:, n:]
    del w1, f
    return torch.matmul(_round64(y), _decode64(*s["w2"])[:, :n].t())
