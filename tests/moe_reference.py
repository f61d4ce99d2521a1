"""Plain 64-bit restatements of the routed experts' operators for the tests
(CPU or CUDA tensors; no kernel of the library is called)."""
import torch

BLOCK = 32


def silu64(g):
    return g * torch.sigmoid(g)


def to_e4m3(v):
    """float64 v (|v| <= 448, or NaN) rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return torch.round(v / step) * step


def checkpoint(x):
    """(code values [rows, 2n], scale codes [rows, 2 nb]) of the 8-bit checkpoint, float64 / int64."""
    qs, ss = [], []
    for half in x.double().chunk(2, -1):
        rows, n = half.shape
        nb = -(-n // BLOCK)
        b = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
        b[:, :n] = half
        b = b.view(rows, nb, BLOCK)
        amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
        code = torch.zeros(rows, nb, dtype=torch.int64, device=x.device)
        # the smallest code that holds the block, found from the definition
        for c in range(0, 255):
            small = amax <= 448.0 * 2.0 ** (c - 127)
            code = torch.where(small, code, c + 1)
            if bool(small.all()):
                break
        v = torch.where(torch.isfinite(b), b, float("nan")) * torch.exp2((127 - code).double())[..., None]
        v = torch.where((code == 247)[..., None], v.clamp(-240.0, 240.0), v)  # 256 * 2^120 is beyond fp32
        qs.append(to_e4m3(v).view(rows, -1)[:, :n])
        ss.append(code)
    return torch.cat(qs, 1), torch.cat(ss, 1)


def restored(q, scales):
    """The float64 values that q (float8_e4m3fn) and scales (float8_e8m0fnu) stand for."""
    rows, two_n = q.shape
    nb = scales.shape[1] // 2
    f = torch.exp2(scales.view(torch.uint8).double() - 127).view(rows, 2, nb)
    col = torch.arange(two_n // 2, device=q.device) // BLOCK
    v = q.float().double().view(rows, 2, two_n // 2)
    return (v * f[:, :, col]).reshape(rows, two_n)


def swiglu_bwd(dy, x, w=None):
    """(dx, dw, y, sum of |dw terms|) in float64."""
    g, u = x.double().chunk(2, -1)
    d = dy.double()
    s = torch.sigmoid(g)
    term = d * silu64(g) * u
    y = silu64(g) * u
    if w is not None:
        d, y = d * w.double()[:, None], y * w.double()[:, None]
    dx = torch.cat([d * u * s * (1 + g * torch.sigmoid(-g)), d * silu64(g)], -1)
    return dx, term.sum(-1), y, term.abs().sum(-1)


def bounds(ends, rows):
    """[(start, end)] of every group: the running maximum of ends, within [0, rows]."""
    out, at = [], 0
    for e in ends.tolist():
        end = max(at, min(max(e, 0), rows))
        out.append((at, end))
        at = end
    return out


def mm(x, w, ends):
    """(W[e] x[t], the sums of |products|), float64; zero in no group."""
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device=x.device)
    a = torch.zeros_like(y)
    for e, (s, t) in enumerate(bounds(ends, x.shape[0])):
        if t > s:
            y[s:t] = x[s:t].double() @ w[e].double().T
            a[s:t] = x[s:t].double().abs() @ w[e].double().abs().T
    return y, a


def dgrad(dy, w, ends):
    return mm(dy, w.transpose(1, 2), ends)


def wgrad(dy, x, ends, groups):
    dw = torch.zeros(groups, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    a = torch.zeros_like(dw)
    for e, (s, t) in enumerate(bounds(ends, x.shape[0])):
        if t > s:
            dw[e] = dy[s:t].double().T @ x[s:t].double()
            a[e] = dy[s:t].double().abs().T @ x[s:t].double().abs()
    return dw, a
