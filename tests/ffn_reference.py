"""64-bit forms of the gated feed-forward block over expert segments and of
MXFP4, for the tests: plain torch, one expert at a time, with bounds on what
the kernels may be off by.

Bounds.  u is the largest relative error of one rounding to the type (half of
torch.finfo(t).eps); a sum of K products in fp32, in any order and rounded to
nearest or toward zero, is off by at most K * 2^-23 times the sum of the
magnitudes.  1 / (1 + e^-a) in fp32 from the library exponential is off by less
than 2^-20 of itself.  Every bound adds these up through the formulas."""
import torch

F32_STEP = 2.0 ** -23
SIGMOID = 2.0 ** -20


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def segments(offsets, n, rows):
    o = [0, rows] if offsets is None else [int(v) for v in offsets]
    return [slice(o[e], o[e + 1]) for e in range(n)]


def ffn_forward(x, w1, w3, w2, offsets, dtype):
    """-> {name: (value, bound)} of y, gate, up; rows outside the segments zero."""
    u = unit(dtype)
    R, d = x.shape
    n, _, F = w1.shape
    out = {k: (torch.zeros(R, c, dtype=torch.float64), torch.zeros(R, c, dtype=torch.float64))
           for k, c in (("y", d), ("gate", F), ("up", F))}
    x, w1, w3, w2 = (t.double().cpu() for t in (x, w1, w3, w2))
    for e, s in enumerate(segments(offsets, n, R)):
        xe = x[s]
        a, b = xe @ w1[e], xe @ w3[e]
        da, db = (d * F32_STEP * (xe.abs() @ w[e].abs()) for w in (w1, w3))
        sig = torch.sigmoid(a)
        h = a * sig * b
        # |d silu / d a| <= 1.1
        dh = 1.1 * da * b.abs() + (a * sig).abs() * db + (SIGMOID + u) * h.abs()
        y = h @ w2[e]
        mag = h.abs() @ w2[e].abs()
        out["y"][0][s], out["y"][1][s] = y, u * y.abs() + dh @ w2[e].abs() + F * F32_STEP * mag
        out["gate"][0][s], out["gate"][1][s] = a, u * a.abs() + da
        out["up"][0][s], out["up"][1][s] = b, u * b.abs() + db
    return out


def ffn_backward(dy, x, gate, up, w1, w3, w2, offsets, dtype):
    """-> {name: (value, bound)} of dx, dw1, dw3, dw2."""
    u = unit(dtype)
    R, d = x.shape
    n, _, F = w1.shape
    dy, x, gate, up, w1, w3, w2 = (t.double().cpu() for t in (dy, x, gate, up, w1, w3, w2))
    res = {"dx": (torch.zeros_like(x), torch.zeros_like(x))}
    for k, w in (("dw1", w1), ("dw3", w3), ("dw2", w2)):
        res[k] = (torch.zeros_like(w), torch.zeros_like(w))
    for e, s in enumerate(segments(offsets, n, R)):
        xe, g, a, b = x[s], dy[s], gate[s], up[s]
        rows = xe.shape[0]
        sig = torch.sigmoid(a)
        dh = g @ w2[e].T
        ddh = d * F32_STEP * (g.abs() @ w2[e].abs().T)
        h, silu, slope = a * sig * b, a * sig, sig * (1 + a * (1 - sig))
        db, da = dh * silu, dh * b * slope
        # the slope's own error: s and 1 - s each within SIGMOID of 1
        eh = (SIGMOID + u) * h.abs()
        eb = ddh * silu.abs() + (SIGMOID + u) * db.abs()
        ea = ddh * (b * slope).abs() + u * da.abs() + 4 * SIGMOID * (dh * b).abs() * (1 + a.abs()) * sig
        dx = da @ w1[e].T + db @ w3[e].T
        mag = da.abs() @ w1[e].abs().T + db.abs() @ w3[e].abs().T
        res["dx"][0][s] = dx
        res["dx"][1][s] = u * dx.abs() + ea @ w1[e].abs().T + eb @ w3[e].abs().T + 2 * F * F32_STEP * mag
        for k, left, right, eleft, eright in (("dw1", xe, da, None, ea), ("dw3", xe, db, None, eb),
                                              ("dw2", h, g, eh, None)):
            v = left.T @ right
            tol = u * v.abs() + rows * F32_STEP * (left.abs().T @ right.abs())
            tol += left.abs().T @ eright if eright is not None else eleft.T @ right.abs()
            res[k][0][e], res[k][1][e] = v, tol
    return res


def check(got, want, rows=None, roundings=2, dtype=torch.bfloat16):
    """Every value within its bound, and (bf16: `roundings` roundings on the way,
    each at most u of its value and independent, so their 2-norm is at most
    that many u of the result's) the whole within roundings * u."""
    value, bound = want
    g = got.double().cpu()
    if rows is not None:
        g, value, bound = g[rows], value[rows], bound[rows]
    over = (g - value).abs() - bound
    assert not torch.isnan(g).any()
    assert (over <= 1e-30).all(), "worst %.3g over a bound of %.3g" % (
        float(over.max()), float(bound.reshape(-1)[int(over.argmax())]))
    norm = float(value.norm())
    if dtype == torch.bfloat16 and norm > 0:
        rel = float((g - value).norm()) / norm
        assert rel <= roundings * unit(dtype), "relative 2-norm of the error %.3g" % rel


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx_quantize(v):
    """[..., k] float64 -> (codes uint8 [..., k] one per element, scale codes
    [..., k/32]), block by block from the definition."""
    b = v.double().cpu().reshape(*v.shape[:-1], -1, 32)
    finite = torch.isfinite(b).all(-1)
    b = torch.where(finite.unsqueeze(-1), b, torch.zeros_like(b))
    m = b.abs().amax(-1)
    exponent = torch.frexp(m).exponent.to(torch.int64) - 1
    c = torch.where(m > 0, (exponent - 2 + 127).clamp(0, 254), torch.zeros_like(exponent))
    z = torch.ldexp(b.abs(), (127 - c).unsqueeze(-1))
    grid = torch.tensor(E2M1, dtype=torch.float64)
    gap = (z.clamp(max=6.0).unsqueeze(-1) - grid).abs()
    near = gap.min(-1).values
    # the nearest; of two equally near ones the even code
    tie = (gap == near.unsqueeze(-1))
    idx = torch.arange(8)
    even = (tie & (idx % 2 == 0)).long().argmax(-1)
    first = tie.long().argmax(-1)
    code = torch.where(tie.sum(-1) > 1, even, first) | torch.where(torch.signbit(b), 8, 0)
    c = torch.where(finite, c, torch.full_like(c, 255))
    code = torch.where(finite.unsqueeze(-1), code, torch.zeros_like(code))
    return code.reshape(v.shape).to(torch.uint8), c.to(torch.uint8)


def mx_values(codes, scales):
    """Element codes [..., k] and scale codes [..., k/32] -> float64 values."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64)
    q = table[codes.long().cpu()].reshape(*codes.shape[:-1], -1, 32)
    s = scales.long().cpu().unsqueeze(-1)
    v = torch.ldexp(q, s - 127)
    return torch.where(s == 255, torch.full_like(v, float("nan")), v).reshape(codes.shape)


def unpack(codes):
    """Packed codes [..., k/2] -> one code per element [..., k]."""
    c = codes.cpu()
    return torch.stack([c & 15, c >> 4], -1).flatten(-2)


def pack(codes):
    c = codes.reshape(*codes.shape[:-1], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous()


def mx_matmul(a, w, pair, offsets, dtype):
    """a [R][k], w, pair [n][N][k] float64 values -> (value, bound)."""
    u = unit(dtype)
    n, N, k = w.shape
    value = torch.zeros(a.shape[0], N, dtype=torch.float64)
    bound = torch.zeros_like(value)
    for e, s in enumerate(segments(offsets, n, a.shape[0])):
        v, t = a[s] @ w[e].T, k * F32_STEP * (a[s].abs() @ w[e].abs().T)
        if pair is not None:
            p, tp = a[s] @ pair[e].T, k * F32_STEP * (a[s].abs() @ pair[e].abs().T)
            silu = v * torch.sigmoid(v)
            t = 1.1 * t * p.abs() + silu.abs() * tp + SIGMOID * (silu * p).abs()
            v = silu * p
        value[s], bound[s] = v, t + u * v.abs()
    return value, bound
