"""How far fp32 results may lie from the 64-bit forms as a whole (relative 2-norm): the
statistics of fp32 rounding, far closer than the worst case of every single value that
ffn_reference.py bounds (which grows with K, these with the root of K).

One rounding to nearest of s is off by at most half a unit in the last place, at most
U |s| (U = 2^-24), spread evenly: variance at most U^2 s^2 / 3.  A sum of K products
t_1 .. t_K of random signs, added one after the other by fused multiply-adds, has
partial sums of variance t_1^2 + .. + t_k^2; over all K roundings and orders on average
(K + 1) / 2 of the whole, so

    variance of the sum's error  <=  U^2 / 6 (K + 1) (t_1^2 + .. + t_K^2)

and less for sums in several parts.  Errors go on through the formulas by their
derivatives, their variances adding up.  The elementwise part: the exponential is
within 2 units in the last place (4 U), every operation after it within U.

SPREAD is what the 2-norm of a result of at least 64 values may lie above its expected
size: its relative deviation is at most 1 / sqrt(2 * 64), 0.09; five of those are 1.45."""
import torch

U = 2.0 ** -24
SPREAD = 1.5


def _sum(k, squares):
    return U * U / 6 * (k + 1) * squares


def _segments(offsets, n, rows):
    o = [0, rows] if offsets is None else [int(v) for v in offsets]
    return [slice(o[e], o[e + 1]) for e in range(n)]


def ffn_forward(x, w1, w3, w2, offsets):
    """-> {name: (value, variance of its error)} of y, gate, up in 64 bits."""
    x, w1, w3, w2 = (t.double().cpu() for t in (x, w1, w3, w2))
    (R, d), (n, _, F) = x.shape, w1.shape
    out = {k: (torch.zeros(R, c, dtype=torch.float64), torch.zeros(R, c, dtype=torch.float64))
           for k, c in (("y", d), ("gate", F), ("up", F))}
    for e, s in enumerate(_segments(offsets, n, R)):
        a, b = x[s] @ w1[e], x[s] @ w3[e]
        va, vb = (_sum(d, x[s] ** 2 @ w[e] ** 2) for w in (w1, w3))
        sig = torch.sigmoid(a)
        silu = a * sig
        # a / (1 + e^-a) b: 4 U of the exponential, U of the sum, quotient and product
        vh = va * (sig * (1 + a * (1 - sig)) * b) ** 2 + vb * silu ** 2 + (7 * U * silu * b) ** 2
        for k, v, var in (("gate", a, va), ("up", b, vb),
                          ("y", (silu * b) @ w2[e], vh @ w2[e] ** 2 + _sum(F, (silu * b) ** 2 @ w2[e] ** 2))):
            out[k][0][s], out[k][1][s] = v, var
    return out


def ffn_backward(dy, x, gate, up, w1, w3, w2, offsets):
    """-> {name: (value, variance of its error)} of dx, dw1, dw3, dw2 in 64 bits."""
    dy, x, gate, up, w1, w3, w2 = (t.double().cpu() for t in (dy, x, gate, up, w1, w3, w2))
    (R, d), (n, _, F) = x.shape, w1.shape
    out = {k: (torch.zeros_like(t), torch.zeros_like(t)) for k, t in (("dx", x), ("dw1", w1), ("dw3", w3), ("dw2", w2))}
    for e, s in enumerate(_segments(offsets, n, R)):
        xe, g, a, b = x[s], dy[s], gate[s], up[s]
        dh, vdh = g @ w2[e].T, _sum(d, g ** 2 @ (w2[e] ** 2).T)
        sig = torch.sigmoid(a)  # within 6 U
        rest = 1 + a * (1 - sig)
        h, db, da = a * sig * b, dh * a * sig, dh * b * sig * rest
        vh, vdb = (8 * U * h) ** 2, vdh * (a * sig) ** 2 + (8 * U * db) ** 2
        # 1 - s is off by 6 U s + U (1 - s), its product with a by another U
        off = (dh * b).abs() * sig * (a.abs() * (6 * sig + 2 * (1 - sig)) + 10 * rest.abs()) * U
        vda = vdh * (b * sig * rest) ** 2 + off ** 2
        out["dx"][0][s] = da @ w1[e].T + db @ w3[e].T
        out["dx"][1][s] = (_sum(2 * F, da ** 2 @ (w1[e] ** 2).T + db ** 2 @ (w3[e] ** 2).T)
                           + vda @ (w1[e] ** 2).T + vdb @ (w3[e] ** 2).T)
        for k, left, right, vleft, vright in (("dw1", xe, da, 0 * xe, vda), ("dw3", xe, db, 0 * xe, vdb),
                                              ("dw2", h, g, vh, 0 * g)):
            out[k][0][e] = left.T @ right
            out[k][1][e] = (_sum(xe.shape[0], (left ** 2).T @ right ** 2) + (left ** 2).T @ vright
                            + vleft.T @ right ** 2)
    return out


def check(got, want, rows=None):
    """The 2-norm of the error within SPREAD of its expected size."""
    value, var = want
    g = got.double().cpu()
    if rows is not None:
        g, value, var = g[rows], value[rows], var[rows]
    assert value.numel() >= 64
    error, limit = float((g - value).norm()), SPREAD * float(var.sum().sqrt())
    assert error <= limit, "relative 2-norm of the error %.3g over %.3g" % (
        error / float(value.norm()), limit / float(value.norm()))


def mx_matmul(a, w, pair, offsets):
    """fp32 outputs of the MXFP4 product: a [R][k], w, pair [n][N][k] float64 values ->
    (value, size of its error).  The products are exact; the accumulator is truncated
    once per 64 of K, by up to a unit in the last place (2 U |s|) and evenly spread, so by
    2 U / sqrt(3) of the partial sum in the root of the mean square, all toward zero: the
    sizes add up.  The gated pair divides within 4 U more than the block above."""
    (R, k), (n, N, _) = a.shape, w.shape
    value, size = torch.zeros(R, N, dtype=torch.float64), torch.zeros(R, N, dtype=torch.float64)

    def product(x, m):
        s, e = torch.zeros(x.shape[0], N, dtype=torch.float64), torch.zeros(x.shape[0], N, dtype=torch.float64)
        for k0 in range(0, k, 64):
            s = s + x[:, k0:k0 + 64] @ m[:, k0:k0 + 64].T
            e += 2 * U / 3 ** 0.5 * s.abs()
        return s, e

    for e, s in enumerate(_segments(offsets, n, R)):
        v, ev = product(a[s], w[e])
        if pair is not None:
            p, ep = product(a[s], pair[e])
            sig = torch.sigmoid(v)
            silu = v * sig
            ev = ev * (sig * (1 + v * (1 - sig)) * p).abs() + ep * silu.abs() + 11 * U * (silu * p).abs()
            v = silu * p
        value[s], size[s] = v, ev
    return value, size


def mx_check(got, want, rows=slice(None)):
    value, size = (t[rows] for t in want)
    error, limit = float((got.double().cpu()[rows] - value).norm()), float(size.norm())
    assert error <= limit, "relative 2-norm of the error %.3g over %.3g" % (
        error / float(value.norm()), limit / float(value.norm()))
