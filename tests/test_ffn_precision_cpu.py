"""The whole-result bounds on fp32 outputs (ffn_precision.py) on the CPU: plain fp32
stands within them, products of fewer bits do not."""
import pytest
import torch

import ffn_precision as prec


def tf32(t):
    """To 10 fraction bits, to nearest (ties away: the operands are random)."""
    return ((t.float().contiguous().view(torch.int32) + 0x1000) & ~0x1FFF).view(torch.float32).double()


def split(t):
    hi = t.bfloat16().double()
    return hi, (t.double() - hi).bfloat16().double()


def product_tf32(a, b):
    return tf32(a) @ tf32(b)


def product_split(a, b):
    """Two bf16 parts each, without the product of the two small ones."""
    (a1, a2), (b1, b2) = split(a), split(b)
    return a1 @ b1 + a1 @ b2 + a2 @ b1


def product_f32(a, b):
    return a.float() @ b.float()


def block(x, w1, w3, w2, dy, gate, up, mm):
    """The block with every product by mm, the rest in the product's type."""
    a, b = mm(x, w1), mm(x, w3)
    y = mm(a * torch.sigmoid(a) * b, w2)
    sig = torch.sigmoid(gate.to(a.dtype))
    dh = mm(dy, w2.T)
    h, db = gate * sig * up, dh * gate * sig
    da = dh * up * sig * (1 + gate * (1 - sig))
    dx = mm(torch.cat([da, db], 1), torch.cat([w1.T, w3.T], 0))
    return dict(gate=a, up=b, y=y, dx=dx, dw1=mm(x.T, da), dw3=mm(x.T, db), dw2=mm(h.T, dy))


@pytest.mark.parametrize("R,d,F", [(64, 64, 64), (200, 256, 192), (1024, 512, 704), (96, 1792, 1024), (64, 640, 2816)])
def test_plain_fp32_passes_and_fewer_bits_do_not(R, d, F):
    g = torch.Generator().manual_seed(R + d)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w1, w3, w2 = r(R, d), r(d, F) * d ** -0.5, r(d, F) * d ** -0.5, r(F, d) * F ** -0.5
    dy, gate, up = r(R, d), r(R, F), r(R, F)
    w = [t[None] for t in (w1, w3, w2)]
    want = {**prec.ffn_forward(x, *w, None), **prec.ffn_backward(dy, x, gate, up, *w, None)}
    for k, v in block(x, w1, w3, w2, dy, gate, up, product_f32).items():
        prec.check(v if v.shape == want[k][0].shape else v[None], want[k])
    for mm in (product_tf32, product_split):
        for k, v in block(x, w1, w3, w2, dy, gate, up, mm).items():
            with pytest.raises(AssertionError, match="2-norm"):
                prec.check(v if v.shape == want[k][0].shape else v[None], want[k])


@pytest.mark.parametrize("k", [96, 1024, 4096])
@pytest.mark.parametrize("pair", [False, True])
def test_mxfp4_bound_is_one_truncation_per_step(k, pair):
    """An accumulator truncated to 24 bits once per 64 of K stands within the bound, one of
    20 bits does not."""
    g = torch.Generator().manual_seed(k)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).float().double()  # noqa: E731
    a, w, p = r(40, k), r(1, 50, k) * k ** -0.5, r(1, 50, k) * k ** -0.5 if pair else None

    def cut(t, bits):
        m, e = torch.frexp(t)
        return torch.ldexp(torch.trunc(torch.ldexp(m, torch.tensor(bits))), e - bits)

    def accumulate(m, bits):
        s = torch.zeros(40, 50, dtype=torch.float64)
        for k0 in range(0, k, 64):
            s = cut(s + a[:, k0:k0 + 64] @ m[0, :, k0:k0 + 64].T, bits)
        return s

    want = prec.mx_matmul(a, w, p, None)
    for bits in (24, 20):
        v = accumulate(w, bits)
        if pair:
            v = v * torch.sigmoid(v) * accumulate(p, bits)
        if bits == 24:
            prec.mx_check(v, want)
        else:
            with pytest.raises(AssertionError, match="2-norm"):
                prec.mx_check(v, want)
