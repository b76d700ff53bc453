"""The 64-bit forms that the feed-forward and MXFP4 kernels are tested against,
on the CPU: gradients against autograd, the format against hand-worked values."""
import torch

import ffn_reference as ref


def test_backward_form_equals_autograd():
    g = torch.Generator().manual_seed(0)
    n, d, F, offsets = 3, 8, 12, [1, 4, 4, 9]
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w1, w3, w2, dy = r(10, d), r(n, d, F), r(n, d, F), r(n, F, d), r(10, d)
    leaves = [t.requires_grad_() for t in (x, w1, w3, w2)]
    loss = 0.0
    gate, up = torch.zeros(10, F, dtype=torch.float64), torch.zeros(10, F, dtype=torch.float64)
    for e, s in enumerate(ref.segments(offsets, n, 10)):
        a, b = x[s] @ w1[e], x[s] @ w3[e]
        gate[s], up[s] = a.detach(), b.detach()
        loss = loss + ((torch.nn.functional.silu(a) * b) @ w2[e] * dy[s]).sum()
    want = torch.autograd.grad(loss, leaves)
    with torch.no_grad():
        got = ref.ffn_backward(dy, x, gate, up, w1, w3, w2, offsets, torch.float32)
    for k, v in zip(("dx", "dw1", "dw3", "dw2"), want):
        assert torch.allclose(got[k][0], v, rtol=1e-12, atol=1e-12)
    assert (got["dx"][0][0] == 0).all() and (got["dx"][0][9] == 0).all()  # rows outside the segments
    assert (got["dw1"][0][1] == 0).all()                                   # an expert without rows


def test_format_values_worked_by_hand():
    v = torch.zeros(7, 32, dtype=torch.float64)
    v[0, :9] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.3])   # scale 1: ties to even codes
    v[1, :2] = torch.tensor([7.9, -7.0])                                          # above 6: to 6
    v[2, :2] = torch.tensor([8.0, 1.0])                                           # scale 2
    v[3, 0] = 2.0 ** -140                                                         # the smallest scale
    v[4, 0] = float("nan")
    v[5, 3] = float("inf")
    codes, scales = ref.mx_quantize(v)
    assert scales[:, 0].tolist() == [127, 127, 128, 0, 255, 255, 0]
    assert codes[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8 | 1]
    assert codes[1, :2].tolist() == [7, 15]
    assert codes[2, :2].tolist() == [6, 1]
    assert codes[3, 0] == 0 and not codes[4:].any()
    val = ref.mx_values(codes, scales)
    assert val[0, :9].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -0.5]
    assert torch.isnan(val[4]).all() and torch.isnan(val[5]).all() and val[2, 1] == 1.0
    assert torch.equal(ref.unpack(ref.pack(codes)), codes)
