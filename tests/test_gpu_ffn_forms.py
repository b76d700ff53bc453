"""Kernel forms that only larger arrays or many experts reach, and calls that the other
tests do not make (needs a B200)."""
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m():
    require_cuda()
    import sparse_mixture_experts_24_b200 as m
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1201, 8224), (310001, 32)])
def test_rows_that_fill_the_machine(m, rows, cols, dtype):
    """From 8 blocks of 256 threads per SM on, a thread takes four pieces of eight elements:
    the codes, scales and values of small calls on slices of the same rows, and (their
    first and last rows) of the 64-bit form.  Neither size is whole rounds of pieces."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert rows * cols // 8 >= sms * 8 * 256 * 4 and rows * cols // 8 % 1024
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(
        3 * torch.randn(cols, generator=g, device="cuda"))
    x[::7] = 0.0
    x[5, 3], x[rows - 2, cols - 1] = float("nan"), float("inf")
    x = x.to(DT[dtype])
    got = m.quantize_mxfp4(x, values=True)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], m.quantize_mxfp4(x)))
    step = max(1, 100000 // cols)
    for r in range(0, rows, step):
        for a, b in zip(got, m.quantize_mxfp4(x[r:r + step], values=True)):
            assert torch.equal(a[r:r + step].nan_to_num(7.0), b.nan_to_num(7.0))
    for part in (slice(0, 12), slice(rows - 12, rows)):
        codes, scales = ref.mx_quantize(x[part].double().cpu())
        assert torch.equal(got[1][part].cpu(), scales) and torch.equal(ref.unpack(got[0][part]), codes)
        want = ref.mx_values(codes, scales)
        assert torch.equal(got[2][part].double().cpu().nan_to_num(7.0), want.nan_to_num(7.0))


def random_mx(shape, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
    scales = torch.randint(122, 129, (*shape[:-1], shape[-1] // 32), generator=g, dtype=torch.uint8)
    return codes, scales


# counts of rows, columns, K: tiles of 256 columns and of 64 rows (at most 48 rows per
# expert on average) or 128 rows, as many as SMs or more
MANY_EXPERTS = [
    ([17, 0, 1, 100, 64, 65, 3, 30] * 5, 1000, 288),
    ([17, 0, 1, 100, 64, 65, 3, 30] * 5, 1003, 544),
    ([300, 0, 129, 1, 128] * 4, 2056, 320),
    ([300, 0, 129, 1, 128] * 4, 2059, 1184),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N,K", MANY_EXPERTS)
def test_products_of_many_experts(m, counts, N, K, dtype):
    n, offsets = len(counts), [2]
    for c in counts:
        offsets.append(offsets[-1] + c)
    R = offsets[-1] + 3
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    height = 64 if R <= 48 * n else 128
    assert max(-(-R // height), min(n, R)) * -(-N // 256) >= sms and R < 256 * n
    a, w = random_mx((R, K), 1), random_mx((n, N, K), 2)
    want = ref.mx_matmul(ref.mx_values(*a), ref.mx_values(*w), None, offsets, DT[dtype])
    layer = m.MoELayer(n, 1, 64, 64, dtype)
    try:
        out = torch.full((R, N), 7.0, dtype=DT[dtype], device="cuda")
        layer.matmul_mxfp4((ref.pack(a[0]).cuda(), a[1].cuda()), (ref.pack(w[0]).cuda(), w[1].cuda()),
                           offsets=torch.tensor(offsets, dtype=torch.int32).cuda(), out=out)
        layer.sync_status()
        ref.check(out, want, slice(2, R - 3), roundings=1, dtype=DT[dtype])
        assert (out[:2] == 7).all() and (out[R - 3:] == 7).all()
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,d,F", [
    ([0, 0, 180, 0, 0, 0, 0, 0], 192, 320),          # far above the average that the rules go by
    ([0, 1500, 0, 0, 3, 0, 0, 1], 256, 448),
    ([2, 0, 700, 1] + [0] * 60, 128, 192),
])
def test_one_expert_gets_nearly_every_row(m, counts, d, F, dtype):
    n, R = len(counts), sum(counts)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    g = torch.Generator().manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).cuda()  # noqa: E731
    x, dy, gate, up = r(R, d), r(R, d), r(R, F), r(R, F)
    w1, w3, w2 = r(n, d, F) * d ** -0.5, r(n, d, F) * d ** -0.5, r(n, F, d) * F ** -0.5
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        want = ref.ffn_forward(x, w1, w3, w2, offsets, DT[dtype])
        for k, v in zip(("y", "gate", "up"), layer.ffn_forward(x, w1, w3, w2, offsets=off, keep=True)):
            ref.check(v, want[k], dtype=DT[dtype])
        want = ref.ffn_backward(dy, x, gate, up, w1, w3, w2, offsets, DT[dtype])
        for k, v in zip(("dx", "dw1", "dw3", "dw2"), layer.ffn_backward(dy, x, gate, up, w1, w3, w2, offsets=off)):
            ref.check(v, want[k], dtype=DT[dtype])
        layer.sync_status()
    finally:
        layer.close()


def test_inside_an_autograd_function(m):
    """The two calls wrapped as a user would: torch's own backward pass gives them the
    gradient of what follows and hands theirs on."""
    n, d, F, R = 3, 128, 192, 90
    off = torch.tensor([0, 31, 31, 90], dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, "bf16")

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w1, w3, w2):
            y, gate, up = layer.ffn_forward(x, w1, w3, w2, offsets=off, keep=True)
            ctx.save_for_backward(x, gate, up, w1, w3, w2)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, gate, up, w1, w3, w2 = ctx.saved_tensors
            return layer.ffn_backward(dy.contiguous(), x, gate, up, w1, w3, w2, offsets=off)

    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    leaves = [t.bfloat16().cuda().requires_grad_() for t in (
        r(R, d), r(n, d, F) * d ** -0.5, r(n, d, F) * d ** -0.5, r(n, F, d) * F ** -0.5)]
    weight = r(R, d).bfloat16().cuda()
    try:
        got = torch.autograd.grad((Block.apply(*leaves) * weight).sum(), leaves)
        with torch.no_grad():
            _, gate, up = layer.ffn_forward(*leaves, offsets=off, keep=True)
        want = ref.ffn_backward(weight, leaves[0].detach(), gate, up, *(t.detach() for t in leaves[1:]),
                                off.tolist(), torch.bfloat16)
        for k, v in zip(("dx", "dw1", "dw3", "dw2"), got):
            ref.check(v, want[k])
        with pytest.raises(m.MoEError) as ei:
            layer.ffn_forward(*leaves, offsets=off)
        assert "x requires a gradient" in str(ei.value)
        layer.sync_status()
    finally:
        layer.close()
