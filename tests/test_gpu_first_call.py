"""A handle's first call, on a stream of the caller's while the default stream is busy
(needs a B200): what the library initialises must not land in the middle of it."""
import pytest
import torch

from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    require_cuda()
    import sparse_mixture_experts_24_b200 as m
    return m


def occupy_default_stream(products=40):
    """Some tens of milliseconds of work on the default stream (8,192-cubed products of
    about 0.8 ms), which a side stream does not wait for.  The operands are returned:
    they are to live as long."""
    a = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(a)
    for _ in range(products):
        torch.mm(a, a, out=out)
    return a, out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_workspace_is_not_wiped_under_a_first_call(m, dtype):
    T, n, K, d, F = 96, 8, 2, 128, 192
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, W_g = r(T, d).to(dt).cuda(), (r(d, n) * d ** -0.5).cuda()
    w1, w3 = ((r(n, d, F) * d ** -0.5).to(dt).cuda() for _ in range(2))
    w2 = (r(n, F, d) * F ** -0.5).to(dt).cuda()
    layers = [m.MoELayer(n, K, d, F, dtype) for _ in range(2)]
    try:
        want = layers[0].forward(x, W_g, w1, w3, w2)
        layers[0].sync_status()
        side = torch.cuda.Stream()
        outs = [tuple(torch.empty_like(t) for t in want) for _ in range(400)]
        torch.cuda.synchronize()
        busy = occupy_default_stream()
        for y, idx, gates in outs:
            layers[1].forward(x, W_g, w1, w3, w2, y=y, topk_idx=idx, topk_w=gates, stream=side)
        layers[1].sync_status(side)
        torch.cuda.synchronize()
        del busy
        for got in outs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        for layer in layers:
            layer.close()


@pytest.mark.parametrize("reserve", [False, True])
@pytest.mark.parametrize("call", ["ffn_forward", "ffn_backward", "matmul_mxfp4"])
def test_a_first_call_reports_its_bad_offsets(m, call, reserve):
    """Nothing that was queued before the call may clear the status that it sets, nor
    may the report of one call clear the next one's."""
    n, d, F, R = 2, 64, 128, 60
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    x, gate, up, w1, w3, w2 = r(R, d), r(R, F), r(R, F), r(n, d, F), r(n, d, F), r(n, F, d)
    a, w = m.quantize_mxfp4(x), m.quantize_weights_mxfp4(w1)
    bad = torch.tensor([0, 50, 40], dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, "bf16")
    try:
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        busy = occupy_default_stream()
        if reserve:
            layer.reserve_ffn(R)
            layer.reserve_matmul_mxfp4(R, F, d)
        for _ in range(3):
            if call == "ffn_forward":
                layer.ffn_forward(x, w1, w3, w2, offsets=bad, stream=side)
            elif call == "ffn_backward":
                layer.ffn_backward(x, x, gate, up, w1, w3, w2, offsets=bad, stream=side)
            else:
                layer.matmul_mxfp4(a, w, offsets=bad, stream=side)
            with pytest.raises(m.MoEError) as ei:
                layer.sync_status(side)
            assert ei.value.status == m.MOE_ERR_INVALID_ARG and "offsets" in str(ei.value)
        torch.cuda.synchronize()
        layer.sync_status(side)
        del busy
    finally:
        layer.close()
