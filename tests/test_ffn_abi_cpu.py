"""What the feed-forward and MXFP4 entry points refuse on the host (CPU only:
none of these calls reaches the GPU)."""
import pytest

GOOD = 1 << 20  # a 16-byte aligned stand-in address; never dereferenced


@pytest.fixture(scope="module")
def m():
    import sparse_mixture_experts_24_b200 as m
    return m


@pytest.fixture()
def h(m):
    h = m.moe_create(8, 2, 128, 256, m.MOE_BF16)
    yield h
    m.moe_destroy(h)


def refused(m, call, *args, says):
    with pytest.raises(m.MoEError) as ei:
        call(*args)
    assert ei.value.status == m.MOE_ERR_INVALID_ARG
    assert says in str(ei.value)


def forward_args(h, **change):
    a = dict(h=h, R=4, offsets=GOOD, x=GOOD, w1=GOOD, w3=GOOD, w2=GOOD, gate=None, up=None, y=GOOD, stream=0)
    a.update(change)
    return list(a.values())


def backward_args(h, **change):
    a = dict(h=h, R=4, offsets=GOOD, x=GOOD, w1=GOOD, w3=GOOD, w2=GOOD, gate=GOOD, up=GOOD, dy=GOOD, dx=GOOD,
             dw1=GOOD, dw3=GOOD, dw2=GOOD, stream=0)
    a.update(change)
    return list(a.values())


def matmul_args(h, **change):
    a = dict(h=h, R=4, N=64, K=64, offsets=GOOD, a_codes=GOOD, a_scales=GOOD, w_codes=GOOD, w_scales=GOOD,
             pair_codes=None, pair_scales=None, out=GOOD, stream=0)
    a.update(change)
    return list(a.values())


@pytest.mark.parametrize("change,says", [
    (dict(R=-1), "R = -1 < 0"),
    (dict(R=2 ** 31 - 256), "exceeds 2^31 - 257"),
    (dict(x=None), "x is NULL"),
    (dict(w1=GOOD + 8), "w1 is not 16-byte aligned"),
    (dict(w3=None), "w3 is NULL"),
    (dict(w2=None), "w2 is NULL"),
    (dict(y=GOOD + 4), "y is not 16-byte aligned"),
    (dict(gate=GOOD), "gate and up must both"),
    (dict(gate=GOOD, up=GOOD + 2), "up is not 16-byte aligned"),
])
def test_forward_refusals(m, h, change, says):
    refused(m, m.moe_ffn_forward, *forward_args(h, **change), says=says)


@pytest.mark.parametrize("change,says", [
    (dict(R=-3), "R = -3 < 0"),
    (dict(dw3=None), "dw1, dw3 and dw2 must all"),
    (dict(dx=None, dw1=None, dw3=None, dw2=None), "neither dx nor"),
    (dict(gate=None), "gate is NULL"),
    (dict(up=GOOD + 8), "up is not 16-byte aligned"),
    (dict(dy=None), "dy is NULL"),
    (dict(dx=GOOD + 8), "dx is not 16-byte aligned"),
    (dict(R=0, dw2=GOOD + 8), "dw2 is not 16-byte aligned"),
])
def test_backward_refusals(m, h, change, says):
    refused(m, m.moe_ffn_backward, *backward_args(h, **change), says=says)


@pytest.mark.parametrize("change,says", [
    (dict(R=-1), "R = -1 < 0"),
    (dict(N=0), "N = 0"),
    (dict(N=2 ** 20 + 1), "outside [1, 1048576]"),
    (dict(K=48), "K = 48"),
    (dict(K=0), "K = 0"),
    (dict(pair_codes=GOOD), "pair_codes and pair_scales must both"),
    (dict(a_codes=GOOD + 8), "a_codes is not 16-byte aligned"),
    (dict(w_codes=None), "w_codes is NULL"),
    (dict(a_scales=None), "a_scales is NULL"),
    (dict(w_scales=None), "w_scales is NULL"),
    (dict(out=None), "out is NULL"),
])
def test_matmul_refusals(m, h, change, says):
    refused(m, m.moe_matmul_mxfp4, *matmul_args(h, **change), says=says)


def test_null_handles_and_nothing_to_do(m, h):
    for call, args in ((m.moe_ffn_forward, forward_args(None)), (m.moe_ffn_backward, backward_args(None)),
                       (m.moe_matmul_mxfp4, matmul_args(None)), (m.moe_reserve_ffn, (None, 4, 1))):
        refused(m, call, *args, says="null handle")
    refused(m, m.moe_reserve_ffn, h, -1, 1, says="R_max = -1")
    refused(m, m.moe_reserve_ffn, h, 4, 2, says="backward = 2")
    refused(m, m.moe_reserve_matmul_mxfp4, None, 4, 64, 64, 0, says="null handle")
    refused(m, m.moe_reserve_matmul_mxfp4, h, -4, 64, 64, 0, says="R_max = -4")
    refused(m, m.moe_reserve_matmul_mxfp4, h, 4, 0, 64, 0, says="N = 0")
    refused(m, m.moe_reserve_matmul_mxfp4, h, 4, 64, 65, 0, says="K = 65")
    refused(m, m.moe_reserve_matmul_mxfp4, h, 4, 64, 64, 3, says="pair = 3")
    m.moe_reserve_matmul_mxfp4(h, 0, 64, 64, 1)
    # nothing to do: no pointer is looked at
    m.moe_reserve_ffn(h, 0, 1)
    m.moe_ffn_forward(h, 0, None, None, None, None, None, None, None, None, 0)
    m.moe_matmul_mxfp4(h, 0, 64, 64, None, None, None, None, None, None, None, None, 0)
    m.moe_quantize_mxfp4(0, 64, None, m.MOE_BF16, None, None, None, 0)


@pytest.mark.parametrize("args,says", [
    ((-1, 64, GOOD, 1, GOOD, GOOD, None, 0), "rows = -1"),
    ((4, 48, GOOD, 1, GOOD, GOOD, None, 0), "cols = 48"),
    ((4, 0, GOOD, 1, GOOD, GOOD, None, 0), "cols = 0"),
    ((4, 64, GOOD, 5, GOOD, GOOD, None, 0), "dtype = 5"),
    ((4, 64, GOOD + 2, 1, GOOD, GOOD, None, 0), "x is not 16-byte aligned"),
    ((4, 64, GOOD, 1, None, GOOD, None, 0), "codes is NULL"),
    ((4, 64, GOOD, 1, GOOD, None, None, 0), "scales is NULL"),
    ((4, 64, GOOD, 1, GOOD, GOOD, GOOD + 4, 0), "values is not 16-byte aligned"),
])
def test_quantize_refusals(m, args, says):
    refused(m, m.moe_quantize_mxfp4, *args, says=says)


@pytest.mark.parametrize("args,says", [
    ((0, 64, 64, GOOD, 1, GOOD, GOOD, None, 0), "n = 0"),
    ((1, 40, 64, GOOD, 1, GOOD, GOOD, None, 0), "rows = 40"),
    ((1, 64, 0, GOOD, 1, GOOD, GOOD, None, 0), "cols = 0"),
    ((1, 64, 64, GOOD, 3, GOOD, GOOD, None, 0), "dtype = 3"),
    ((1, 64, 64, None, 1, GOOD, GOOD, None, 0), "w is NULL"),
])
def test_quantize_weights_refusals(m, args, says):
    refused(m, m.moe_quantize_weights_mxfp4, *args, says=says)


def test_tensor_wrappers_refuse_what_the_abi_would_misread(m):
    import torch
    layer = m.MoELayer(2, 1, 64, 64, "bf16")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    for call in (lambda: layer.ffn_forward(x, w, w, w), lambda: layer.ffn_backward(x, x, x, x, w, w, w),
                 lambda: m.quantize_mxfp4(x), lambda: m.quantize_weights_mxfp4(w),
                 lambda: layer.matmul_mxfp4((x.view(torch.uint8), x), (w.view(torch.uint8), w))):
        with pytest.raises(m.MoEError) as ei:
            call()
        assert ei.value.status == m.MOE_ERR_INVALID_ARG and "not a CUDA tensor" in str(ei.value)
    layer.close()
