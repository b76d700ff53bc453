"""Batches whose arrays have more than 2^31 elements: every offset that passes 32 bits
(needs a B200; holds up to 85 GB)."""
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROWS, EDGE = 34_000_003, 300


@pytest.fixture(scope="module")
def m():
    require_cuda()
    import sparse_mixture_experts_24_b200 as m
    return m


def long(cols, dtype, seed):
    """Random first and last rows, zeros between -> the whole, and those rows together."""
    g = torch.Generator().manual_seed(seed)
    ends = torch.randn(2 * EDGE, cols, generator=g).to(DT[dtype])
    t = torch.zeros(ROWS, cols, dtype=DT[dtype], device="cuda")
    t[:EDGE], t[-EDGE:] = ends[:EDGE].cuda(), ends[EDGE:].cuda()
    return t, ends


def ends_of(t):
    """First and last rows; what lies between must be zero."""
    for r in range(EDGE, ROWS - EDGE, 1 << 22):
        assert not t[r:min(r + (1 << 22), ROWS - EDGE)].any()
    return torch.cat([t[:EDGE], t[-EDGE:]])


# the middle expert holds all but a few rows
OFFSETS, SHORT = [0, 5, ROWS - 100, ROWS], [0, 5, 2 * EDGE - 100, 2 * EDGE]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block(m, dtype):
    n, d, F = 3, 64, 64
    assert ROWS * d > 2 ** 31
    g = torch.Generator().manual_seed(9)
    w1, w3, w2 = ((torch.randn(n, 64, 64, generator=g) / 8).to(DT[dtype]).cuda() for _ in range(3))
    off = torch.tensor(OFFSETS, dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        x, sx = long(d, dtype, 1)
        want = ref.ffn_forward(sx, w1, w3, w2, SHORT, DT[dtype])
        for k, v in zip(("y", "gate", "up"), layer.ffn_forward(x, w1, w3, w2, offsets=off, keep=True)):
            ref.check(ends_of(v), want[k], dtype=DT[dtype])
        del v
        (dy, sdy), (gate, sgate), (up, sup) = (long(64, dtype, seed) for seed in (2, 3, 4))
        want = ref.ffn_backward(sdy, sx, sgate, sup, w1, w3, w2, SHORT, DT[dtype])
        for k, v in zip(("dx", "dw1", "dw3", "dw2"), layer.ffn_backward(dy, x, gate, up, w1, w3, w2, offsets=off)):
            ref.check(ends_of(v) if k == "dx" else v, want[k], dtype=DT[dtype])
        layer.sync_status()
    finally:
        layer.close()
        torch.cuda.empty_cache()


def test_mxfp4(m):
    n, K, N = 3, 128, 64
    assert ROWS * K // 2 > 2 ** 31 and ROWS * N > 2 ** 31
    g = torch.Generator().manual_seed(5)
    w = (torch.randn(n, K, N, generator=g) / 8).bfloat16()
    q = m.quantize_weights_mxfp4(w.cuda())
    off = torch.tensor(OFFSETS, dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, 64, 64, "bf16")
    try:
        x, sx = long(K, "bf16", 1)
        a = m.quantize_mxfp4(x)
        codes, scales = ref.mx_quantize(sx.double())
        assert torch.equal(ref.unpack(ends_of(a[0])), codes) and torch.equal(ends_of(a[1]).cpu(), scales)
        del x
        want = ref.mx_matmul(ref.mx_values(codes, scales), ref.mx_values(*ref.mx_quantize(w.double().transpose(1, 2))),
                             None, SHORT, torch.bfloat16)
        ref.check(ends_of(layer.matmul_mxfp4(a, q, offsets=off)), want, roundings=1)
        layer.sync_status()
    finally:
        layer.close()
        torch.cuda.empty_cache()
