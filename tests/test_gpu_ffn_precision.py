"""fp32 outputs of the feed-forward block and of the MXFP4 product as a whole against
their 64-bit forms, at the size of error that fp32 sums have (needs a B200)."""
import pytest
import torch

import ffn_precision as prec
import ffn_reference as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    require_cuda()
    import sparse_mixture_experts_24_b200 as m
    return m


# n, offsets (None: all rows), rows, d, ffn
BLOCKS = [
    (1, None, 64, 64, 64),
    (1, None, 10, 256, 4096),                                   # few rows: groups of warps, clusters
    (1, None, 33, 4096, 192),                                   # long reductions
    (1, None, 8000, 64, 128),                                   # weight gradients over many rows
    (3, [0, 1, 1, 701], 701, 1024, 2112),
    (8, [0, 139, 244, 244, 399, 531, 700, 847, 1021], 1021, 512, 1408),
]


@pytest.mark.parametrize("n,offsets,R,d,F", BLOCKS)
def test_fp32_block(m, n, offsets, R, d, F):
    g = torch.Generator().manual_seed(R)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(x=r(R, d), w1=r(n, d, F) * d ** -0.5, w3=r(n, d, F) * d ** -0.5, w2=r(n, F, d) * F ** -0.5, dy=r(R, d),
             gate=r(R, F), up=r(R, F))
    dev = {k: v.cuda() for k, v in t.items()}
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, "f32")
    try:
        got = layer.ffn_forward(dev["x"], dev["w1"], dev["w3"], dev["w2"], offsets=off, keep=True)
        want = prec.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets)
        for k, v in zip(("y", "gate", "up"), got):
            prec.check(v, want[k])
        args = ("dy", "x", "gate", "up", "w1", "w3", "w2")
        got = layer.ffn_backward(*(dev[k] for k in args), offsets=off)
        want = prec.ffn_backward(*(t[k] for k in args), offsets)
        for k, v in zip(("dx", "dw1", "dw3", "dw2"), got):
            prec.check(v, want[k])
        layer.sync_status()
    finally:
        layer.close()


# n, offsets, rows, N, K: one CTA per tile of 64 and 128 rows, CTA pairs
PRODUCTS = [
    (1, None, 17, 136, 96),
    (1, None, 40, 200, 4096),
    (2, [0, 100, 231], 231, 300, 1056),
    (1, None, 1051, 4608, 2080),
]


@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("n,offsets,R,N,K", PRODUCTS)
def test_fp32_outputs_of_the_mxfp4_product(m, n, offsets, R, N, K, pair):
    g = torch.Generator().manual_seed(K)

    def mx(*shape, mid):
        codes = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
        # 12 binades of scales in one reduction: the sums are not exact in fp32
        scales = torch.randint(mid - 6, mid + 6, (*shape[:-1], K // 32), generator=g, dtype=torch.uint8)
        return (ref.pack(codes).cuda(), scales.cuda()), ref.mx_values(codes, scales)

    (a, av), (w, wv) = mx(R, K, mid=127), mx(n, N, K, mid=118)
    p, pv = mx(n, N, K, mid=118) if pair else (None, None)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, 64, 64, "f32")
    try:
        out = layer.matmul_mxfp4(a, w, pair=p, offsets=off)
        layer.sync_status()
        prec.mx_check(out, prec.mx_matmul(av, wv, pv, offsets))
    finally:
        layer.close()
