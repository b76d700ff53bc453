"""MXFP4 quantisation and the grouped MXFP4 product on the GPU against their
64-bit forms, and the two together with the feed-forward block (needs a B200)."""
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


def hard(shape, dtype, seed):
    """Values of many sizes, exact ties, powers of two, zeros and extremes."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(shape, generator=g, dtype=torch.float64) * torch.exp(3 * torch.randn(shape[-1], generator=g,
                                                                                       dtype=torch.float64))
    flat = v.reshape(-1, 32)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64)
    for i in range(0, flat.shape[0], 7):
        flat[i] = ties.repeat(4) * torch.tensor([1.0, -1.0], dtype=torch.float64).repeat(16) * 2.0 ** (i % 40 - 20)
    flat[::11] = 0.0
    flat[3 % flat.shape[0]] *= 2.0 ** 100
    flat[5 % flat.shape[0]] *= 2.0 ** -110
    flat[8 % flat.shape[0]] = 2.0 ** -130   # below the smallest normal number
    return v.to(DT[dtype])


def same_values(got, want):
    g, w = got.double().cpu(), want
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(w))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (17, 4096), (129, 160), (2, 5, 64), (4097, 32)])
def test_rows(m, shape, dtype):
    x = hard(shape, dtype, seed=shape[0])
    codes, scales = ref.mx_quantize(x.double())
    c, s, v = m.quantize_mxfp4(x.cuda(), values=True)
    c2, s2 = m.quantize_mxfp4(x.cuda())
    assert torch.equal(c, c2) and torch.equal(s, s2)
    assert torch.equal(s.cpu(), scales) and torch.equal(ref.unpack(c), codes)
    same_values(v, ref.mx_values(codes, scales))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,rows,cols", [(1, 32, 1), (2, 96, 33), (3, 128, 64), (1, 160, 200), (2, 4096, 7)])
def test_weights(m, n, rows, cols, dtype):
    w = hard((n, cols, rows), dtype, seed=cols).transpose(1, 2).contiguous()
    codes, scales = ref.mx_quantize(w.double().transpose(1, 2))
    c, s, v = m.quantize_weights_mxfp4(w.cuda(), values=True)
    assert torch.equal(s.cpu(), scales) and torch.equal(ref.unpack(c), codes)
    same_values(v, ref.mx_values(codes, scales))
    c2, s2 = m.quantize_weights_mxfp4(w.cuda())
    assert torch.equal(c, c2) and torch.equal(s, s2)


def test_blocks_that_are_not_finite(m):
    x = torch.ones(4, 96, dtype=torch.float32)
    x[0, 40], x[1, 0], x[2, 95] = float("nan"), float("inf"), float("-inf")
    for dt in (torch.float32, torch.bfloat16):
        c, s, v = m.quantize_mxfp4(x.to(dt).cuda(), values=True)
        codes, scales = ref.mx_quantize(x.double())
        assert torch.equal(s.cpu(), scales) and torch.equal(ref.unpack(c), codes)
        same_values(v, ref.mx_values(codes, scales))
        c, s, v = m.quantize_weights_mxfp4(x.to(dt).t().contiguous()[None].cuda(), values=True)
        assert torch.equal(s.cpu()[0], scales) and torch.equal(ref.unpack(c)[0], codes)


def random_mx(shape, seed, spread=3):
    g = torch.Generator().manual_seed(seed)
    k = shape[-1]
    codes = torch.randint(0, 16, shape, generator=g, dtype=torch.uint8)
    scales = torch.randint(125 - spread, 126 + spread, (*shape[:-1], k // 32), generator=g, dtype=torch.uint8)
    return codes, scales


def dev_mx(c):
    return ref.pack(c[0]).cuda(), c[1].cuda()


# n, offsets (None: all rows), rows, N, K
PRODUCTS = [
    (1, None, 1, 1, 32),
    (1, None, 1, 64, 4096),
    (1, None, 17, 136, 96),
    (1, None, 200, 300, 288),
    (1, [3, 40], 50, 129, 160),
    (3, [0, 0, 1, 1], 1, 64, 64),
    (4, [2, 130, 130, 260, 263], 270, 256, 512),
    (5, [0, 64, 129, 130, 385, 642], 642, 72, 544),
    (2, [0, 31, 63], 63, 513, 1056),
    (9, [0, 1, 3, 6, 10, 15, 21, 28, 36, 45], 45, 256, 2048),
    (2, [0, 300, 300], 300, 1000, 768),
    # more tiles than SMs, and scale rows that are not whole words
    (4, [0, 500, 500, 777, 1201], 1201, 4104, 1184),
    # many rows per expert: CTA pairs, ragged ends, columns that are no whole vectors
    (1, None, 1300, 5000, 480),
    (3, [5, 300, 300, 1103], 1110, 4999, 320),
    (2, [0, 1000, 2051], 2051, 4608, 2080),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("n,offsets,R,N,K", PRODUCTS)
def test_product(m, n, offsets, R, N, K, pair, dtype):
    a, w = random_mx((R, K), 1), random_mx((n, N, K), 2)
    # small enough that the gated product stays within the types' range
    p = random_mx((n, N, K), 3) if pair else None
    want = ref.mx_matmul(ref.mx_values(*a), ref.mx_values(*w), ref.mx_values(*p) if pair else None, offsets, DT[dtype])
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    inside = slice(0, R) if offsets is None else slice(offsets[0], offsets[-1])
    layer = m.MoELayer(n, 1, 64, 64, dtype)
    try:
        out = torch.full((R, N), 7.0, dtype=DT[dtype], device="cuda")
        layer.matmul_mxfp4(dev_mx(a), dev_mx(w), pair=dev_mx(p) if pair else None, offsets=off, out=out)
        layer.sync_status()
        ref.check(out, want, inside, roundings=1, dtype=DT[dtype])
        assert (out[:inside.start] == 7).all() and (out[inside.stop:] == 7).all()
        again = layer.matmul_mxfp4(dev_mx(a), dev_mx(w), pair=dev_mx(p) if pair else None, offsets=off)
        assert torch.equal(again[inside], out[inside])
    finally:
        layer.close()


def test_scales_at_the_ends_of_their_range(m):
    """Scales far apart in one reduction, the smallest and largest codes, and NaN
    scales: of a row (its outputs only) and of a matrix column (that column)."""
    R, N, K = 5, 70, 128
    a, w = random_mx((R, K), 4), random_mx((1, N, K), 5)
    a[1][:] = torch.tensor([0, 60, 127, 200], dtype=torch.uint8)
    w[1][:] = torch.tensor([200, 190, 127, 60], dtype=torch.uint8)
    want = ref.mx_matmul(ref.mx_values(*a), ref.mx_values(*w), None, None, torch.float32)
    layer = m.MoELayer(1, 1, 64, 64, "f32")
    try:
        ref.check(layer.matmul_mxfp4(dev_mx(a), dev_mx(w)), want, dtype=torch.float32)
        a[1][2, 1] = 255
        w[1][0, 69, 0] = 255
        out = layer.matmul_mxfp4(dev_mx(a), dev_mx(w)).cpu()
        nan = torch.zeros(R, N, dtype=torch.bool)
        nan[2], nan[:, 69] = True, True
        assert torch.equal(torch.isnan(out), nan)
        ref.check(out[[0, 1, 3, 4]][:, :69], tuple(t[[0, 1, 3, 4]][:, :69] for t in want), dtype=torch.float32)
    finally:
        layer.close()


def test_scales_need_no_alignment(m):
    a, w = random_mx((9, 96), 6), random_mx((1, 50, 96), 7)
    layer = m.MoELayer(1, 1, 64, 64, "f32")
    try:
        out = []
        for shift in (0, 1):
            moved = []
            for c, s in (a, w):
                room = torch.zeros(s.numel() + 16, dtype=torch.uint8, device="cuda")
                room[shift:shift + s.numel()] = s.reshape(-1).cuda()
                moved.append((ref.pack(c).cuda(), room[shift:shift + s.numel()].view(s.shape)))
            out.append(layer.matmul_mxfp4(*moved))
            x = torch.randn(9, 96, generator=torch.Generator().manual_seed(0)).cuda()
            codes = torch.empty(9, 48, dtype=torch.uint8, device="cuda")
            room = torch.zeros(64, dtype=torch.uint8, device="cuda")
            m.moe_quantize_mxfp4(9, 96, x, m.MOE_F32, codes, room.data_ptr() + shift)
            assert torch.equal(room[shift:shift + 27].view(9, 3), m.quantize_mxfp4(x)[1])
        assert torch.equal(*out)
    finally:
        layer.close()


@pytest.mark.parametrize("bad", [[0, 50, 40], [-1, 10, 20], [0, 10, 61]])
def test_bad_offsets_are_reported(m, bad):
    a, w = random_mx((60, 64), 1), random_mx((2, 64, 64), 2)
    layer = m.MoELayer(2, 1, 64, 64, "bf16")
    try:
        out = torch.full((60, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        layer.matmul_mxfp4(dev_mx(a), dev_mx(w), offsets=torch.tensor(bad, dtype=torch.int32).cuda(), out=out)
        with pytest.raises(m.MoEError) as ei:
            layer.sync_status()
        assert ei.value.status == m.MOE_ERR_INVALID_ARG and (out == 7).all()
    finally:
        layer.close()


def test_product_refuses_tensors_that_it_would_misread(m):
    a, w = dev_mx(random_mx((8, 64), 1)), dev_mx(random_mx((2, 64, 64), 2))
    off = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    layer = m.MoELayer(2, 1, 64, 64, "bf16")
    try:
        for args, says in ((dict(a=a, w=w), "offsets is NULL"), (dict(a=a, w=(w[0][:1], w[1]), offsets=off), "w codes has shape"),
                           (dict(a=a, w=(w[0], w[1][:, :, :1]), offsets=off), "w scales has shape"),
                           (dict(a=(a[0][:, :20].contiguous(), a[1]), w=w, offsets=off), "K = 40"),
                           (dict(a=a, w=w, pair=(w[0][:, :32], w[1]), offsets=off), "pair codes has shape"),
                           (dict(a=a, w=w, offsets=off, out=torch.empty(8, 64, device="cuda")), "out is torch.float32")):
            with pytest.raises(m.MoEError) as ei:
                layer.matmul_mxfp4(**args)
            assert says in str(ei.value)
        with pytest.raises(m.MoEError) as ei:
            m.quantize_mxfp4(torch.zeros(4, 48, device="cuda"))
        assert "multiple of 32" in str(ei.value)
        with pytest.raises(m.MoEError) as ei:
            m.quantize_mxfp4(torch.zeros(4, 128, device="cuda")[:, ::2])
        assert "not contiguous" in str(ei.value)
    finally:
        layer.close()


def test_a_layer_is_trained_a_step_and_then_served_in_four_bits(m):
    """Route and dispatch with the layer, run the experts on the grouped rows, take
    the gradients, make a step, hold the new matrices in MXFP4 and multiply."""
    T, d, F, n, K = 70, 128, 192, 4, 2
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, W_g = r(T, d).bfloat16().cuda(), (r(d, n) * d ** -0.5).cuda()
    w1, w3 = ((r(n, d, F) * d ** -0.5).bfloat16().cuda() for _ in range(2))
    w2 = (r(n, F, d) * F ** -0.5).bfloat16().cuda()
    target = r(T, d).cuda()
    layer = m.MoELayer(n, K, d, F, "bf16")
    try:
        idx, gates = layer.route(x, W_g)
        counts, offsets, row_token, token_row = layer.dispatch(idx)
        rows = x[row_token.long()]
        o, gate, up = layer.ffn_forward(rows, w1, w3, w2, offsets=offsets, keep=True)
        y = (gates[..., None] * o.float()[token_row.long()]).sum(1)
        # the layer's own forward pass does the same with the same kernels' rounding of h and o
        whole = layer.forward_with_routing(x, idx, gates, w1, w3, w2)
        assert (y - whole.float()).abs().max() <= 2 * 2.0 ** -8 * y.abs().max()
        dyt = (y - target) / T
        row_gate = torch.empty(T * K, device="cuda")
        row_gate[token_row.long().reshape(-1)] = gates.reshape(-1)
        do = (row_gate[:, None] * dyt[row_token.long()]).bfloat16()
        dx, dw1, dw3, dw2 = layer.ffn_backward(do, rows, gate, up, w1, w3, w2, offsets=offsets)
        layer.sync_status()
        # 64-bit autograd of the whole layer under the same routing.  gate, up, do and
        # da, db are rounded to bf16 on the way, the gradient once more: five roundings
        leaves = [t.double().cpu().requires_grad_() for t in (x, w1, w3, w2)]
        xd, v1, v3, v2 = leaves
        loss = 0.0
        yd = torch.zeros(T, d, dtype=torch.float64)
        for k in range(K):
            for e in range(n):
                at = (idx[:, k] == e).nonzero()[:, 0].cpu()
                h = torch.nn.functional.silu(xd[at] @ v1[e]) * (xd[at] @ v3[e])
                yd = yd.index_add(0, at, gates[at.cuda(), k].double().cpu()[:, None] * (h @ v2[e]))
        loss = ((yd - target.double().cpu()) ** 2).sum() / (2 * T)
        want = torch.autograd.grad(loss, leaves)
        dxt = dx.double().cpu()[token_row.long().cpu()].sum(1)
        for got, w in zip((dxt, dw1, dw3, dw2), want):
            assert float((got.double().cpu() - w).norm() / w.norm()) <= 5 * 2.0 ** -8
        # a step, then 4 bits
        new = [(w.float() - 0.1 * dw.float()).bfloat16() for w, dw in ((w1, dw1), (w3, dw3), (w2, dw2))]
        q1, q3, q2 = (m.quantize_weights_mxfp4(w) for w in new)
        h = layer.matmul_mxfp4(m.quantize_mxfp4(rows), q1, pair=q3, offsets=offsets)
        o4 = layer.matmul_mxfp4(m.quantize_mxfp4(h), q2, offsets=offsets)
        layer.sync_status()
        qx, qh = (ref.mx_values(*ref.mx_quantize(t.double())) for t in (rows, h))
        e1, e3, e2 = (ref.mx_values(*ref.mx_quantize(w.double().transpose(1, 2))) for w in new)
        ref.check(h, ref.mx_matmul(qx, e1, e3, offsets, torch.bfloat16), roundings=1)
        ref.check(o4, ref.mx_matmul(qh, e2, None, offsets, torch.bfloat16), roundings=1)
    finally:
        layer.close()


def test_under_a_captured_graph(m):
    x = torch.randn(40, 128, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    w = dev_mx(random_mx((2, 96, 128), 2))
    off = torch.tensor([0, 13, 40], dtype=torch.int32).cuda()
    layer = m.MoELayer(2, 1, 64, 64, "bf16")
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        a = m.quantize_mxfp4(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(m.MoEError) as ei:  # no scratch yet, and none can be made here
                layer.matmul_mxfp4(a, w, offsets=off)
            assert "moe_reserve_matmul_mxfp4" in str(ei.value)
        layer.reserve_matmul_mxfp4(40, 96, 128)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = layer.matmul_mxfp4(m.quantize_mxfp4(x), w, offsets=off)
        for seed in (1, 2):
            x.copy_(torch.randn(40, 128, generator=torch.Generator().manual_seed(seed)).bfloat16())
            off.copy_(torch.tensor([0, 13, 40] if seed == 1 else [0, 40, 40], dtype=torch.int32))
            graph.replay()
            assert torch.equal(out, layer.matmul_mxfp4(m.quantize_mxfp4(x), w, offsets=off))
        layer.sync_status()
    finally:
        layer.close()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_products(m, seed):
    import random
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    dtype, pair = rng.choice(["bf16", "f32"]), rng.random() < 0.4
    n, K, N = rng.choice([1, 1, 3, 8, 30]), 32 * log(1, 90), log(1, 3000)
    offsets = [rng.choice([0, 2])]
    for _ in range(n):
        offsets.append(offsets[-1] + (0 if rng.random() < 0.2 else log(1, 900 if n < 8 else 80)))
    R = offsets[-1] + rng.choice([0, 3])
    if offsets[-1] == offsets[0]:
        return
    a, w = random_mx((R, K), seed), random_mx((n, N, K), seed + 100)
    p = random_mx((n, N, K), seed + 200) if pair else None
    want = ref.mx_matmul(ref.mx_values(*a), ref.mx_values(*w), ref.mx_values(*p) if pair else None, offsets, DT[dtype])
    layer = m.MoELayer(n, 1, 64, 64, dtype)
    try:
        out = layer.matmul_mxfp4(dev_mx(a), dev_mx(w), pair=dev_mx(p) if pair else None,
                                 offsets=torch.tensor(offsets, dtype=torch.int32).cuda())
        layer.sync_status()
        ref.check(out, want, slice(offsets[0], offsets[-1]), roundings=1, dtype=DT[dtype])
    finally:
        layer.close()


def test_a_graph_keeps_its_scratch_when_later_calls_need_more(m):
    a = random_mx((30, 64), 1)
    w, wide = dev_mx(random_mx((1, 40, 64), 2)), dev_mx(random_mx((1, 4000, 64), 3))
    layer = m.MoELayer(1, 1, 64, 64, "bf16")
    try:
        x = dev_mx(a)
        want = layer.matmul_mxfp4(x, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = layer.matmul_mxfp4(x, w)
        layer.matmul_mxfp4(x, wide)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        layer.sync_status()
    finally:
        layer.close()
