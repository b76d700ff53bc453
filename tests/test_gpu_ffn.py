"""The gated feed-forward block over expert segments, forward and backward, on
the GPU against its 64-bit form (needs a B200)."""
import pytest
import torch

import ffn_reference as ref
from gpu_helpers import require_cuda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("dx", "dw1", "dw3", "dw2")


@pytest.fixture(scope="module")
def m():
    require_cuda()
    import sparse_mixture_experts_24_b200 as m
    return m


def make(n, R, d, F, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    t = dict(x=r(R, d), w1=r(n, d, F) * d ** -0.5, w3=r(n, d, F) * d ** -0.5, w2=r(n, F, d) * F ** -0.5, dy=r(R, d),
             gate=r(R, F), up=r(R, F))
    return {k: v.to(DT[dtype]).cuda() for k, v in t.items()}


def offsets_of(counts, before=0):
    o = [before]
    for c in counts:
        o.append(o[-1] + c)
    return o


# (n, counts or None for one dense segment, rows before and after, d, ffn)
SHAPES = [
    (1, None, 1, 0, 0, 64, 64),
    (1, None, 130, 0, 0, 192, 320),
    (1, [37], 37, 5, 9, 64, 192),
    (3, [0, 1, 0], 1, 0, 0, 128, 64),
    (4, [127, 0, 129, 3], 259, 0, 7, 256, 192),
    (5, [64, 65, 1, 255, 257], 642, 3, 0, 320, 448),
    (8, [16, 15, 17, 0, 33, 32, 31, 2], 146, 1, 1, 192, 576),
    (2, [300, 513], 813, 0, 0, 512, 256),
    (33, [7, 0, 1] * 11, 88, 0, 0, 64, 128),
    (256, [1, 0, 2, 0] * 64, 192, 2, 1, 64, 64),
    # few rows: reductions split over clusters of 2, 4 and 8, one and several row blocks
    (1, None, 5, 0, 0, 1024, 1536),
    (1, None, 2, 0, 0, 64, 4096),
    (2, [40, 3], 43, 0, 2, 1024, 704),
    (3, [90, 0, 131], 221, 4, 0, 576, 1088),
    (2, [150, 300], 450, 1, 2, 640, 1792),
    (1, None, 276, 0, 0, 640, 3584),
    # narrow outputs, many rows: weight gradients split over clusters too
    (1, None, 3000, 0, 0, 192, 320),
    (2, [1500, 0], 1500, 3, 70, 128, 64),
    # fp32 tiles of 16, 32 and more rows, split over the block's warps
    (4, [17, 33, 16, 49], 115, 0, 1, 256, 512),
    # more tiles than SMs: every CTA pair runs several, through both accumulators
    (3, [700, 0, 1001], 1701, 0, 3, 1024, 2112),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,counts,rows,before,after,d,F", SHAPES)
def test_forward_and_backward(m, n, counts, rows, before, after, d, F, dtype):
    R = before + rows + after
    t = make(n, R, d, F, dtype, seed=n * 1000 + rows)
    host = None if counts is None else offsets_of(counts, before)
    off = None if host is None else torch.tensor(host, dtype=torch.int32).cuda()
    inside = slice(before, before + rows) if host is not None else slice(0, R)
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        want = ref.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], host, DT[dtype])
        only = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off)
        y, gate, up = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True)
        layer.sync_status()
        assert torch.equal(only[inside], y[inside])
        for k, v in (("y", y), ("gate", gate), ("up", up)):
            ref.check(v, want[k], inside, roundings=2, dtype=DT[dtype])
        want = ref.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), host, DT[dtype])
        got = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off)
        layer.sync_status()
        for k, v in zip(NAMES, got):
            ref.check(v, want[k], inside if k == "dx" else None, roundings=2, dtype=DT[dtype])
        again = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off)
        part = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off,
                                  need_dx=False)
        for i, (a, b) in enumerate(zip(got, again)):
            assert torch.equal(a[inside] if i == 0 else a, b[inside] if i == 0 else b)
        assert part[0] is None and all(torch.equal(a, b) for a, b in zip(got[1:], part[1:]))
        alone = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off,
                                   need_dw=False)
        assert alone[1:] == (None, None, None) and torch.equal(alone[0][inside], got[0][inside])
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_outside_the_segments_are_left_alone(m, dtype):
    n, d, F, R = 2, 64, 128, 150
    t = make(n, R, d, F, dtype)
    off = torch.tensor([3, 100, 140], dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        y, dx = torch.full_like(t["x"], 7.0), torch.full_like(t["x"], 7.0)
        gate, up = torch.full_like(t["gate"], 7.0), torch.full_like(t["gate"], 7.0)
        dw = [torch.empty_like(t[k]) for k in ("w1", "w3", "w2")]
        m.moe_ffn_forward(layer.h, R, off, t["x"], t["w1"], t["w3"], t["w2"], gate, up, y)
        m.moe_ffn_backward(layer.h, R, off, t["x"], t["w1"], t["w3"], t["w2"], t["gate"], t["up"], t["dy"], dx, *dw)
        layer.sync_status()
        for v in (y, dx, gate, up):
            assert (v[:3] == 7).all() and (v[140:] == 7).all() and not (v[3:140] == 7).all()
    finally:
        layer.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_stays_with_its_expert(m, bad):
    """Segments end inside the kernels' tiles: the next expert's rows, and rows
    past the last segment, lie in the same tiles."""
    n, d, F, R = 3, 128, 128, 200
    t = make(n, R, d, F, "bf16")
    off = torch.tensor([0, 70, 71, 190], dtype=torch.int32).cuda()
    args = ("dy", "x", "gate", "up", "w1", "w3", "w2")
    layer = m.MoELayer(n, 1, d, F, "bf16")
    try:
        clean = layer.ffn_backward(*(t[k] for k in args), offsets=off)
        y0 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off)
        for k in ("x", "dy", "gate", "up"):
            t[k][70] = bad
            t[k][190:] = bad
        got = layer.ffn_backward(*(t[k] for k in args), offsets=off)
        y1 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off)
        layer.sync_status()
        keep = [i for i in range(190) if i != 70]
        assert torch.equal(y0[keep], y1[keep]) and torch.equal(clean[0][keep], got[0][keep])
        for a, b in zip(clean[1:], got[1:]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
            assert not torch.isfinite(b[1]).any()  # infinite or NaN, as the formula has it
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,rows,d,F", [
    ([2, 70, 71, 190], 200, 512, 1024),      # 256 x 256 tiles for the weight gradients
    ([5, 1007, 1090, 2001], 2030, 128, 64),  # reductions over rows split over clusters
    ([1, 9, 12, 30], 33, 640, 1216),         # few rows
    ([0, 300, 310, 700], 705, 640, 1792),    # several row blocks, split reductions
])
def test_bad_experts_and_bad_rows_outside_stay_there(m, off, rows, d, F, dtype):
    t = make(3, rows, d, F, dtype)
    offsets = torch.tensor(off, dtype=torch.int32).cuda()
    args = ("dy", "x", "gate", "up", "w1", "w3", "w2")
    layer = m.MoELayer(3, 1, d, F, dtype)
    try:
        clean = layer.ffn_backward(*(t[k] for k in args), offsets=offsets)
        y0 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=offsets)
        for k in ("x", "dy", "gate", "up"):
            t[k][: off[0]] = float("nan")
            t[k][off[1] : off[2]] = float("nan")
            t[k][off[3] :] = float("nan")
        got = layer.ffn_backward(*(t[k] for k in args), offsets=offsets)
        y1 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=offsets)
        layer.sync_status()
        for part in (slice(off[0], off[1]), slice(off[2], off[3])):
            assert torch.equal(y0[part], y1[part]) and torch.equal(clean[0][part], got[0][part])
        for a, b in zip(clean[1:], got[1:]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.isnan(b[1]).all()
    finally:
        layer.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [[0, 50, 40, 60], [-1, 10, 20, 30], [0, 10, 20, 61], [5, 2 ** 31 - 1, -7, 0]])
def test_bad_offsets_are_reported_and_nothing_is_addressed(m, bad, dtype):
    n, d, F, R = 3, 64, 64, 60
    t = make(n, R, d, F, dtype)
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        off = torch.tensor(bad, dtype=torch.int32).cuda()
        y = torch.full_like(t["x"], 7.0)
        m.moe_ffn_forward(layer.h, R, off, t["x"], t["w1"], t["w3"], t["w2"], None, None, y)
        with pytest.raises(m.MoEError) as ei:
            layer.sync_status()
        assert ei.value.status == m.MOE_ERR_INVALID_ARG and "offsets" in str(ei.value)
        assert (y == 7).all()
        got = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off)
        with pytest.raises(m.MoEError):
            layer.sync_status()
        assert all((g == 0).all() for g in got[1:])
        layer.sync_status()  # the report is cleared
    finally:
        layer.close()


def test_no_rows(m):
    layer = m.MoELayer(2, 1, 64, 128, "bf16")
    try:
        t = make(2, 1, 64, 128, "bf16")
        x, f = t["x"][:0], t["gate"][:0]
        off = torch.zeros(3, dtype=torch.int32).cuda()
        assert layer.ffn_forward(x, t["w1"], t["w3"], t["w2"], offsets=off).shape == (0, 64)
        dx, *dw = layer.ffn_backward(x, x, f, f, t["w1"], t["w3"], t["w2"], offsets=off)
        assert dx.shape == (0, 64) and all((w == 0).all() for w in dw)
        # rows, all of them outside the segments
        t = make(2, 5, 64, 128, "bf16")
        _, *dw = layer.ffn_backward(*(t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")), offsets=off)
        assert all((w == 0).all() for w in dw)
    finally:
        layer.close()


def test_gradients_against_differences(m):
    """d/de of sum(dy * y(x + e p, w + e q)) by central differences of the fp32
    forward pass.  With unit-size directions the third derivative along them is
    of the size of the first, so a step of 2^-5 truncates to about 2^-10 / 6 of
    it; y's own error (2^-20 of the sum's root-mean-square terms) over the step
    adds 2^-15: 1e-2 of the gradient's scale holds both with room."""
    n, d, F, R = 2, 64, 128, 96
    t = make(n, R, d, F, "f32", seed=5)
    off = torch.tensor([0, 40, 96], dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, "f32")
    try:
        _, gate, up = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True)
        grads = layer.ffn_backward(t["dy"], t["x"], gate, up, t["w1"], t["w3"], t["w2"], offsets=off)
        g = torch.Generator().manual_seed(9)
        for i, k in enumerate(("x", "w1", "w3", "w2")):
            p = torch.randn(t[k].shape, generator=g).cuda() * (1.0 if k == "x" else t[k].std())
            want = float((grads[i].double() * p.double()).sum())
            step = 2.0 ** -5
            at = []
            for sign in (1, -1):
                u = {**t, k: t[k] + sign * step * p}
                y = layer.ffn_forward(u["x"], u["w1"], u["w3"], u["w2"], offsets=off)
                at.append(float((t["dy"].double() * y.double()).sum()))
            got = (at[0] - at[1]) / (2 * step)
            scale = float(grads[i].double().norm() * p.double().norm()) / p.numel() ** 0.5
            assert abs(got - want) <= 1e-2 * max(abs(want), scale), (k, got, want)
    finally:
        layer.close()


def test_under_a_captured_graph_and_on_another_stream(m):
    n, d, F, R = 3, 128, 192, 150
    t = make(n, R, d, F, "bf16", seed=3)
    off = torch.tensor([0, 61, 61, 150], dtype=torch.int32).cuda()
    args = ("dy", "x", "gate", "up", "w1", "w3", "w2")
    layer = m.MoELayer(n, 1, d, F, "bf16")
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(m.MoEError) as ei:  # no room yet, and none can be made here
                layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off)
            assert "moe_reserve_ffn" in str(ei.value)
        layer.reserve_ffn(R)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y, gate, up = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True)
            grads = layer.ffn_backward(t["dy"], t["x"], gate, up, t["w1"], t["w3"], t["w2"], offsets=off)
        # a later, larger call replaces the workspace: the graph keeps the old one
        big = make(n, 600, d, F, "bf16", seed=4)
        layer.ffn_backward(*(big[k] for k in args), offsets=torch.tensor([0, 200, 400, 600], dtype=torch.int32).cuda())
        for seed in (3, 8):
            new = make(n, R, d, F, "bf16", seed=seed)
            for k in t:
                t[k].copy_(new[k])
            off.copy_(torch.tensor([0, 61, 61, 150] if seed == 3 else [0, 20, 130, 149], dtype=torch.int32))
            graph.replay()
            torch.cuda.synchronize()
            y2, g2, u2 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True)
            e2 = layer.ffn_backward(t["dy"], t["x"], g2, u2, t["w1"], t["w3"], t["w2"], offsets=off)
            last = int(off[-1])
            assert torch.equal(y[:last], y2[:last]) and torch.equal(grads[0][:last], e2[0][:last])
            assert all(torch.equal(a, b) for a, b in zip(grads[1:], e2[1:]))
        # another stream than the tensors' own
        side.wait_stream(torch.cuda.current_stream())
        y3 = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, stream=side)
        side.synchronize()
        assert torch.equal(y3[:last], y2[:last])
        layer.sync_status()
    finally:
        layer.close()


def test_refuses_tensors_that_it_would_misread(m):
    n, d, F = 2, 64, 128
    t = make(n, 8, d, F, "bf16")
    off = torch.tensor([0, 4, 8], dtype=torch.int32).cuda()
    layer = m.MoELayer(n, 1, d, F, "bf16")
    args = dict(x=t["x"], w1=t["w1"], w3=t["w3"], w2=t["w2"], offsets=off)
    try:
        for change, says in ((dict(x=t["x"].float()), "x is torch.float32"),
                             (dict(x=t["x"][:, :32]), "shape"),
                             (dict(x=t["dy"].new_zeros(8, 2 * d)[:, ::2]), "not contiguous"),
                             (dict(w1=t["w1"][:1]), "w1 has shape"),
                             (dict(w2=t["w2"].transpose(1, 2)), "w2 has shape"),
                             (dict(offsets=off.long()), "offsets is torch.int64"),
                             (dict(offsets=off[:2]), "offsets has shape"),
                             (dict(offsets=None), "offsets is NULL"),
                             (dict(y=t["x"][:4]), "y has shape")):
            with pytest.raises(m.MoEError) as ei:
                layer.ffn_forward(**{**args, **change})
            assert ei.value.status == m.MOE_ERR_INVALID_ARG and says in str(ei.value)
        with pytest.raises(m.MoEError) as ei:
            layer.ffn_backward(t["dy"], t["x"], t["gate"][:, :64], t["up"], t["w1"], t["w3"], t["w2"], offsets=off)
        assert "gate has shape" in str(ei.value)
    finally:
        layer.close()


def test_two_layers_at_once_on_two_streams(m):
    """Handles share nothing: calls of two of them, interleaved on two streams with
    growing batches, give what they give one after the other."""
    n, d, F = 3, 192, 320
    layers = [m.MoELayer(n, 1, d, F, "bf16") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    try:
        jobs = []
        for i, R in enumerate((40, 300, 150, 700)):
            for k in range(2):
                t = make(n, R, d, F, "bf16", seed=10 * i + k)
                off = torch.tensor([0, R // 3, R // 2 + k, R], dtype=torch.int32).cuda()
                jobs.append((k, t, off))
        torch.cuda.synchronize()

        def run(k, t, off, stream):
            y, gate, up = layers[k].ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True,
                                                stream=stream)
            return (y, *layers[k].ffn_backward(t["dy"], t["x"], gate, up, t["w1"], t["w3"], t["w2"], offsets=off,
                                               stream=stream))

        both = [run(k, t, off, streams[k] if i % 4 else streams[k].cuda_stream) for i, (k, t, off) in enumerate(jobs)]
        torch.cuda.synchronize()
        for (k, t, off), got in zip(jobs, both):
            assert all(torch.equal(a, b) for a, b in zip(got, run(k, t, off, None)))
        for layer in layers:
            layer.sync_status()
    finally:
        for layer in layers:
            layer.close()


@pytest.mark.parametrize("seed", range(12))
def test_drawn_sizes(m, seed):
    import random
    rng = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    dtype = rng.choice(["bf16", "bf16", "f32"])
    n, d, F = rng.choice([1, 1, 2, 5, 9, 40]), 64 * log(1, 20), 64 * log(1, 24)
    counts = [0 if rng.random() < 0.2 else log(1, 600 if n < 9 else 60) for _ in range(n)]
    before, after = rng.choice([(0, 0), (1, 5)])
    host = None if n == 1 and not before else offsets_of(counts, before)
    R = before + sum(counts) + after
    if host is None:
        R = max(R, 1)
    if R == 0:
        return
    t = make(n, R, d, F, dtype, seed=seed)
    off = None if host is None else torch.tensor(host, dtype=torch.int32).cuda()
    inside = slice(0, R) if host is None else slice(host[0], host[-1])
    layer = m.MoELayer(n, 1, d, F, dtype)
    try:
        want = ref.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], host, DT[dtype])
        got = layer.ffn_forward(t["x"], t["w1"], t["w3"], t["w2"], offsets=off, keep=True)
        for k, v in zip(("y", "gate", "up"), got):
            ref.check(v, want[k], inside, dtype=DT[dtype])
        args = [t[k] for k in ("dy", "x", "gate", "up", "w1", "w3", "w2")]
        want = ref.ffn_backward(*args, host, DT[dtype])
        for k, v in zip(NAMES, layer.ffn_backward(*args, offsets=off)):
            ref.check(v, want[k], inside if k == "dx" else None, dtype=DT[dtype])
        layer.sync_status()
    finally:
        layer.close()
