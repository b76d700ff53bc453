"""Cases, plain forms and 64-bit forms of the operators that train an expert's
gated feed-forward block and then hold and multiply its matrices in 4 bits:

  ffn_forward    y = (silu(x . w1) * (x . w3)) . w2 over expert segments of rows,
                 with the two projections kept for the backward pass or not
  ffn_backward   dx, dw1, dw3, dw2 from dy and the kept projections
  quantize       MXFP4: E2M1 values with a power-of-two scale per 32 elements
  matmul         the product of MXFP4 rows with the MXFP4 matrices of their expert,
                 plain or as the gated pair silu(x . w1) * (x . w3)

Rows of expert e are offsets[e] .. offsets[e+1]-1 of the row-major inputs;
weights are [n][in][out] as the layer has them, and their MXFP4 form is
[n][out][in/2] codes with [n][out][in/32] scales.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a shared (dense) expert serving one token: the three matrices are streamed once
        dict(name="ffn_one_token", op="ffn_forward", dtype="bf16", n=1, rows=1, d=4096, ffn=14336, keep=False),
        # a decode batch of 64 rows over 8 experts
        dict(name="ffn_decode_8_experts", op="ffn_forward", dtype="bf16", n=8, rows=64, d=4096, ffn=14336, keep=False),
        # the training forward of a prefill-sized batch: 4,096 tokens, two experts each
        dict(name="ffn_train_8_experts", op="ffn_forward", dtype="bf16", n=8, rows=8192, d=4096, ffn=14336, keep=True),
        # the backward pass of the same batch
        dict(name="ffn_bwd_8_experts", op="ffn_backward", dtype="bf16", n=8, rows=8192, d=4096, ffn=14336),
        # many small experts: 128 of 2,048 x 768, about 128 rows each, ragged
        dict(name="ffn_bwd_128_experts", op="ffn_backward", dtype="bf16", n=128, rows=16384, d=2048, ffn=768),
        # an fp32 layer in training, with odd row counts
        dict(name="ffn_bwd_f32", op="ffn_backward", dtype="f32", n=8, rows=1021, d=512, ffn=1408),
        # activations of a decode batch: the smallest call
        dict(name="quant_decode_rows", op="quantize", dtype="bf16", form="rows", n=1, rows=32, cols=4096),
        # hidden rows of a prefill batch, as the values that the 4-bit layer would see
        dict(name="quant_prefill_rows", op="quantize", dtype="bf16", form="rows", n=1, rows=8191, cols=14336),
        # one set of expert matrices [in][out], blocks along the reduction
        dict(name="quant_weights", op="quantize", dtype="f32", form="weights", n=8, rows=2048, cols=768),
        # a decode batch through one dense 4-bit matrix
        dict(name="mx_decode", op="matmul", dtype="bf16", n=1, rows=17, k=4096, cols=14336, pair=False),
        # the gate and up projections of a prefill batch over 8 experts, with the gated product
        dict(name="mx_prefill_pair", op="matmul", dtype="bf16", n=8, rows=8192, k=4096, cols=14336, pair=True),
        # the down projection of many small experts, fp32 out
        dict(name="mx_128_experts", op="matmul", dtype="f32", n=128, rows=4099, k=768, cols=2048, pair=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_forward", "ffn_forward", "ffn_backward", "ffn_backward", "quantize", "matmul", "matmul"])
    if op in ("ffn_forward", "ffn_backward"):
        if rng.random() < 0.2:
            c = dict(op=op, dtype="f32", n=rng.choice([1, 2, 5, 8]), rows=_log(rng, 1, 1500),
                     d=64 * _log(rng, 2, 12), ffn=64 * _log(rng, 2, 24))
        else:
            n = rng.choice([1, 1, 2, 3, 8, 8, 32, 128])
            # matrices get smaller as there are more of them, rows have all sizes
            d = 64 * _log(rng, 2, 64 if n <= 8 else 32)
            ffn = 64 * _log(rng, 2, 224 if n <= 8 else 16)
            c = dict(op=op, dtype="bf16", n=n, rows=_log(rng, 1, 8192), d=d, ffn=ffn)
        if op == "ffn_forward":
            c["keep"] = rng.random() < 0.5
        return c
    if op == "quantize":
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), form=rng.choice(["rows", "rows", "weights"]))
        if c["form"] == "rows":
            c.update(n=1, rows=_log(rng, 1, 8192), cols=32 * _log(rng, 2, 448))
        else:
            c.update(n=rng.choice([1, 2, 8]), rows=32 * _log(rng, 2, 128), cols=32 * _log(rng, 2, 128))
        return c
    n = rng.choice([1, 1, 2, 8, 32, 128])
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), n=n, rows=_log(rng, 1, 8192),
                k=32 * _log(rng, 2, 128 if n <= 8 else 64), cols=8 * _log(rng, 4, 1024 if n <= 8 else 256),
                pair=rng.random() < 0.4)


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("ffn_forward", "ffn_backward"):
        r, d, f = c["rows"], c["d"], c["ffn"]
        used = min(c["n"], r)  # an expert without rows is not read
        if c["op"] == "ffn_forward":
            rows = 2 * r * d + (2 * r * f if c["keep"] else 0)
            return {"bytes": size * (3 * used * d * f + rows), "flops": 6 * r * d * f}
        return {"bytes": size * (3 * used * d * f + 3 * c["n"] * d * f + 3 * r * d + 2 * r * f), "flops": 12 * r * d * f}
    if c["op"] == "quantize":
        e = c["n"] * c["rows"] * c["cols"]
        return {"bytes": 2 * size * e + e // 32, "flops": 4 * e}
    r, k, o = c["rows"], c["k"], c["cols"]
    mats = (2 if c["pair"] else 1) * min(c["n"], r)
    return {"bytes": 2 * r * k + mats * o * (k // 2 + k // 32) + size * r * o, "flops": 2 * (2 if c["pair"] else 1) * r * k * o}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _segments(n, rows, seed):
    """Ragged row counts of n experts that sum to `rows`, one of them empty
    where there are more than four."""
    g = torch.Generator().manual_seed(seed)
    p = 0.6 + 0.8 * torch.rand(n, generator=g, dtype=torch.float64)
    if n > 4:
        p[int(torch.randint(n, (1,), generator=g))] = 0.0
    edge = torch.round(torch.cumsum(p, 0) / p.sum() * rows).to(torch.int64)
    return torch.cat([torch.zeros(1, dtype=torch.int64), edge]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = {"case": case}
    if case["op"] == "quantize":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        # channels of very different sizes, and some empty rows
        x = normal(n, rows, cols, dtype=torch.float32)
        x *= torch.exp(1.5 * torch.randn(1, 1, cols, generator=g, device="cuda"))
        x[:, ::13, : cols // 2] = 0
        s["x"] = x.to(dt) if case["form"] == "weights" else x[0].to(dt)
        return s
    n, rows = case["n"], case["rows"]
    host = _segments(n, rows, seed)
    off = host.cuda()
    expert = torch.searchsorted(off[1:].contiguous(), torch.arange(rows, device="cuda", dtype=torch.int32), right=True)
    s["offsets"] = None if n == 1 else off
    # where row r stands in a [n][most rows of an expert] layout
    s["expert"], s["place"] = expert, torch.arange(rows, device="cuda") - off[expert].long()
    s["most"] = max(1, int((host[1:] - host[:-1]).max()))
    if case["op"] == "matmul":
        k, o = case["k"], case["cols"]
        s["x"] = (normal(rows, k, dtype=torch.float32)
                  * torch.exp(0.5 * torch.randn(1, k, generator=g, device="cuda"))).to(torch.bfloat16)
        mats = []
        for _ in range(2 if case["pair"] else 1):
            codes = torch.randint(0, 256, (n, o, k // 2), generator=g, device="cuda", dtype=torch.uint8)
            # about 1 / sqrt(k) with the E2M1 values' own spread of about 3
            mid = 127 - round(math.log2(3 * math.sqrt(k)))
            scales = torch.randint(mid - 1, mid + 2, (n, o, k // 32), generator=g, device="cuda", dtype=torch.uint8)
            mats.append((codes, scales))
        s["w"], s["w_pair"] = mats[0], (mats[1] if case["pair"] else None)
        if own:
            import sparse_mixture_experts_24_b200 as m
            s["layer"] = m.MoELayer(n, 1, 64, 64, case["dtype"])
        return s
    d, f = case["d"], case["ffn"]
    s["x"] = normal(rows, d)
    s["w1"], s["w3"] = normal(n, d, f, scale=d ** -0.5), normal(n, d, f, scale=d ** -0.5)
    s["w2"] = normal(n, f, d, scale=f ** -0.5)
    if case["op"] == "ffn_backward":
        s["dy"] = normal(rows, d)
        xp = _spread(s["x"], s)
        s["gate"], s["up"] = _gather(torch.bmm(xp, s["w1"]), s), _gather(torch.bmm(xp, s["w3"]), s)
    if own:
        import sparse_mixture_experts_24_b200 as m
        s["layer"] = m.MoELayer(n, 1, d, f, case["dtype"])
        s["layer"].reserve_ffn(rows)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _spread(rows, s):
    """[rows][c] -> [n][most][c], zeros behind each expert's last row."""
    out = torch.zeros(s["case"]["n"], s["most"], rows.shape[1], dtype=rows.dtype, device=rows.device)
    out[s["expert"], s["place"]] = rows
    return out


def _gather(p, s):
    return p[s["expert"], s["place"]]


def _plain_ffn_forward(s):
    dt = s["x"].dtype
    xp = _spread(s["x"].float(), s)
    gate, up = torch.bmm(xp, s["w1"].float()), torch.bmm(xp, s["w3"].float())
    y = _gather(torch.bmm(gate * torch.sigmoid(gate) * up, s["w2"].float()), s).to(dt)
    if not s["case"]["keep"]:
        return {"y": y}
    return {"y": y, "gate": _gather(gate, s).to(dt), "up": _gather(up, s).to(dt)}


def _plain_ffn_backward(s):
    dt = s["x"].dtype
    xp, dyp = _spread(s["x"].float(), s), _spread(s["dy"].float(), s)
    gate, up = _spread(s["gate"].float(), s), _spread(s["up"].float(), s)
    sig = torch.sigmoid(gate)
    dh = torch.bmm(dyp, s["w2"].float().transpose(1, 2))
    dw2 = torch.bmm((gate * sig * up).transpose(1, 2), dyp).to(dt)
    dup = dh * gate * sig
    dgate = dh * up * sig * (1 + gate * (1 - sig))
    del dh
    dx = torch.bmm(dgate, s["w1"].float().transpose(1, 2)) + torch.bmm(dup, s["w3"].float().transpose(1, 2))
    xt = xp.transpose(1, 2)
    return {"dx": _gather(dx, s).to(dt), "dw1": torch.bmm(xt, dgate).to(dt), "dw3": torch.bmm(xt, dup).to(dt), "dw2": dw2}


def _plain_mxfp4(v):
    """[..., k] -> the E2M1 values (sign and magnitude) and the scale codes of
    blocks of 32: scale 2^(floor(log2 max) - 2), nearest value, ties to even,
    magnitudes above 6 to 6."""
    b = v.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(top)[1] - 3 + 127
    e = torch.where(top > 0, e, torch.zeros_like(e)).clamp(0, 254)
    # 2^(127 - e) as two exact factors: the whole may lie outside fp32
    half = (127 - e).div(2, rounding_mode="floor")
    a = b.abs() * _power(half) * _power(127 - e - half)
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5).float() + (a >= 3.5) + 2 * (a > 5).float()
    q = torch.where(b.signbit(), -q, q)
    return q, e.squeeze(-1).to(torch.uint8)


def _power(e):
    """2^e for whole e within fp32's normal range, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scaled(q, e):
    """E2M1 values [..., k/32, 32] times 2^(e - 127), exactly (zero blocks have e = 0)."""
    e = e.to(torch.int32).unsqueeze(-1) - 127
    half = e.div(2, rounding_mode="floor")
    return (q * _power(half) * _power(e - half)).flatten(-2)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_decode(codes, scales):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    q = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return _scaled(q.unflatten(-1, (-1, 32)), scales)


def _plain_quantize(s):
    x = s["x"]
    if s["case"]["form"] == "weights":  # blocks along the rows: [n][in][out] -> [n][out][in]
        x = x.transpose(1, 2)
    q, e = _plain_mxfp4(x)
    return {"values": _scaled(q, e).to(x.dtype), "scales": e}


def _plain_matmul(s):
    xp = _spread(_scaled(*_plain_mxfp4(s["x"])), s)
    out = torch.bmm(xp, _plain_decode(*s["w"]).transpose(1, 2))
    if s["w_pair"] is not None:
        out = out * torch.sigmoid(out) * torch.bmm(xp, _plain_decode(*s["w_pair"]).transpose(1, 2))
    return {"out": _gather(out, s).to(_DTYPES[s["case"]["dtype"]])}


_PLAIN = {"ffn_forward": _plain_ffn_forward, "ffn_backward": _plain_ffn_backward, "quantize": _plain_quantize,
          "matmul": _plain_matmul}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own_ffn_forward(s):
    r = s["layer"].ffn_forward(s["x"], s["w1"], s["w3"], s["w2"], offsets=s["offsets"], keep=s["case"]["keep"])
    return dict(zip(("y", "gate", "up"), r)) if s["case"]["keep"] else {"y": r}


def _own_ffn_backward(s):
    r = s["layer"].ffn_backward(s["dy"], s["x"], s["gate"], s["up"], s["w1"], s["w3"], s["w2"], offsets=s["offsets"])
    return dict(zip(("dx", "dw1", "dw3", "dw2"), r))


def _own_quantize(s):
    import sparse_mixture_experts_24_b200 as m
    call = m.quantize_weights_mxfp4 if s["case"]["form"] == "weights" else m.quantize_mxfp4
    codes, scales, values = call(s["x"], values=True)
    return {"values": values, "scales": scales}


def _own_matmul(s):
    import sparse_mixture_experts_24_b200 as m
    return {"out": s["layer"].matmul_mxfp4(m.quantize_mxfp4(s["x"]), s["w"], pair=s["w_pair"], offsets=s["offsets"])}


_OWN = {"ffn_forward": _own_ffn_forward, "ffn_backward": _own_ffn_backward, "quantize": _own_quantize,
        "matmul": _own_matmul}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, expert by expert
# ---------------------------------------------------------------------------
def _powers(device):
    return torch.tensor([2.0 ** k for k in range(-127, 130)], dtype=torch.float64, device=device)


def _exact_values(v):
    """v [..., k] -> what its MXFP4 form stands for, and the scale codes, in
    64 bits: nearest of the fifteen E2M1 values to v / 2^(code - 127)."""
    b = v.double().reshape(*v.shape[:-1], -1, 32)
    powers = _powers(v.device)
    # how many of 2^-127 .. 2^129 are at most the largest magnitude gives floor(log2) + 128
    code = (torch.bucketize(b.abs().max(dim=-1).values, powers, right=True) - 128 - 2 + 127).clamp(0, 254)
    unit = powers[code].unsqueeze(-1)
    z = (b.abs() / unit).clamp(max=6.0)
    # the step between neighbours is 0.5 below 2, 1 below 4 and 2 above
    step = 0.5 + 0.5 * (z >= 2).double() + (z >= 4).double()
    z = torch.round(z / step) * step  # torch.round takes ties to even
    return (torch.copysign(z, b) * unit).reshape(v.shape), code.to(torch.uint8)


def _exact_decode(codes, scales):
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    nib = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int64, device=codes.device)
    nib[..., 0::2], nib[..., 1::2] = (codes % 16).long(), (codes // 16).long()
    v = torch.tensor(mag, dtype=torch.float64, device=codes.device)[nib % 8] * (1.0 - 2.0 * (nib // 8).double())
    return v * _powers(codes.device)[scales.long()].repeat_interleave(32, dim=-1)


def exact(case, seed):
    if 24 * case["rows"] * case.get("d", case.get("k", 0)) * case.get("ffn", case["cols"] if "cols" in case else 0) > 3e13:
        return None
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"] if case["form"] == "rows" else s["x"].transpose(1, 2).contiguous()
        values, scales = _exact_values(x)
        return {"values": values, "scales": scales}
    edges = [0, case["rows"]] if s["offsets"] is None else s["offsets"].tolist()
    parts = []
    for e in range(case["n"]):
        at = slice(edges[e], edges[e + 1])
        x = s["x"][at].double()
        if case["op"] == "matmul":
            x = _exact_values(s["x"][at])[0] if x.numel() else x
            out = x @ _exact_decode(s["w"][0][e], s["w"][1][e]).T
            if case["pair"]:
                up = x @ _exact_decode(s["w_pair"][0][e], s["w_pair"][1][e]).T
                out = out / (1 + torch.exp(-out)) * up
            parts.append({"out": out})
            continue
        w1, w3, w2 = (s[k][e].double() for k in ("w1", "w3", "w2"))
        if case["op"] == "ffn_forward":
            a, b = x @ w1, x @ w3
            part = {"y": (a / (1 + torch.exp(-a)) * b) @ w2}
            parts.append({**part, "gate": a, "up": b} if case["keep"] else part)
            continue
        a, b, dy = s["gate"][at].double(), s["up"][at].double(), s["dy"][at].double()
        p = 1 / (1 + torch.exp(-a))
        dh = dy @ w2.T
        da, db = dh * b * (p + a * p * (1 - p)), dh * a * p
        parts.append({"dx": da @ w1.T + db @ w3.T, "dw1": x.T @ da, "dw3": x.T @ db, "dw2": (a * p * b).T @ dy})
    join = {k: (torch.stack if k.startswith("dw") else torch.cat) for k in parts[0]}
    return {k: join[k]([p[k] for p in parts]) for k in parts[0]}
