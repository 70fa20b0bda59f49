"""Cases of the block-scaled FP8 operators: quantization with a scale for each
block of 128, the gated activation and the RMSNorm that write such codes, and
the matrix product that reads them.

A quantized matrix of ``rows`` x ``cols`` is a pair (q, s): E4M3 codes
[rows, cols] whose rows start on multiples of 16 bytes, and fp32 scales with
one row for each block of 128 columns, s[c // 128, r] (a scale for each row) or
s[c // 128, r // 128] (one for each 128 x 128 block); an element stands for
q * s.  With amax the largest magnitude of a block, r = 448 / amax and
s = amax / 448 in fp32, and q is the E4M3 value nearest to x * r, ties to even.
A matrix of zeros has s = 1.
"""

import math

import torch

own = False

GROUP = 128          # elements that share a scale
TOP = 448.0          # the largest E4M3 value
FLOOR = 2.0 ** -100  # a smaller largest magnitude counts as this one
EPS = 1e-5


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the layer's second MLP weight after an optimizer step: codes for the
        # forward product and, transposed, for the input gradient's
        dict(name="quantize weight 8192x28672", op="quantize", rows=8192,
             cols=28672, group="block", out="both"),
        # an output gradient of a short ragged batch: rows for the input
        # gradient's product, columns for the weight gradient's
        dict(name="quantize gradient 777x1000", op="quantize", rows=777,
             cols=1000, group="row", out="both"),
        # the SwiGLU MLP's activation in a training step
        dict(name="swiglu 8192x11008", op="swiglu", rows=8192, f=11008,
             out="both"),
        # the same of the wide layer for one token that is being generated
        dict(name="swiglu 1x28672", op="swiglu", rows=1, f=28672, out="row"),
        # its backward in a training step
        dict(name="swiglu backward 8192x11008", op="swiglu_bwd", rows=8192,
             f=11008, out="both"),
        # residual and norm in front of a block, one token
        dict(name="norm 1x8192", op="norm", rows=1, h=8192, y=False),
        # the same for a training batch, which keeps the norm's output too
        dict(name="norm 8192x8192", op="norm", rows=8192, h=8192, y=True),
        # a ragged prompt at an odd width
        dict(name="norm 1001x4100", op="norm", rows=1001, h=4100, y=False),
        # one token through a square projection: latency
        dict(name="product 1x4096x4096", op="gemm", m=1, n=4096, k=4096,
             groups="forward", out="bf16"),
        # a batch of generated tokens through the layer's second MLP weight
        dict(name="product 48x8192x28672", op="gemm", m=48, n=8192, k=28672,
             groups="forward", out="bf16"),
        # the same weight in training
        dict(name="product 8192x8192x28672", op="gemm", m=8192, n=8192,
             k=28672, groups="forward", out="bf16"),
        # a weight gradient: both operands with a scale for each row, and a
        # ragged number of tokens to sum over
        dict(name="weight gradient 11008x4096x4100", op="gemm", m=11008,
             n=4096, k=4100, groups="gradient", out="f32"),
    ]


def _size(rng, lo, hi):
    """A size of [lo, hi], even over its logarithm; one in three is a multiple
    of 128 or of 16, where it is large enough."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 1, 1, 1, 16, 128))
    if v > 2 * step:
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("quantize", "swiglu", "swiglu_bwd", "norm", "gemm",
                     "gemm"))
    if op == "quantize":
        return dict(op=op, rows=_size(rng, 1, 8192), cols=_size(rng, 8, 28672),
                    group=rng.choice(("row", "block")),
                    out=rng.choice(("row", "both")))
    if op in ("swiglu", "swiglu_bwd"):
        return dict(op=op, rows=_size(rng, 1, 8192), f=_size(rng, 8, 11008),
                    out=rng.choice(("row", "both")))
    if op == "norm":
        return dict(op=op, rows=_size(rng, 1, 8192), h=_size(rng, 8, 8192),
                    y=rng.random() < 0.5)
    groups = rng.choice(("forward", "forward", "gradient"))
    while True:
        m, n, k = _size(rng, 1, 11008), _size(rng, 16, 28672), _size(rng, 16,
                                                                     28672)
        if m * n * k <= 8192 * 8192 * 28672 // 4 and m * n <= 1 << 28 and \
                n * k <= 1 << 28 and m * k <= 1 << 28:
            return dict(op=op, m=m, n=n, k=k, groups=groups,
                        out=rng.choice(("bf16", "f32")))


# ------------------------------------------------------------------ inputs --
def _blocks(n):
    return (n + GROUP - 1) // GROUP


def _codes(rows, cols):
    """Room for codes [rows, cols] with rows on multiples of 16 bytes."""
    return torch.empty((rows, (cols + 15) // 16 * 16),
                       dtype=torch.float8_e4m3fn, device="cuda")[:, :cols]


def _scales(rows, cols, group):
    return torch.empty((_blocks(cols), rows if group == "row" else
                        _blocks(rows)), dtype=torch.float32, device="cuda")


def _room(rows, cols, group, out):
    """q, s and, for out "both", qt, st of the transposed matrix."""
    r = dict(q=_codes(rows, cols), s=_scales(rows, cols, group))
    if out == "both":
        r.update(qt=_codes(cols, rows), st=_scales(cols, rows, group))
    return r


def _normal(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std)


def _activation(gen, rows, cols):
    """Normal values whose tokens differ in scale, a few channels far out."""
    x = _normal(gen, rows, cols)
    x *= torch.exp(0.5 * _normal(gen, rows, 1))
    x *= 1.0 + 15.0 * (torch.rand((1, cols), generator=gen, device="cuda") <
                       0.004)
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = dict(case=case)
    op, bf16 = case["op"], torch.bfloat16
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        x = _normal(gen, rows, cols, std=0.02) if case["group"] == "block" \
            else _activation(gen, rows, cols).mul_(1e-3)
        st.update(x=x.to(bf16), **_room(rows, cols, case["group"],
                                        case["out"]))
    elif op in ("swiglu", "swiglu_bwd"):
        rows, f = case["rows"], case["f"]
        st["gu"] = _activation(gen, rows, 2 * f).to(bf16)
        if op == "swiglu":
            st.update(_room(rows, f, "row", case["out"]))
        else:
            st["da"] = _normal(gen, rows, f, std=1e-3).to(bf16)
            st.update(_room(rows, 2 * f, "row", case["out"]))
    elif op == "norm":
        rows, h = case["rows"], case["h"]
        st.update(x=_activation(gen, rows, h).to(bf16),
                  r=_normal(gen, rows, h, std=0.5).to(bf16),
                  gamma=(1.0 + _normal(gen, h, std=0.02)).to(bf16),
                  x1=torch.empty((rows, h), dtype=bf16, device="cuda"),
                  rstd=torch.empty(rows, dtype=torch.float32, device="cuda"),
                  **_room(rows, h, "row", "row"))
        st["y"] = torch.empty_like(st["x1"]) if case["y"] else None
    else:
        m, n, k = case["m"], case["n"], case["k"]
        fwd = case["groups"] == "forward"
        a = _activation(gen, m, k).to(bf16)
        b = (_normal(gen, n, k, std=0.02) if fwd
             else _activation(gen, n, k)).to(bf16)
        st["qa"], st["qb"] = _codes(m, k), _codes(n, k)
        q, st["sa"] = _quantize(a.float(), "row")
        st["qa"].copy_(q)
        q, st["sb"] = _quantize(b.float(), "block" if fwd else "row")
        st["qb"].copy_(q)
        st["c"] = torch.empty((m, n), device="cuda", dtype=bf16
                              if case["out"] == "bf16" else torch.float32)
    return st


# --------------------------------------------------------------- plain form --
def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0,
                                       rows - x.shape[0]))


def _quantize(x, group):
    """(q, s) of the fp32 matrix x."""
    rows, cols = x.shape
    kb = _blocks(cols)
    if group == "row":
        v = _pad(x, rows, kb * GROUP).view(rows, kb, GROUP)
        amax = v.abs().amax(dim=2)                      # [rows, kb]
    else:
        rb = _blocks(rows)
        v = _pad(x, rb * GROUP, kb * GROUP).view(rb, GROUP, kb, GROUP)
        amax = v.abs().amax(dim=(1, 3))                 # [rb, kb]
    a = amax.clamp(min=FLOOR)
    r = torch.full_like(a, TOP) / a
    s = torch.where(amax == 0, torch.ones_like(a), a / TOP)
    v = v * (r[:, :, None] if group == "row" else r[:, None, :, None])
    q = v.reshape(-1, kb * GROUP)[:rows, :cols].to(torch.float8_e4m3fn)
    return q, s.t().contiguous()


def _dequantize(q, s):
    """The fp32 values that codes and scales stand for."""
    rows, cols = q.shape
    e = s.t()                                           # [rows or rb, kb]
    if s.shape[1] != rows:
        e = e.repeat_interleave(GROUP, 0)[:rows]
    return q.float() * e.repeat_interleave(GROUP, 1)[:, :cols]


def _outputs(v, group, both):
    q, s = _quantize(v, group)
    out = dict(q=q, s=s)
    if both:
        out["qt"], out["st"] = _quantize(v.t(), group)
    return out


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        c = _dequantize(st["qa"], st["sa"]) @ _dequantize(st["qb"],
                                                          st["sb"]).t()
        return dict(c=c.to(st["c"].dtype))
    if op == "norm":
        x1 = (st["x"].float() + st["r"].float()).to(torch.bfloat16)
        v = x1.float()
        rstd = 1.0 / torch.sqrt((v * v).mean(dim=1) + EPS)
        y = v * rstd[:, None] * st["gamma"].float()
        out = dict(x1=x1, rstd=rstd, **_outputs(y, "row", False))
        if case["y"]:
            out["y"] = y.to(torch.bfloat16)
        return out
    both = case["out"] == "both"
    if op == "quantize":
        return _outputs(st["x"].float(), case["group"], both)
    f = case["f"]
    g, u = st["gu"][:, :f].float(), st["gu"][:, f:].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    if op == "swiglu":
        return _outputs(g * sig * u, "row", both)
    da = st["da"].float()
    v = torch.cat((da * u * sig * (1.0 + g * (1.0 - sig)), da * g * sig), 1)
    return _outputs(v, "row", both)


def run(st):
    if not own:
        return _plain(st)
    from megatron_tensor_transformer_gate_gb300 import binding as tp
    op = st["case"]["op"]
    if op == "gemm":
        tp.gemm_fp8_block(st["qa"], st["sa"], st["qb"], st["sb"], st["c"])
        return dict(c=st["c"])
    if op == "norm":
        tp.add_rmsnorm_fp8_fwd(st["x"], st["r"], st["gamma"], st["x1"],
                               st["q"], st["s"], st["rstd"], y=st["y"],
                               eps=EPS)
        names = ("x1", "rstd", "q", "s", "y")
    else:
        t = dict(qt=st.get("qt"), st=st.get("st"))
        if op == "quantize":
            tp.quantize_fp8_block(st["x"], st["q"], st["s"], **t)
        elif op == "swiglu":
            tp.swiglu_fp8_fwd(st["gu"], st["q"], st["s"], **t)
        else:
            tp.swiglu_fp8_bwd(st["da"], st["gu"], st["q"], st["s"], **t)
        names = ("q", "s", "qt", "st")
    return {k: st[k] for k in names if st.get(k) is not None}


# -------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        sb = _blocks(n) if case["groups"] == "forward" else n
        return dict(bytes=m * k + n * k + 4 * _blocks(k) * (m + sb) +
                    (2 if case["out"] == "bf16" else 4) * m * n,
                    flops=2 * m * n * k)
    rows = case["rows"]
    if op == "norm":
        h = case["h"]
        return dict(bytes=rows * h * (7 + 2 * case["y"]) + 2 * h +
                    4 * rows * (1 + _blocks(h)), flops=8 * rows * h)
    cols = case["cols"] if op == "quantize" else case["f"]
    read = {"quantize": 2, "swiglu": 4, "swiglu_bwd": 6}[op] * rows * cols
    cols *= 2 if op == "swiglu_bwd" else 1
    both = case["out"] == "both"
    row = case.get("group", "row") == "row"
    scales = _blocks(cols) * (rows if row else _blocks(rows))
    if both:
        scales += _blocks(rows) * (cols if row else _blocks(cols))
    return dict(bytes=read + rows * cols * (2 if both else 1) + 4 * scales,
                flops=(4 + 6 * (op != "quantize")) * rows * cols)


# ------------------------------------------------------------------- exact --
def _e4m3(v):
    """The E4M3 value nearest to each value of v, ties to even, in 64 bits."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30)))
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_quantized(v, group):
    """Codes' values and scales of the fp64 matrix v, block column by block
    column."""
    rows, cols = v.shape
    q, s = torch.empty_like(v), []
    for c in range(0, cols, GROUP):
        part = v[:, c:c + GROUP]
        amax = part.abs().amax(dim=1)
        if group == "block":
            amax = torch.stack([b.amax() for b in amax.split(GROUP)])
        scale = torch.where(amax > 0, amax / TOP, torch.ones_like(amax))
        s.append(scale)
        if group == "block":
            scale = scale.repeat_interleave(GROUP)[:rows]
        q[:, c:c + GROUP] = _e4m3(part / scale[:, None])
    return q, torch.stack(s)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        c = torch.zeros((m, n), dtype=torch.float64, device="cuda")
        for b in range(_blocks(k)):
            at = slice(b * GROUP, (b + 1) * GROUP)
            sa, sb = st["sa"][b].double(), st["sb"][b].double()
            if case["groups"] == "forward":
                sb = sb.repeat_interleave(GROUP)[:n]
            c += (st["qa"][:, at].double() * sa[:, None]) @ (
                st["qb"][:, at].double() * sb[:, None]).t()
        return dict(c=c)
    if op == "norm":
        x1 = st["x"].double() + st["r"].double()
        v = x1.to(torch.bfloat16).double()
        rstd = (v.square().sum(dim=1) / case["h"] + EPS).rsqrt()
        y = v * rstd[:, None] * st["gamma"].double()
        q, s = _exact_quantized(y, "row")
        out = dict(x1=x1, rstd=rstd, q=q, s=s)
        if case["y"]:
            out["y"] = y
        return out
    if op == "quantize":
        v = st["x"].double()
    else:
        g, u = st["gu"].double().split(case["f"], dim=1)
        sig = torch.sigmoid(g)
        if op == "swiglu":
            v = g * sig * u
        else:
            da = st["da"].double()
            v = torch.cat((da * u * (sig + g * sig * (1.0 - sig)),
                           da * (g * sig)), 1)
    group = case.get("group", "row")
    q, s = _exact_quantized(v, group)
    out = dict(q=q, s=s)
    if case["out"] == "both":
        out["qt"], out["st"] = _exact_quantized(v.t().contiguous(), group)
    return out
