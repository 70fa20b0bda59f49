"""Cases of the paged key-value cache and its attention: keys and values of new
tokens written into the cache's pages (as they are, or quantized), whole
sequences read back out of it, and the attention of a sequence's newest tokens
over what it has cached.

A cache is two pools of pages, k and v [pages, page, n_kv, d], in bf16, fp16 or
E4M3 (then with fp32 scales ks and vs [pages, page, n_kv]: a head's vector of a
token stands for code * scale, scale = amax / 448).  Row i of ``table`` lists
the pages of sequence i in order and ``lens[i]`` says how many tokens it has,
the new ones among them: its new tokens are the last ones of these.  With
``start`` their rows are start[i] to start[i + 1] of the tensors with a row a
token, without it every sequence has the same number.  Rows that would lie in
front of a sequence (an idle one has no tokens) and behind the last one's are
neither read nor written.
"""

import math

import torch

own = False

TOP = 448.0          # the largest E4M3 value
FLOOR = 2.0 ** -100  # a smaller largest magnitude counts as this one
TYPES = dict(bf16=torch.bfloat16, f16=torch.float16, e4m3=torch.float8_e4m3fn)


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # a short chat, one token at a time: latency
        dict(name="attend 1x777 bf16", op="attend", b=1, longest=777,
             shortest=777, idle=0, new=1, n_q=32, n_kv=8, d=128, page=16,
             q="bf16", cache="bf16"),
        # a whole book in front of one user
        dict(name="attend 1x131072 bf16", op="attend", b=1, longest=131072,
             shortest=131072, idle=0, new=1, n_q=64, n_kv=8, d=128, page=64,
             q="bf16", cache="bf16"),
        # a server's batch of very different ages, some of its places empty
        dict(name="attend 64x8192 e4m3", op="attend", b=64, longest=8192,
             shortest=61, idle=9, new=1, n_q=64, n_kv=8, d=128, page=64,
             q="bf16", cache="e4m3"),
        # one rank's heads of a layer on eight, many short sequences
        dict(name="attend 256x1000 f16", op="attend", b=256, longest=1000,
             shortest=120, idle=0, new=1, n_q=8, n_kv=1, d=128, page=100,
             q="f16", cache="f16"),
        # four tokens at once (three of them drafted) over long documents
        dict(name="attend 16x65536 e4m3, 4 new", op="attend", b=16,
             longest=65536, shortest=30000, idle=0, new=4, n_q=64, n_kv=8,
             d=128, page=128, q="bf16", cache="e4m3"),
        # heads of 64, each with its own keys, an fp16 cache
        dict(name="attend 31x2047 f16, heads of 64", op="attend", b=31,
             longest=2047, shortest=300, idle=0, new=1, n_q=16, n_kv=16,
             d=64, page=32, q="bf16", cache="f16"),
        # the one new token of one user
        dict(name="write 1 token bf16", op="write", b=1, longest=778,
             shortest=778, idle=0, new=1, n_q=32, n_kv=8, d=128, page=16,
             src="bf16", cache="bf16"),
        # the new tokens of a server's batch, quantized
        dict(name="write 256 tokens e4m3", op="write", b=256, longest=4000,
             shortest=1, idle=9, new=1, n_q=64, n_kv=8, d=128, page=64,
             src="bf16", cache="e4m3"),
        # prompts of a batch after the layer's forward, whose keys are fp16
        dict(name="write prompts 24x8192 e4m3", op="write", b=24,
             longest=8192, shortest=801, idle=0, new=0, n_q=0, n_kv=8, d=128,
             page=64, src="f16", cache="e4m3"),
        # a cached prefix read back in front of a prompt's forward
        dict(name="read 1x1500 bf16", op="read", b=1, longest=1500,
             shortest=1500, idle=0, new=0, n_kv=8, d=128, page=16,
             out="bf16", cache="bf16"),
        # the same of a ragged batch out of a quantized cache
        dict(name="read 24x8192 e4m3", op="read", b=24, longest=8192,
             shortest=801, idle=5, new=0, n_kv=8, d=128, page=64, out="f16",
             cache="e4m3"),
    ]


def _size(rng, lo, hi):
    """A size of [lo, hi], even over its logarithm; one in three is a multiple
    of 16 or of 128, where it is large enough."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice((1, 1, 1, 1, 16, 128))
    if v > 2 * step:
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("attend", "attend", "write", "read"))
    most = 1 << 30 if op == "attend" else 1 << 27
    while True:
        b, longest = _size(rng, 1, 256), _size(rng, 1, 131072)
        n_kv, d = rng.choice((1, 2, 3, 4, 8, 16)), rng.choice((64, 128, 128))
        group = rng.choice((1, 2, 4, 5, 8))
        if b * longest * n_kv * d <= most:
            break
    case = dict(op=op, b=b, longest=longest,
                shortest=_size(rng, 1, longest), idle=rng.choice((0, 0, 3, 7)),
                n_kv=n_kv, d=d, page=rng.choice((1, 8, 16, 24, 64, 100, 256)),
                cache=rng.choice(("bf16", "f16", "e4m3", "e4m3")))
    if op == "attend":
        case.update(n_q=n_kv * group, new=rng.choice((1, 1, 1, 2, 3, 4)),
                    q="bf16" if case["cache"] == "bf16"
                    else rng.choice(("bf16", "f16")))
    else:
        # a step's tokens of each sequence, or (0) all that it has
        case["new"] = rng.choice((0, 0, 1, 5))
        if op == "write":
            case.update(n_q=n_kv * group, src=rng.choice(("bf16", "f16")))
        else:
            case["out"] = rng.choice(("bf16", "f16"))
    return case


def _lens(case):
    """How many tokens each sequence has: the longest first, the others spread
    evenly over the logarithm; every idle-th has none."""
    lo, hi = case["shortest"], case["longest"]
    lens = []
    for i in range(case["b"]):
        at = (i * 0.6180339887498949) % 1.0
        lens.append(int(round(hi * (lo / hi) ** at)))
        if case["idle"] and i % case["idle"] == case["idle"] - 1:
            lens[-1] = 0
    return lens


def _starts(case):
    """First rows of the sequences' new tokens, and the end."""
    starts = [0]
    for n in _lens(case):
        starts.append(starts[-1] + (case["new"] or n))
    return starts


# ------------------------------------------------------------------ inputs --
def _normal(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(std)


def _channels(gen, n_kv, d):
    """Keys' channels: a few of them far larger than the others."""
    far = torch.rand((n_kv, d), generator=gen, device="cuda") < 0.03
    return 0.8 + 3.0 * far


def _pages(case):
    return [(n + case["page"] - 1) // case["page"] for n in _lens(case)]


def _pool(case, values=None):
    """A pool [pages, page, n_kv, d], memory in the order of pages, heads,
    tokens; its last page, which no sequence has, is for the plain form alone
    and is not part of the cache."""
    n, page, n_kv, d = sum(_pages(case)) + 2, case["page"], case["n_kv"], \
        case["d"]
    whole = torch.zeros((n, n_kv, page, d), device="cuda",
                        dtype=TYPES[case["cache"]])
    scales = None
    if case["cache"] == "e4m3":
        scales = torch.ones((n, n_kv, page), device="cuda")
    if values is not None:
        for i in range(0, n, 1024):
            x = values(min(n, i + 1024) - i, n_kv, page, d)
            if scales is None:
                whole[i:i + 1024] = x.to(whole.dtype)
            else:
                whole[i:i + 1024], scales[i:i + 1024] = _quantize(x)
    return whole.permute(0, 2, 1, 3), \
        scales if scales is None else scales.permute(0, 2, 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    lens, need, op = _lens(case), _pages(case), case["op"]
    b, n_kv, d = case["b"], case["n_kv"], case["d"]
    st = dict(case=case, lens=torch.tensor(lens, dtype=torch.int32,
                                           device="cuda"))
    # pages are handed out in any order; unused places of the table hold -1
    order = torch.randperm(sum(need), generator=gen, device="cuda") + 1
    table = torch.full((b, max(max(need), 1)), -1, dtype=torch.int32)
    at, order = 0, order.to(torch.int32).cpu()
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    st["table"] = table.to("cuda")
    starts = _starts(case)
    st["start"] = None
    if op != "attend" and not case["new"]:
        st["start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    T = starts[-1]
    if op == "write":
        # rows of the projection's output: queries, keys, values
        rows = T + (5 if st["start"] is not None else 0)
        width = case["n_q"] + 2 * n_kv
        x = _normal(gen, rows, width, d)
        x[:, case["n_q"]:case["n_q"] + n_kv] *= _channels(gen, n_kv, d)
        x = x.to(TYPES[case["src"]])
        st["k"], st["v"] = x[:, case["n_q"]:].split(n_kv, dim=1)
        st["kc"], st["ks"] = _pool(case)
        st["vc"], st["vs"] = _pool(case)
        return st
    wide = _channels(gen, n_kv, d)[:, None]
    st["kc"], st["ks"] = _pool(case, lambda *s: _normal(gen, *s) * wide)
    st["vc"], st["vs"] = _pool(
        case, lambda *s: _normal(gen, *s) *
        torch.exp(0.5 * _normal(gen, *s[:3], 1)))
    if op == "attend":
        q = TYPES[case["q"]]
        st["q"] = _normal(gen, T, case["n_q"], d, std=1.5).to(q)
        st["out"] = torch.empty((T, case["n_q"], d), dtype=q, device="cuda")
        st["lse"] = torch.empty((T, case["n_q"]), device="cuda")
    else:
        rows = T + (5 if st["start"] is not None else 0)
        for name in "kv":
            st[name] = torch.zeros((rows, n_kv, d), dtype=TYPES[case["out"]],
                                   device="cuda")
    return st


# --------------------------------------------------------------- plain form --
def _quantize(x):
    """(codes, scales) of fp32 vectors [..., d]."""
    amax = x.abs().amax(dim=-1)
    a = amax.clamp(min=FLOOR)
    s = torch.where(amax == 0, torch.ones_like(a), a / TOP)
    r = torch.full_like(a, TOP) / a
    return (x * r[..., None]).to(torch.float8_e4m3fn), s


def _gather(pool, scales, page, offset):
    """The fp32 vectors of the pool at these pages and offsets."""
    if scales is None:
        return pool[page, offset].float()
    codes = pool.view(torch.uint8)[page, offset].view(pool.dtype)
    return codes.float() * scales[page, offset][..., None]


def _rows(st):
    """Of each row of the tensors with a row a token: whether it is a token of
    a sequence, the page and the offset where the cache has it."""
    case, lens = st["case"], st["lens"].long()
    row = torch.arange(st["k"].shape[0], device="cuda")
    if st["start"] is None:
        seq = row // case["new"]
        end = (seq + 1) * case["new"]
        inside = row >= 0
    else:
        start = st["start"].long()
        seq = torch.searchsorted(start, row, right=True) - 1
        inside = seq < case["b"]
        seq = seq.clamp(max=case["b"] - 1)
        end = start[seq + 1]
    pos = lens[seq] - (end - row)
    there = inside & (pos >= 0)
    pos = torch.where(there, pos, torch.zeros_like(pos))
    page = st["table"][seq, pos // case["page"]].long()
    return there, page, pos % case["page"]


def _plain_write(st):
    there, page, offset = _rows(st)
    # what is no token goes to the page behind the cache's
    page = torch.where(there, page, torch.full_like(page, -1))
    for x, pool, scales in ((st["k"], st["kc"], st["ks"]),
                            (st["v"], st["vc"], st["vs"])):
        if scales is None:
            pool[page, offset] = x.to(pool.dtype)
        else:
            codes, s = _quantize(x.float())
            pool.view(torch.uint8)[page, offset] = codes.view(torch.uint8)
            scales[page, offset] = s


def _plain_read(st):
    there, page, offset = _rows(st)
    page = page.clamp(min=0)
    for out, pool, scales in ((st["k"], st["kc"], st["ks"]),
                              (st["v"], st["vc"], st["vs"])):
        x = _gather(pool, scales, page, offset).to(out.dtype)
        out.copy_(torch.where(there[:, None, None], x, out))


def _plain_attend(st):
    case = st["case"]
    b, m, n_kv, d = case["b"], case["new"], case["n_kv"], case["d"]
    group = case["n_q"] // n_kv
    pos = torch.arange(case["longest"], device="cuda")
    page = st["table"][:, pos // case["page"]].long().clamp(min=0)
    offset = (pos % case["page"]).expand_as(page)
    q = st["q"].float().view(b, m, n_kv, group, d).transpose(1, 2)
    q = q.reshape(b, n_kv, m * group, d)
    keys = _gather(st["kc"], st["ks"], page, offset).permute(0, 2, 3, 1)
    scores = (q @ keys) / math.sqrt(d)              # [b, n_kv, m·group, len]
    del keys
    # the i-th of m new tokens sees the sequence up to itself
    seen = st["lens"].long()[:, None] - m + 1 + torch.arange(m, device="cuda")
    seen = (pos < seen[..., None]).repeat_interleave(group, 1)[:, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(dim=-1, keepdim=True)
    values = _gather(st["vc"], st["vs"], page, offset).transpose(1, 2)
    out = (p @ values) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + torch.log(total)                    # -inf of an empty row

    def rows(x):
        x = x.view(b, n_kv, m, group, -1).transpose(1, 2)
        return x.reshape(b * m, n_kv * group, -1)

    return dict(out=rows(out).to(st["out"].dtype), lse=rows(lse)[..., 0])


def run(st):
    op = st["case"]["op"]
    kc, vc, ks, vs = st["kc"][:-1], st["vc"][:-1], st["ks"], st["vs"]
    if ks is not None:
        ks, vs = ks[:-1], vs[:-1]
    if not own:
        if op == "attend":
            return _plain_attend(st)
        if op == "read":
            _plain_read(st)
        else:
            _plain_write(st)
    else:
        from megatron_tensor_transformer_gate_gb300 import binding as tp
        cache, table, lens = (kc, vc, ks, vs), st["table"], st["lens"]
        if op == "attend":
            tp.attn_decode(st["q"], cache, table, lens, st["out"],
                           lse=st["lse"])
            return dict(out=st["out"], lse=st["lse"])
        if op == "read":
            tp.kv_cache_read(cache, table, lens, st["k"], st["v"],
                             start=st["start"])
        else:
            tp.kv_cache_write(st["k"], st["v"], cache, table, lens,
                              start=st["start"])
    if op == "read":
        return dict(k=st["k"], v=st["v"])
    out = dict(kc=kc, vc=vc)
    if ks is not None:
        out.update(ks=ks, vs=vs)
    return out


# -------------------------------------------------------------------- work --
def work(case):
    lens, m, b = _lens(case), case["new"], case["b"]
    n_kv, d = case["n_kv"], case["d"]
    size = d + 4 if case["cache"] == "e4m3" else 2 * d
    lists = 4 * (sum(_pages(case)) + b)
    if case["op"] == "attend":
        n_q = case["n_q"]
        seen = sum(max(0, n - i) for n in lens for i in range(m))
        return dict(bytes=2 * n_kv * size * sum(lens) + lists +
                    b * m * n_q * (4 * d + 4), flops=4 * d * n_q * seen)
    tokens = sum(min(n, m) if m else n for n in lens)
    if m:
        lists = 4 * b + 4 * sum((min(n, m) + case["page"] - 1) //
                                case["page"] for n in lens)
    return dict(bytes=2 * n_kv * (size + 2 * d) * tokens + lists,
                flops=(6 if case["cache"] == "e4m3" else 2) * n_kv * d *
                tokens)


# ------------------------------------------------------------------- exact --
def _places(st, i):
    """Pages and offsets of sequence i's tokens."""
    n, page = int(st["lens"][i]), st["case"]["page"]
    t = torch.arange(n, device="cuda")
    return st["table"][i].long()[torch.div(t, page, rounding_mode="floor")], \
        torch.remainder(t, page)


def _cached(st, i, name):
    """Sequence i's vectors in 64 bits, [len, n_kv, d]."""
    at = _places(st, i)
    x = st[name + "c"][at].double()
    return x if st[name + "s"] is None else \
        x * st[name + "s"][at].double()[:, :, None]


def _e4m3(v):
    """The E4M3 value nearest to each value of v, ties to even, in 64 bits."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30)))
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def exact(case, seed):
    st = prepare(case, seed)
    lens, starts, m = _lens(case), _starts(case), case["new"]
    if case["op"] == "attend":
        group = case["n_q"] // case["n_kv"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64,
                         device="cuda")
        for i, n in enumerate(lens):
            if n == 0:
                continue
            k, v = _cached(st, i, "k"), _cached(st, i, "v")
            first = max(0, m - n)       # rows in front of the sequence
            q = st["q"][i * m + first:(i + 1) * m].double()
            t = torch.arange(n, device="cuda")
            last = torch.arange(n - m + first, n, device="cuda")
            for h in range(case["n_kv"]):
                heads = slice(h * group, (h + 1) * group)
                s = torch.einsum("rgd,td->rgt", q[:, heads], k[:, h])
                s /= case["d"] ** 0.5
                s[(t > last[:, None])[:, None].expand_as(s)] = -math.inf
                rows = slice(i * m + first, (i + 1) * m)
                lse[rows, heads] = torch.logsumexp(s, 2)
                out[rows, heads] = torch.softmax(s, 2) @ v[:, h]
        return dict(out=out, lse=lse)
    if case["op"] == "read":
        out = {x: st[x].double() for x in "kv"}
        for i, n in enumerate(lens):
            c = min(n, m) if m else n
            for x in "kv":
                if c:
                    out[x][starts[i + 1] - c:starts[i + 1]] = \
                        _cached(st, i, x)[n - c:]
        return out
    out = {x: st[x][:-1].double() for x in ("kc", "vc", "ks", "vs")
           if st[x] is not None}
    for i, n in enumerate(lens):
        c = min(n, m) if m else n
        if c == 0:
            continue
        at = tuple(x[n - c:] for x in _places(st, i))
        for x in "kv":
            new = st[x][starts[i + 1] - c:starts[i + 1]].double()
            if st[x + "s"] is not None:
                amax = new.abs().amax(dim=2)
                scale = torch.where(amax > 0, amax / TOP,
                                    torch.ones_like(amax))
                out[x + "s"][at] = scale
                new = _e4m3(new / scale[:, :, None])
            out[x + "c"][at] = new
    return out
