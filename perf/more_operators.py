"""Workloads of the operators around a decoder's cache: per-head norms of queries and keys with rotary positions of
several axes, and a paged key-value cache held in 4 bits (append, read back, attention of one new token per sequence).

A case is a dict of plain values; its "op" is "rotate", "append4", "read4" or "decode4".  `run` computes a case with
elementary torch operations (`own` false) or with the library's calls (`own` true).

Values of a 4-bit cache: 32 consecutive dims of a token's head share a scale s, max|x| / 7 rounded to bf16; an element
is c s with c = x / s rounded to the nearest whole number (ties to even) within -7..7.  Byte i of a row holds c + 8 of
dim 2i in its low and of dim 2i + 1 in its high half.  Rows have room for an even number of scales.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32
SPREAD = 3.0  # standard deviation of the scores: trained heads favour a few keys
LARGEST_ROWS = 16384 * 40 * 128 * 2  # bytes of the largest rotate case's queries and keys
LARGEST_TOKENS = 16 * 2048 * 8 * 256 * 2  # bytes of the largest append and read cases' tokens
LARGEST_CACHE = 8 * 131072 * 8 * 256  # elements of the largest decode case's cache


def rotate(name, b, l, hq, hkv, d, rotary, axes, order, dtype="bf16", adjacent=False, norm=True, past=0):
    return {"name": name, "op": "rotate", "b": b, "l": l, "hq": hq, "hkv": hkv, "d": d, "rotary": rotary, "axes": axes,
            "order": order, "dtype": dtype, "adjacent": adjacent, "norm": norm, "past": past}


def append4(name, b, t, hkv, dk, dv, page, past, dtype="bf16", ragged=False, tokens_first=False):
    return {"name": name, "op": "append4", "b": b, "t": t, "hkv": hkv, "dk": dk, "dv": dv, "page": page, "past": past,
            "dtype": dtype, "ragged": ragged, "tokens_first": tokens_first}


def read4(name, b, t, hkv, dk, dv, page, past, dtype="bf16", ragged=False, tokens_first=False):
    return dict(append4(name, b, t, hkv, dk, dv, page, past, dtype, ragged, tokens_first), op="read4")


def decode4(name, b, lo, hi, hq, hkv, dk, dv, page, dtype="bf16", cap=0.0, bias=False, first=False, tokens_first=False):
    return {"name": name, "op": "decode4", "b": b, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "page": page, "dtype": dtype, "cap": cap, "bias": bias, "first": first, "tokens_first": tokens_first}


def listed():
    return [
        # one new token for each of 64 sequences: latency
        rotate("rotate_token_b64", 64, 1, 32, 8, 128, 128, 3, "parts", past=2000),
        # a batch of 20x20 feature maps in the framework's default type: two axes, each with its own frequencies
        rotate("rotate_map_20x20_f32", 32, 400, 8, 2, 32, 32, 2, "axial", dtype="f32", adjacent=True),
        # a long prompt of text and image tokens, three axes
        rotate("rotate_prompt_16k", 1, 16384, 32, 8, 128, 128, 3, "parts"),
        # one new token for each of 64 sequences into the cache
        append4("append4_token_b64", 64, 1, 8, 128, 128, 16, 2000),
        # a batch of prompts into the cache, ragged
        append4("append4_prompts", 16, 2048, 8, 128, 128, 64, 0, ragged=True),
        # fp32 tokens of odd counts
        append4("append4_f32_odd", 5, 77, 4, 32, 64, 20, 13, dtype="f32"),
        # a long cached prompt that further prompt tokens will attend to, as values
        read4("read4_prompt_16k", 1, 16384, 8, 128, 128, 64, 0),
        # the newest tokens of a few sequences
        read4("read4_f32_few", 3, 50, 4, 64, 64, 20, 301, dtype="f32", ragged=True),
        # one sequence right after its image prefix: latency
        decode4("decode4_one_400", 1, 421, 421, 8, 2, 64, 64, 16),
        # ordinary serving: 64 sequences of ragged lengths, capped scores
        decode4("decode4_b64_ragged", 64, 130, 4000, 32, 8, 128, 128, 64, cap=30.0),
        # fp32, as many key heads as query heads, a bias by distance and sequences that start at a later key
        decode4("decode4_f32_mha", 8, 300, 1700, 12, 12, 64, 64, 32, dtype="f32", bias=True, first=True),
        # the largest cache: a few very long sequences
        decode4("decode4_long_131072", 8, 65536, 131072, 32, 8, 128, 128, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rotate", "rotate", "append4", "read4", "decode4", "decode4", "decode4"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    es = 2 if dtype == "bf16" else 4
    hkv = rng.choice((1, 2, 3, 4, 8))
    hq = hkv * rng.choice((1, 1, 2, 4, 5, 8))
    b = _log(rng, 1, 256)
    if op == "rotate":
        d = rng.choice((32, 40, 64, 72, 96, 128, 128))
        l = _log(rng, 1, 16384)
        while b > 1 and b * l * (hq + hkv) * d * es > LARGEST_ROWS:
            b = (b + 1) // 2
        while b * l * (hq + hkv) * d * es > LARGEST_ROWS:
            l = (l + 1) // 2
        return {"op": op, "b": b, "l": l, "hq": hq, "hkv": hkv, "d": d, "rotary": rng.choice((d, d, d // 2)),
                "axes": rng.choice((1, 2, 3)), "order": rng.choice(("parts", "turns", "axial")), "dtype": dtype,
                "adjacent": rng.random() < 0.4, "norm": rng.random() < 0.75, "past": _log(rng, 1, 100000) - 1}
    dk, dv = rng.choice(((32, 64), (64, 64), (96, 96), (128, 128), (128, 128), (40, 72), (64, 128)))
    page = rng.choice((16, 20, 32, 64, 128))
    tokens_first = rng.random() < 0.3
    if op != "decode4":
        t = _log(rng, 1, 2048 if op == "append4" else 16384)
        while b > 1 and b * t * hkv * (dk + dv) * es > LARGEST_TOKENS:
            b = (b + 1) // 2
        return {"op": op, "b": b, "t": t, "hkv": hkv, "dk": dk, "dv": dv, "page": page, "past": _log(rng, 1, 4000) - 1,
                "dtype": dtype, "ragged": rng.random() < 0.4, "tokens_first": tokens_first}
    hi = _log(rng, 1, 131072)
    # fp32 has no tensor-core product of full precision: its largest caches are smaller
    most = LARGEST_CACHE // (2 if dtype == "bf16" else 8)
    while b > 1 and b * hi * hkv * (dk + dv) > most:
        b = (b + 1) // 2
    return {"op": op, "b": b, "lo": rng.randint(max(1, hi // 4), hi), "hi": hi, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "page": page, "dtype": dtype, "cap": rng.choice((0.0, 0.0, 30.0)), "bias": rng.random() < 0.35,
            "first": rng.random() < 0.3, "tokens_first": tokens_first}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _counts(c):
    return _spread(c["b"], (c["t"] + 1) // 2, c["t"]) if c["ragged"] else [c["t"]] * c["b"]


def _lens(c):
    return _spread(c["b"], c["lo"], c["hi"])


def _first(length):
    return length // 5


def _scales(dim):
    """Room for scales in a row: an even number."""
    return 2 * ((dim + 2 * GROUP - 1) // (2 * GROUP))


def _row_bytes(dim):
    return (dim + 1) // 2 + 2 * _scales(dim)


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rotate":
        tokens = c["b"] * c["l"]
        elements = tokens * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 2 * elements * es + 4 * tokens * c["axes"], "flops": 7 * elements}
    cached = _row_bytes(c["dk"]) + _row_bytes(c["dv"])
    d = c["dk"] + c["dv"]
    if c["op"] == "decode4":
        keys = sum(n - _first(n) if c["first"] else n for n in _lens(c))
        return {"bytes": keys * c["hkv"] * cached + c["b"] * c["hq"] * d * es, "flops": 2 * d * c["hq"] * keys}
    rows = sum(_counts(c)) * c["hkv"]
    if c["op"] == "read4":
        return {"bytes": rows * (cached + d * es), "flops": rows * d}
    # tokens in, codes out; then the codes as the values they stand for
    return {"bytes": rows * 2 * (cached + d * es), "flops": 8 * rows * d}


# ------------------------------------------------------------------ inputs
def _turns(c):
    """Each pair's axis and its frequency in radians per position."""
    n, a = c["rotary"] // 2, c["axes"]
    if c["order"] == "turns":  # axes take pairs in turn
        axis = [i % a for i in range(n)]
    else:  # each axis a part; the first is shorter where there are three
        edges = [n * i // a for i in range(1, a)] if a < 3 else [n // 4, n // 4 + 3 * n // 8]
        axis = [sum(i >= e for e in edges) for i in range(n)]
    freq = []
    for i in range(n):
        at, of = (i, n) if c["order"] != "axial" else (i - axis.index(axis[i]), axis.count(axis[i]))
        freq.append(10000.0 ** (-at / of))
    return axis, freq


def _positions(c, dev):
    """int32 [axes, b, l]: half the tokens are an image's (one time, rows, columns), the others are text."""
    b, l, a = c["b"], c["l"], c["axes"]
    i = torch.arange(l, device=dev)
    image = l if c["order"] == "axial" else l // 2
    width = max(1, math.isqrt(image))
    text = i - image + (image + width - 1) // width
    at = [torch.where(i < image, torch.zeros_like(i), text), torch.where(i < image, i // width, text),
          torch.where(i < image, i % width, text)][3 - a:]
    shift = c["past"] + 3 * torch.arange(b, device=dev)
    return (torch.stack(at)[:, None, :] + shift[None, :, None]).to(torch.int32).contiguous()


def _pages4(c, tokens, g, dev):
    """Pages with room for `tokens` tokens of each sequence, at random places, and the table that names them (-1: none):
    codes and scales [pages, page, heads, .] of keys and of values."""
    need = [(n + c["page"] - 1) // c["page"] for n in tokens]
    count = sum(need) + 3
    pages = []
    for dim in (c["dk"], c["dv"]):
        shape = (count, c["page"], c["hkv"]) if c["tokens_first"] else (count, c["hkv"], c["page"])
        value = torch.randn(*shape, (dim + 1) // 2, 2, generator=g, device=dev, dtype=torch.bfloat16)
        nibble = ((value * 2.6).round().clamp(-7, 7) + 8).to(torch.uint8)
        codes = nibble[..., 0] | (nibble[..., 1] << 4)
        scales = torch.rand(*shape, _scales(dim), generator=g, device=dev, dtype=torch.float32) * 0.2 + 0.2
        scales = scales.to(torch.bfloat16)
        pages += [codes, scales] if c["tokens_first"] else [codes.transpose(1, 2), scales.transpose(1, 2)]
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    width = max(need) + 1
    slot = torch.arange(width, device=dev)[None, :]
    need_t = torch.tensor(need, device=dev)[:, None]
    start = torch.cumsum(need_t, 0) - need_t
    table = torch.where(slot < need_t, order[(start + slot).clamp(max=count - 1)], torch.full_like(order[:1], -1))
    return pages, table.contiguous()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 11)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if own:
        from conv_bn_activation_gb300 import binding as cb
    if c["op"] == "rotate":
        b, l, hq, hkv, d = (c[n] for n in ("b", "l", "hq", "hkv", "d"))
        row = torch.randn(b, l, (hq + 2 * hkv) * d, generator=g, device=dev, dtype=dt)  # a projection's output
        q, k, _ = torch.split(row, [hq * d, hkv * d, hkv * d], dim=-1)
        st.update(q=q.unflatten(-1, (hq, d)), k=k.unflatten(-1, (hkv, d)), pos=_positions(c, dev))
        axis, freq = _turns(c)
        st["axis"] = torch.tensor(axis, dtype=torch.int32, device=dev)
        st["freq"] = torch.tensor(freq, dtype=torch.float32, device=dev)
        weight = 1.0 + 0.1 * torch.randn(2, d, generator=g, device=dev)
        st["q_weight"], st["k_weight"] = (weight[0], weight[1]) if c["norm"] else (None, None)
        st["q_out"], st["k_out"] = (torch.empty(b, l, h, d, device=dev, dtype=dt) for h in (hq, hkv))
        if own:
            st["rule"] = cb.Rotation(st["freq"], axis=st["axis"], axes=c["axes"], adjacent=c["adjacent"], norm=c["norm"], eps=1e-6,
                                     q_weight=st["q_weight"], k_weight=st["k_weight"])
        return st
    if c["op"] == "decode4":
        b = c["b"]
        lens = torch.tensor(_lens(c))[torch.randperm(b, generator=torch.Generator().manual_seed(int(seed)))]
        st["pages"], st["table"] = _pages4(c, lens.tolist(), g, dev)
        st["length"] = lens.to(device=dev, dtype=torch.int32)
        st["first"] = _first(lens).to(device=dev, dtype=torch.int32) if c["first"] else None
        st["slopes"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], dtype=torch.float32, device=dev)
                        if c["bias"] else None)
        st["q"] = torch.randn(b, c["hq"], c["dk"], generator=g, device=dev, dtype=dt) * (SPREAD / 0.8)
        st["out"] = torch.empty(b, c["hq"], c["dv"], device=dev, dtype=dt)
    else:
        b, t, dk, dv = (c[n] for n in ("b", "t", "dk", "dv"))
        st["pages"], st["table"] = _pages4(c, [c["past"] + t] * b, g, dev)
        new = torch.randn(b, t, c["hkv"] * (dk + dv), generator=g, device=dev, dtype=dt)
        k, v = torch.split(new, [c["hkv"] * dk, c["hkv"] * dv], dim=-1)
        st.update(k=k.unflatten(-1, (c["hkv"], dk)), v=v.unflatten(-1, (c["hkv"], dv)))
        perm = torch.randperm(b, generator=g, device=dev)
        st["pos"] = torch.full((b,), c["past"], dtype=torch.int32, device=dev)
        st["count"] = torch.tensor(_counts(c), dtype=torch.int32, device=dev)[perm].contiguous() if c["ragged"] else None
        st["k_out"], st["v_out"] = (torch.zeros(b, t, c["hkv"], d, device=dev, dtype=dt) for d in (dk, dv))
    if own:
        st["cache"] = cb.PagedCache4(*st["pages"], st["table"], dim_k=c["dk"], dim_v=c["dv"])
        if c["op"] == "decode4":
            st["workspace"] = torch.empty(cb.attention_decode4_workspace(st["q"], st["cache"]), dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------- plain forms
def _turned(x, weight, cos, sin, c):
    y = x.float()
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
    n = c["rotary"] // 2
    if c["adjacent"]:
        y1, y2 = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
        first, second = y1 * cos - y2 * sin, y2 * cos + y1 * sin
        turned = torch.stack([first, second], dim=-1).flatten(-2)
    else:
        y1, y2 = y[..., :n], y[..., n:2 * n]
        turned = torch.cat([y1 * cos - y2 * sin, y2 * cos + y1 * sin], dim=-1)
    return torch.cat([turned, y[..., 2 * n:]], dim=-1).to(x.dtype)


def _rotate(st):
    angle = st["pos"][st["axis"].long()].permute(1, 2, 0).double() * st["freq"].double()  # far positions: in 64 bits
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    return _turned(st["q"], st["q_weight"], cos, sin, st["case"]), _turned(st["k"], st["k_weight"], cos, sin, st["case"])


def _grouped(x):
    """[..., dim] as [..., groups, 32], zeros behind the last dim."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _to_codes(x):
    """Codes' bytes and scales of rows [..., dim]; in 64 bits: a step's border is as near as fp32's rounding."""
    dim = x.shape[-1]
    y = _grouped(x.double())
    bits = (y.abs().amax(-1) / 7).view(torch.int64)  # to 8 significant bits, ties to even
    bits = bits + ((1 << 44) - 1) + ((bits >> 45) & 1)
    scale = ((bits >> 45) << 45).view(torch.float64)[..., None]
    code = torch.where(scale == 0, torch.zeros_like(y), torch.round(y / scale)).clamp(-7, 7)
    nibble = (code + 8).to(torch.uint8).flatten(-2)[..., :dim + dim % 2]
    scale = scale[..., 0].to(torch.bfloat16)
    scale = torch.nn.functional.pad(scale, (0, _scales(dim) - scale.shape[-1]))
    return nibble[..., 0::2] | (nibble[..., 1::2] << 4), scale


def _to_values(codes, scales, dim):
    nibble = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)[..., :dim]
    return (nibble.float() - 8) * scales.float().repeat_interleave(GROUP, dim=-1)[..., :dim]


def _places(st):
    """Page and slot of every token of the call, and whether it is one of the sequence's."""
    c = st["case"]
    t = torch.arange(c["t"], device=st["pos"].device)[None, :].expand(c["b"], c["t"])
    real = torch.ones_like(t, dtype=torch.bool) if st["count"] is None else t < st["count"][:, None]
    at = st["pos"][:, None].long() + torch.where(real, t, torch.zeros_like(t))
    return st["table"].gather(1, at // c["page"]).long(), at % c["page"], real, torch.where(real, t, torch.zeros_like(t))


def _read4(st):
    c = st["case"]
    page, slot, real, _ = _places(st)
    out = []
    for i, (name, dim) in enumerate((("k", c["dk"]), ("v", c["dv"]))):
        values = _to_values(st["pages"][2 * i][page, slot], st["pages"][2 * i + 1][page, slot], dim)
        out.append(torch.where(real[:, :, None, None], values, torch.zeros_like(values)).to(st[name].dtype))
    return tuple(out)


def _append4(st):
    page, slot, _, t = _places(st)  # a place past a sequence's count takes its first token a second time
    row = torch.arange(st["case"]["b"], device=page.device)[:, None]
    for i, name in enumerate(("k", "v")):
        codes, scales = _to_codes(st[name][row, t])
        st["pages"][2 * i][page, slot] = codes
        st["pages"][2 * i + 1][page, slot] = scales
    return _read4(st)


def _decode4(st):
    c, dev = st["case"], st["q"].device
    group = c["hq"] // c["hkv"]
    table = st["table"].clamp(min=0).long()
    k, v = (_to_values(st["pages"][2 * i][table], st["pages"][2 * i + 1][table], c[n]).flatten(1, 2)
            for i, n in enumerate(("dk", "dv")))
    q = st["q"].float().reshape(c["b"], c["hkv"], group, c["dk"])
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * c["dk"] ** -0.5
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    j = torch.arange(s.shape[-1], device=dev)[None, :]
    if st["slopes"] is not None:
        far = (st["length"][:, None] - 1 - j).float()
        s = s - st["slopes"].reshape(1, c["hkv"], group, 1) * far[:, None, None, :]
    keep = j < st["length"][:, None]
    if st["first"] is not None:
        keep = keep & (j >= st["first"][:, None])
    s = torch.where(keep[:, None, None, :], s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.transpose(1, 2)) / torch.where(total == 0, torch.ones_like(total), total)
    return out.reshape(c["b"], c["hq"], c["dv"]).to(st["q"].dtype)


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"rotate": _rotate, "append4": _append4, "read4": _read4, "decode4": _decode4}[c["op"]](st)
    from conv_bn_activation_gb300 import binding as cb
    if c["op"] == "rotate":
        cb.norm_rotate(st["q"], st["k"], st["pos"], st["rule"], st["q_out"], st["k_out"])
        return st["q_out"], st["k_out"]
    if c["op"] == "decode4":
        return cb.attention_decode4(st["q"], st["cache"], st["length"], st["out"], st["workspace"], scale=c["dk"] ** -0.5,
                                    softcap=c["cap"], slopes=st["slopes"], first=st["first"])
    if c["op"] == "append4":
        cb.cache4_append(st["k"], st["v"], st["cache"], st["pos"], count=st["count"])
    cb.cache4_read(st["cache"], st["k_out"], st["v_out"], first=st["pos"], count=st["count"])
    return st["k_out"], st["v_out"]


# ------------------------------------------------------------------- exact
def _exact_turn(x, weight, angle, c):
    y = x.double()
    if c["norm"]:
        y = y / (y.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
    out = y.clone()
    n = c["rotary"] // 2
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if c["adjacent"] else (i, n + i)
        co, si = torch.cos(angle[i])[:, :, None], torch.sin(angle[i])[:, :, None]
        out[..., a] = co * y[..., a] - si * y[..., b]
        out[..., b] = si * y[..., a] + co * y[..., b]
    return out


def _exact_stored(x):
    """The values that rows [..., dim] are stored as."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for lo in range(0, x.shape[-1], GROUP):
        y = x[..., lo:lo + GROUP].double()
        top = y.abs().max(dim=-1, keepdim=True).values / 7.0
        wide = top * (2.0 ** 45 + 1)
        s = wide - (wide - top)  # the nearest number of 8 significant bits
        steps = torch.round(y / torch.where(s > 0, s, torch.ones_like(s)))
        out[..., lo:lo + GROUP] = s * torch.minimum(steps.abs(), torch.full_like(steps, 7)) * torch.sign(steps)
    return out


def _exact_cached(codes, scales, dim):
    """Values of cached rows [n, bytes], dim by dim."""
    out = torch.empty(*codes.shape[:-1], dim, dtype=torch.float64, device=codes.device)
    for d in range(dim):
        byte = codes[..., d // 2].to(torch.int32)
        out[..., d] = ((byte // 16 if d % 2 else byte % 16) - 8).double() * scales[..., d // GROUP].double()
    return out


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    if c["op"] == "rotate":
        angle = [st["pos"][int(a)].double() * f for a, f in zip(st["axis"].tolist(), st["freq"].double())]
        return tuple(_exact_turn(st[n], st[n + "_weight"], angle, c) for n in ("q", "k"))
    if c["op"] == "append4":
        out = [_exact_stored(st[n]) for n in ("k", "v")]
        if st["count"] is not None:
            for b in range(c["b"]):
                for x in out:
                    x[b, int(st["count"][b]):] = 0
        return tuple(out)
    group = c["hq"] // c["hkv"] if c["op"] == "decode4" else 1

    def cached(b, lo, n):
        at = torch.arange(lo, n, device=st["table"].device)
        page, slot = st["table"][b].long()[at // c["page"]], at % c["page"]
        return [_exact_cached(st["pages"][2 * i][page, slot], st["pages"][2 * i + 1][page, slot], c[d])
                for i, d in enumerate(("dk", "dv"))]

    if c["op"] == "read4":
        out = [torch.zeros(c["b"], c["t"], c["hkv"], c[d], dtype=torch.float64, device=st["table"].device) for d in ("dk", "dv")]
        for b in range(c["b"]):
            n = c["t"] if st["count"] is None else int(st["count"][b])
            for x, y in zip(out, cached(b, c["past"], c["past"] + n)):
                x[b, :n] = y
        return tuple(out)
    out = torch.zeros(c["b"], c["hq"], c["dv"], dtype=torch.float64, device=st["q"].device)
    for b in range(c["b"]):
        n = int(st["length"][b])
        lo = int(st["first"][b]) if st["first"] is not None else 0
        k, v = cached(b, lo, n)
        far = (n - 1 - torch.arange(lo, n, device=k.device)).double()
        for h in range(c["hq"]):
            s = k[:, h // group] @ st["q"][b, h].double() / math.sqrt(c["dk"])
            if c["cap"]:
                s = torch.tanh(s / c["cap"]) * c["cap"]
            if st["slopes"] is not None:
                s = s - st["slopes"][h].double() * far
            out[b, h] = torch.softmax(s, dim=0) @ v[:, h // group]
    return out
