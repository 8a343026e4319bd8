"""Workloads of the attention operators: attention over whole sequences, the paged key-value cache's append, and
attention of one new token per sequence over that cache.

A case is a dict of plain values; its "op" is "attention", "append" or "decode".  `run` computes a case with elementary
torch operations in fp32 (`own` false) or with the library's calls (`own` true).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SPREAD = 3.0  # standard deviation of the scores: trained heads favour a few keys
LARGEST_PAIRS = 16 * 16384 * 16384  # query heads x queries x keys of the largest attention case
LARGEST_CACHE = 8 * 131072 * 8 * 256 * 2  # bytes of the largest decode case's cache
LARGEST_APPEND = 16 * 2048 * 8 * 256 * 2  # bytes of the largest append case's tokens


def attention(name, b, lq, lk, hq, hkv, dk, dv, dtype="bf16", causal=False, prefix=0, offset=0, docs=0, cap=0.0, bias=False,
              padded=False):
    return {"name": name, "op": "attention", "b": b, "lq": lq, "lk": lk, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "dtype": dtype, "causal": causal, "prefix": prefix, "offset": offset, "docs": docs, "cap": cap, "bias": bias,
            "padded": padded}


def append(name, b, t, hkv, dk, dv, page, past, dtype="bf16", ragged=False):
    return {"name": name, "op": "append", "b": b, "t": t, "hkv": hkv, "dk": dk, "dv": dv, "page": page, "past": past,
            "dtype": dtype, "ragged": ragged}


def decode(name, b, lo, hi, hq, hkv, dk, dv, page, dtype="bf16", cap=0.0, bias=False, first=False):
    return {"name": name, "op": "decode", "b": b, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "page": page, "dtype": dtype, "cap": cap, "bias": bias, "first": first}


def listed():
    return [
        # attention block on the 20x20 feature map of a 640x640 detector, batch 32: keys half as wide as values
        attention("map_20x20_b32", 32, 400, 400, 4, 4, 32, 64),
        # the 7x7 map of the small classifier in the framework's default type
        attention("map_7x7_f32", 8, 49, 49, 3, 3, 64, 64, dtype="f32"),
        # feature maps of images of different sizes packed into one row of tokens, each image a document, a padded end
        attention("packed_images", 2, 6400, 6400, 8, 8, 64, 64, docs=11),
        # prompts of a decoder that reads 400 image tokens as a prefix, then text of ragged lengths; capped scores
        attention("image_prefix_capped", 4, 1937, 1937, 16, 4, 128, 128, causal=True, prefix=400, cap=30.0, padded=True),
        # the largest prompt: causal, with a bias by distance
        attention("prompt_16k_bias", 1, 16384, 16384, 16, 4, 128, 128, causal=True, bias=True),
        # one new token for each of 64 sequences, at scattered places of the pages
        append("append_token_b64", 64, 1, 8, 128, 128, 16, 2000),
        # a batch of prompts written to the cache, ragged
        append("append_prompts", 16, 2048, 8, 128, 128, 64, 0, ragged=True),
        # fp32 tokens of odd counts
        append("append_f32_odd", 5, 77, 4, 32, 64, 20, 13, dtype="f32"),
        # one sequence right after its image prefix: latency
        decode("decode_one_400", 1, 421, 421, 8, 2, 64, 64, 16),
        # ordinary serving: 64 sequences of ragged lengths, capped scores
        decode("decode_b64_ragged", 64, 130, 4000, 32, 8, 128, 128, 64, cap=30.0),
        # fp32, as many key heads as query heads, a bias by distance and sequences that start at a later key
        decode("decode_f32_mha", 8, 300, 1700, 12, 12, 64, 64, 32, dtype="f32", bias=True, first=True),
        # the largest cache: a few very long sequences
        decode("decode_long_131072", 8, 65536, 131072, 32, 8, 128, 128, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "append", "decode", "decode"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    dk, dv = rng.choice(((32, 64), (64, 64), (96, 96), (128, 128), (40, 72), (64, 128)))
    hkv = rng.choice((1, 2, 3, 4, 8))
    hq = hkv * rng.choice((1, 1, 2, 4, 5, 8))
    if op == "attention":
        lk = _log(rng, 1, 16384)
        lq = lk if rng.random() < 0.7 else _log(rng, 1, lk)
        causal = rng.random() < 0.6
        # the plain form keeps every score in memory, and fp32 has no tensor-core product of full precision
        most = LARGEST_PAIRS // (8 if dtype == "f32" else 1)
        b = _log(rng, 1, 64)
        while b > 1 and b * hq * lq * lk > most:
            b -= 1
        while hq * lq * lk > most:
            lk = (lk + 1) // 2
            lq = min(lq, lk)
        same = lq == lk
        return {"op": op, "b": b, "lq": lq, "lk": lk, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv, "dtype": dtype,
                "causal": causal, "prefix": _log(rng, 1, lk) if causal and rng.random() < 0.4 else 0,
                "offset": lk - lq if causal else 0, "docs": rng.randint(1, 12) if same and rng.random() < 0.35 else 0,
                "cap": rng.choice((0.0, 0.0, 30.0, 50.0)), "bias": rng.random() < 0.35, "padded": rng.random() < 0.3}
    es = 2 if dtype == "bf16" else 4
    page = rng.choice((16, 20, 32, 64, 128))
    b = _log(rng, 1, 256)
    if op == "append":
        t = _log(rng, 1, 2048)
        while b > 1 and b * t * hkv * (dk + dv) * es > LARGEST_APPEND:
            b -= 1
        return {"op": op, "b": b, "t": t, "hkv": hkv, "dk": dk, "dv": dv, "page": page, "past": _log(rng, 1, 4000) - 1,
                "dtype": dtype, "ragged": rng.random() < 0.4}
    hi = _log(rng, 1, 131072)
    while b > 1 and b * hi * hkv * (dk + dv) * es > LARGEST_CACHE // 2:
        b -= 1
    return {"op": op, "b": b, "lo": rng.randint(max(1, hi // 4), hi), "hi": hi, "hq": hq, "hkv": hkv, "dk": dk, "dv": dv,
            "page": page, "dtype": dtype, "cap": rng.choice((0.0, 0.0, 30.0)), "bias": rng.random() < 0.35,
            "first": rng.random() < 0.3}


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _kv_len(c):
    return _spread(c["b"], (c["lk"] + 1) // 2, c["lk"]) if c["padded"] else [c["lk"]] * c["b"]


def _doc_edges(c):
    """First tokens of a row's documents, then the first token of its padding."""
    end = c["lk"] - c["lk"] // 50
    weights = [1 + (7 * i) % 5 for i in range(c["docs"])]
    edges, at = [0], 0
    for w in weights:
        at += w
        edges.append(end * at // sum(weights))
    return edges


def _slopes(c, device=None):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], dtype=torch.float32, device=device)


def _lens(c):
    return _spread(c["b"], c["lo"], c["hi"])


def _first(length):
    return length // 5


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    d = c["dk"] + c["dv"]
    if c["op"] == "append":
        counts = _spread(c["b"], (c["t"] + 1) // 2, c["t"]) if c["ragged"] else [c["t"]] * c["b"]
        return {"bytes": 2 * sum(counts) * c["hkv"] * d * es, "flops": 0}
    if c["op"] == "decode":
        keys = sum(n - _first(n) if c["first"] else n for n in _lens(c))
        return {"bytes": (keys * c["hkv"] + c["b"] * c["hq"]) * d * es, "flops": 2 * d * c["hq"] * keys}
    # the keys that a query sees are one range [lo, hi) of its row
    i = torch.arange(c["lq"], dtype=torch.int64)
    lo, hi = torch.zeros_like(i), torch.full_like(i, c["lk"])
    if c["causal"]:
        hi = torch.minimum(hi, torch.clamp(i + c["offset"] + 1, min=c["prefix"]))
    if c["docs"]:
        edges = torch.tensor(_doc_edges(c), dtype=torch.int64)
        doc = torch.searchsorted(edges, i, right=True) - 1
        real = doc < c["docs"]
        doc = doc.clamp(max=c["docs"] - 1)
        lo, hi = edges[doc], torch.where(real, torch.minimum(hi, edges[doc + 1]), torch.zeros_like(hi))
    pairs = sum(int((torch.clamp(hi, max=n) - lo).clamp(min=0).sum()) for n in _kv_len(c))
    tokens = c["b"] * c["lq"] * c["hq"] + sum(_kv_len(c)) * c["hkv"]
    return {"bytes": tokens * d * es, "flops": 2 * d * pairs * c["hq"]}


def _pages(c, tokens, g, dev):
    """Pages with room for `tokens` tokens of each sequence, at random places, and the table that names them (-1: none)."""
    need = [(n + c["page"] - 1) // c["page"] for n in tokens]
    count = sum(need) + 3
    dt = DTYPES[c["dtype"]]
    k = torch.randn(count, c["page"], c["hkv"], c["dk"], generator=g, device=dev, dtype=dt)
    v = torch.randn(count, c["page"], c["hkv"], c["dv"], generator=g, device=dev, dtype=dt)
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    width = max(need) + 1
    slot = torch.arange(width, device=dev)[None, :]
    need_t = torch.tensor(need, device=dev)[:, None]
    start = torch.cumsum(need_t, 0) - need_t
    table = torch.where(slot < need_t, order[(start + slot).clamp(max=count - 1)], torch.full_like(order[:1], -1))
    return k, v, table.contiguous()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 11)
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "attention":
        b, lq, lk, hq, hkv, dk, dv = (c[n] for n in ("b", "lq", "lk", "hq", "hkv", "dk", "dv"))
        if lq == lk:  # the slices of a projection's output
            row = torch.randn(b, lq, hq * dk + hkv * (dk + dv), generator=g, device=dev, dtype=dt)
            q, k, v = torch.split(row, [hq * dk, hkv * dk, hkv * dv], dim=-1)
        else:
            q = torch.randn(b, lq, hq * dk, generator=g, device=dev, dtype=dt)
            k, v = torch.split(torch.randn(b, lk, hkv * (dk + dv), generator=g, device=dev, dtype=dt), [hkv * dk, hkv * dv], dim=-1)
        q *= SPREAD
        st.update(q=q.unflatten(-1, (hq, dk)), k=k.unflatten(-1, (hkv, dk)), v=v.unflatten(-1, (hkv, dv)))
        perm = torch.randperm(b, generator=g, device=dev)
        st["kv_len"] = torch.tensor(_kv_len(c), dtype=torch.int32, device=dev)[perm].contiguous() if c["padded"] else None
        st["prefix_len"] = torch.full((b,), c["prefix"], dtype=torch.int32, device=dev) if c["prefix"] else None
        st["slopes"] = _slopes(c, dev) if c["bias"] else None
        st["doc"] = None
        if c["docs"]:
            at = torch.searchsorted(torch.tensor(_doc_edges(c), device=dev), torch.arange(lk, device=dev), right=True) - 1
            at = torch.where(at < c["docs"], at, torch.full_like(at, -1)).to(torch.int32)
            st["doc"] = at[None, :].expand(b, lk).contiguous()
        st["out"] = torch.empty(b, lq, hq, dv, device=dev, dtype=dt)
        if own:
            from conv_bn_activation_gb300 import binding as cb
            st["score"] = cb.Score(scale=c["dk"] ** -0.5, softcap=c["cap"], slopes=st["slopes"], causal=c["causal"],
                                   q_offset=c["offset"], prefix_len=st["prefix_len"], kv_len=st["kv_len"],
                                   doc_q=st["doc"], doc_k=st["doc"])
        return st
    if c["op"] == "append":
        b, t = c["b"], c["t"]
        st["k_pages"], st["v_pages"], st["table"] = _pages(c, [c["past"] + t] * b, g, dev)
        new = torch.randn(b, t, c["hkv"] * (c["dk"] + c["dv"]), generator=g, device=dev, dtype=dt)
        k, v = torch.split(new, [c["hkv"] * c["dk"], c["hkv"] * c["dv"]], dim=-1)
        st.update(k=k.unflatten(-1, (c["hkv"], c["dk"])), v=v.unflatten(-1, (c["hkv"], c["dv"])))
        perm = torch.randperm(b, generator=g, device=dev)
        st["pos"] = torch.full((b,), c["past"], dtype=torch.int32, device=dev)
        st["count"] = (torch.tensor(_spread(b, (t + 1) // 2, t), dtype=torch.int32, device=dev)[perm].contiguous()
                       if c["ragged"] else None)
    else:
        b = c["b"]
        lens = torch.tensor(_lens(c))[torch.randperm(b, generator=torch.Generator().manual_seed(int(seed)))]
        st["k_pages"], st["v_pages"], st["table"] = _pages(c, lens.tolist(), g, dev)
        st["length"] = lens.to(device=dev, dtype=torch.int32)
        st["first"] = _first(lens).to(device=dev, dtype=torch.int32) if c["first"] else None
        st["slopes"] = _slopes(c, dev) if c["bias"] else None
        st["q"] = torch.randn(b, c["hq"], c["dk"], generator=g, device=dev, dtype=dt) * SPREAD
        st["out"] = torch.empty(b, c["hq"], c["dv"], device=dev, dtype=dt)
    if own:
        from conv_bn_activation_gb300 import binding as cb
        st["cache"] = cb.PagedCache(st["k_pages"], st["v_pages"], st["table"])
        if c["op"] == "decode":
            st["workspace"] = torch.empty(cb.attention_decode_workspace(st["q"], st["cache"]), dtype=torch.uint8, device=dev)
    return st


def _softmax_product(s, keep, v):
    """softmax of `s` over the keys that `keep` marks, times `v`; zero where there are none."""
    s = torch.where(keep, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)


def _attention(st):
    c, dev = st["case"], st["q"].device
    group = c["hq"] // c["hkv"]
    q = st["q"].float().transpose(1, 2)
    k = st["k"].float().transpose(1, 2).repeat_interleave(group, dim=1)
    v = st["v"].float().transpose(1, 2).repeat_interleave(group, dim=1)
    s = torch.matmul(q, k.transpose(-1, -2)) * c["dk"] ** -0.5
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    i = torch.arange(c["lq"], device=dev)[:, None] + c["offset"]
    j = torch.arange(c["lk"], device=dev)[None, :]
    if st["slopes"] is not None:
        s = s - st["slopes"][:, None, None] * (i - j).abs().float()
    keep = torch.ones(1, 1, c["lq"], c["lk"], dtype=torch.bool, device=dev)
    if c["causal"]:
        seen = (j <= i)[None, None]
        keep = seen if st["prefix_len"] is None else seen | (j < st["prefix_len"][:, None, None])[:, None]
    if st["kv_len"] is not None:
        keep = keep & (j < st["kv_len"][:, None, None])[:, None]
    if st["doc"] is not None:
        keep = keep & ((st["doc"][:, :, None] == st["doc"][:, None, :]) & (st["doc"] >= 0)[:, None, :])[:, None]
    return _softmax_product(s, keep, v).transpose(1, 2).to(st["q"].dtype).contiguous()


def _append(st):
    c = st["case"]
    t = torch.arange(c["t"], device=st["pos"].device)[None, :]
    if st["count"] is not None:  # a place past a sequence's count takes its first token a second time
        t = torch.where(t < st["count"][:, None], t, torch.zeros_like(t))
    at = st["pos"][:, None].long() + t.expand(c["b"], c["t"])
    page, slot = st["table"].gather(1, at // c["page"]).long(), at % c["page"]
    row = torch.arange(c["b"], device=t.device)[:, None]
    st["k_pages"][page, slot] = st["k"][row, t]
    st["v_pages"][page, slot] = st["v"][row, t]
    return st["k_pages"], st["v_pages"]


def _decode(st):
    c, dev = st["case"], st["q"].device
    group = c["hq"] // c["hkv"]
    table = st["table"].clamp(min=0).long()
    q = st["q"].float().reshape(c["b"], c["hkv"], group, c["dk"])
    k = st["k_pages"][table].flatten(1, 2).permute(0, 2, 3, 1).float()
    v = st["v_pages"][table].flatten(1, 2).permute(0, 2, 1, 3).float()
    s = torch.matmul(q, k) * c["dk"] ** -0.5
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    j = torch.arange(s.shape[-1], device=dev)[None, :]
    if st["slopes"] is not None:
        far = (st["length"][:, None] - 1 - j).float()
        s = s - st["slopes"].reshape(1, c["hkv"], group, 1) * far[:, None, None, :]
    keep = j < st["length"][:, None]
    if st["first"] is not None:
        keep = keep & (j >= st["first"][:, None])
    out = _softmax_product(s, keep[:, None, None, :], v)
    return out.reshape(c["b"], c["hq"], c["dv"]).to(st["q"].dtype)


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"attention": _attention, "append": _append, "decode": _decode}[op](state)
    from conv_bn_activation_gb300 import binding as cb
    c = state["case"]
    if op == "attention":
        return cb.attention(state["q"], state["k"], state["v"], state["out"], state["score"])
    if op == "append":
        cb.cache_append(state["k"], state["v"], state["cache"], state["pos"], count=state["count"])
        return state["k_pages"], state["v_pages"]
    return cb.attention_decode(state["q"], state["cache"], state["length"], state["out"], state["workspace"],
                               scale=c["dk"] ** -0.5, softcap=c["cap"], slopes=state["slopes"], first=state["first"])


def _exact_rows(q, k, v, keep, bias, c):
    """One head in 64 bits: q [n, dk], k [m, dk], v [m, dv]; keep, bias broadcast over [n, m]."""
    s = (q.double() @ k.double().T) / math.sqrt(c["dk"])
    if c["cap"]:
        s = torch.tanh(s / c["cap"]) * c["cap"]
    if bias is not None:
        s = s + bias
    s = s.masked_fill(~keep, -math.inf)
    norm = torch.logsumexp(s, dim=-1, keepdim=True)
    weight = torch.exp(s - norm).masked_fill(~keep, 0.0)
    return weight @ v.double()


def exact(case, seed):
    c = dict(case)
    st = prepare(case, seed)
    if c["op"] == "append":  # values are moved, not computed
        return None
    dev, group = st["q"].device, c["hq"] // c["hkv"]
    if c["op"] == "attention":
        if 2.0 * (c["dk"] + c["dv"]) * c["b"] * c["hq"] * c["lq"] * c["lk"] > 6e12:
            return None
        out = torch.empty(c["b"], c["lq"], c["hq"], c["dv"], dtype=torch.float64, device=dev)
        at = torch.arange(c["lq"], device=dev).unsqueeze(1) + c["offset"]
        key = torch.arange(c["lk"], device=dev).unsqueeze(0)
        for b in range(c["b"]):
            keep = (key < (st["kv_len"][b] if st["kv_len"] is not None else c["lk"])).expand(c["lq"], c["lk"])
            if c["causal"]:
                keep = keep & ((key <= at) | (key < c["prefix"]))
            if st["doc"] is not None:
                keep = keep & (st["doc"][b].unsqueeze(1) == st["doc"][b].unsqueeze(0)) & (st["doc"][b] != -1).unsqueeze(0)
            for h in range(c["hq"]):
                bias = -st["slopes"][h].double() * (at - key).abs().double() if st["slopes"] is not None else None
                out[b, :, h] = _exact_rows(st["q"][b, :, h], st["k"][b, :, h // group], st["v"][b, :, h // group], keep, bias, c)
        return out
    out = torch.empty(c["b"], c["hq"], c["dv"], dtype=torch.float64, device=dev)
    for b in range(c["b"]):
        n = int(st["length"][b])
        lo = int(st["first"][b]) if st["first"] is not None else 0
        pages = st["table"][b, :(n + c["page"] - 1) // c["page"]].long()
        k, v = st["k_pages"][pages].flatten(0, 1)[lo:n], st["v_pages"][pages].flatten(0, 1)[lo:n]
        for h in range(c["hkv"]):
            keep = torch.ones(group, n - lo, dtype=torch.bool, device=dev)
            bias = None
            if st["slopes"] is not None:
                bias = -st["slopes"][h * group:(h + 1) * group, None].double() * (n - 1 - torch.arange(lo, n, device=dev)).double()
            out[b, h * group:(h + 1) * group] = _exact_rows(st["q"][b, h * group:(h + 1) * group], k[:, h], v[:, h], keep, bias, c)
    return out
