"""Refusals of the head rotation's and the 4-bit cache's entry points, on the host: nothing is launched (no GPU)."""
import ctypes

import pytest

from test_attention_host import DATA, FAR, OnDevice, heads

r = ctypes.byref


def ref(x):
    return r(x) if x is not None else None


def rule(cblib, norm=1, eps=1e-6, rotary=64, adjacent=0, axes=3, freq=DATA, axis=DATA, pos=DATA, **kw):
    h = cblib.CbHeadRule(norm, eps, None, None, rotary, adjacent, axes, freq, axis, pos, 16, 8)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def rotate(cblib, **kw):
    a = {"q": heads(cblib), "k": heads(cblib, h=2, data=DATA + FAR), "rule": rule(cblib), "q_out": heads(cblib, data=DATA + 2 * FAR),
         "k_out": heads(cblib, h=2, data=DATA + 3 * FAR)}
    a.update(kw)
    return cblib.load().cb_norm_rotate(ref(a["q"]), ref(a["k"]), ref(a["rule"]), ref(a["q_out"]), ref(a["k_out"]), None)


@pytest.mark.parametrize("name", ["q", "k", "rule", "q_out", "k_out"])
def test_rotate_null(cblib, name):
    assert rotate(cblib, **{name: None}) == cblib.ERR_INVALID_ARG


def test_rotate_shapes(cblib):
    k = dict(h=2, data=DATA + FAR)
    for kw in ({"k": heads(cblib, d=32, **k)}, {"k": heads(cblib, l=7, **k)}, {"k": heads(cblib, b=1, **k)}, {"k": heads(cblib, dtype=0, **k)},
               {"q_out": heads(cblib, h=3, data=DATA + 2 * FAR)}, {"q_out": heads(cblib, dtype=0, data=DATA + 2 * FAR)},
               {"k_out": heads(cblib, h=2, l=9, data=DATA + 3 * FAR)}, {"q": heads(cblib, dtype=5)}, {"q": heads(cblib, data=0)}):
        assert rotate(cblib, **kw) == cblib.ERR_INVALID_ARG, kw


def test_rotate_rules(cblib):
    inf, nan = float("inf"), float("nan")
    for kw in ({"eps": -1.0}, {"eps": nan}, {"eps": inf}, {"rotary": 63}, {"rotary": 66}, {"rotary": -2}, {"axes": 0}, {"axes": 9},
               {"freq": None}, {"pos": None}, {"pos_stride_axis": -1}, {"pos_stride_b": -1}):
        assert rotate(cblib, rule=rule(cblib, **kw)) == cblib.ERR_INVALID_ARG, kw


def test_rotate_overlaps(cblib):
    I = cblib.ERR_INVALID_ARG
    assert rotate(cblib, q_out=heads(cblib, data=DATA + 2)) == I  # neither in place nor apart
    assert rotate(cblib, q_out=heads(cblib, sh=128, sl=512)) == I  # the queries' data with other strides
    assert rotate(cblib, q_out=heads(cblib, h=4, data=DATA + FAR)) == I  # over the keys
    assert rotate(cblib, k_out=heads(cblib, h=2)) == I  # over the queries
    assert rotate(cblib, k_out=heads(cblib, h=2, data=DATA + 2 * FAR)) == I  # both results
    out = dict(data=DATA + 2 * FAR)
    for kw in ({"sh": 0}, {"sh": 32}, {"sl": 128}, {"sb": 0}, {"sb": 8 * 256 - 64}):  # rows of a result that overlap
        assert rotate(cblib, q_out=heads(cblib, **out, **kw)) == I, kw
        assert rotate(cblib, q=heads(cblib, **kw), q_out=heads(cblib, **kw)) == I, kw  # in place on a broadcast


def test_rotate_unsupported_alignment_and_nothing(cblib):
    one = {n: heads(cblib, d=136, h=2, data=DATA + i * FAR) for i, n in enumerate(("q", "k", "q_out", "k_out"))}
    assert rotate(cblib, **one) == cblib.ERR_UNSUPPORTED
    many = {n: heads(cblib, b=1 << 16, l=1 << 15, h=1, d=2, data=DATA + i * (1 << 40)) for i, n in enumerate(("q", "k", "q_out", "k_out"))}
    assert rotate(cblib, rule=rule(cblib, rotary=2), **many) == cblib.ERR_UNSUPPORTED
    assert rotate(cblib, q=heads(cblib, data=DATA + 1)) == cblib.ERR_ALIGNMENT
    assert rotate(cblib, k_out=heads(cblib, h=2, data=DATA + 3 * FAR + 1)) == cblib.ERR_ALIGNMENT
    none = {n: heads(cblib, b=0, data=0) for n in ("q", "k", "q_out", "k_out")}
    assert rotate(cblib, rule=rule(cblib, pos=None), **none) == cblib.OK


def cache(cblib, P=10, page=16, H=2, dk=64, dv=64, batch=2, width=5, k=DATA, table=DATA, **kw):
    far, (bk, bv), (sk, sv) = 1 << 22, ((dk + 1) // 2, (dv + 1) // 2), (2 * ((dk + 63) // 64), 2 * ((dv + 63) // 64))
    c = cblib.CbPagedCache4(k, DATA + far, DATA + 2 * far, DATA + 3 * far, P, page, H, dk, dv, page * H * bk, H * bk, bk,
                            page * H * bv, H * bv, bv, page * H * sk, H * sk, sk, page * H * sv, H * sv, sv, table, batch, width, width)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def tokens(cblib, name, k=None, v=None, c=None, pos=DATA):
    k = heads(cblib, h=2, data=DATA + FAR) if k is None else k
    v = heads(cblib, h=2, data=DATA + 2 * FAR) if v is None else v
    c = cache(cblib) if c is None else c
    if name == "append":
        return cblib.load().cb_cache4_append(r(k), r(v), pos, None, r(c), None)
    return cblib.load().cb_cache4_read(r(c), pos, None, r(k), r(v), None)


BAD_CACHES = [{"page": 0}, {"P": -1}, {"H": 0}, {"dk": 0}, {"k": 0}, {"k_scale": 0}, {"v_scale": 0}, {"v": 0}, {"table": 0}, {"max_pages": -1},
              {"page": 1 << 20, "width": 1 << 12}, {"k_stride_page": -1}, {"vs_stride_head": -1}, {"table_stride": -1}, {"batch": 3}]


@pytest.mark.parametrize("name", ["append", "read"])
def test_tokens_refusals(cblib, name):
    I, far = cblib.ERR_INVALID_ARG, dict(data=DATA + FAR)
    for kw in BAD_CACHES:
        assert tokens(cblib, name, c=cache(cblib, **kw)) == I, kw
    assert tokens(cblib, name, k=heads(cblib, h=4, **far)) == I and tokens(cblib, name, v=heads(cblib, h=2, d=32, **far)) == I
    assert tokens(cblib, name, k=heads(cblib, h=2, l=3, **far)) == I and tokens(cblib, name, k=heads(cblib, h=2, dtype=0, **far)) == I
    assert tokens(cblib, name, k=heads(cblib, h=2, data=0)) == I
    for at in (DATA, DATA + (1 << 22), DATA + 2 * (1 << 22) + 64, DATA + 3 * (1 << 22), DATA - 2):  # in the pages
        assert tokens(cblib, name, k=heads(cblib, h=2, data=at)) == I and tokens(cblib, name, v=heads(cblib, h=2, data=at)) == I, at
    wide = dict(h=2, d=136)
    assert tokens(cblib, name, k=heads(cblib, **wide, **far), c=cache(cblib, dk=136)) == cblib.ERR_UNSUPPORTED
    assert tokens(cblib, name, k=heads(cblib, h=2, data=DATA + FAR + 1)) == cblib.ERR_ALIGNMENT
    assert tokens(cblib, name, c=cache(cblib, k_scale=DATA + (1 << 23) + 1)) == cblib.ERR_ALIGNMENT
    lib = cblib.load()
    assert lib.cb_cache4_append(None, None, DATA, None, None, None) == I and lib.cb_cache4_read(None, None, None, None, None, None) == I
    empty = heads(cblib, h=2, l=0)
    assert tokens(cblib, name, k=empty, v=empty, pos=None) == cblib.OK
    if name == "append":
        assert tokens(cblib, name, pos=None) == I
    else:
        assert tokens(cblib, name, v=heads(cblib, h=2, **far)) == I  # both results
        for kw in ({"sh": 0}, {"sl": 64}, {"sb": 0}):
            assert tokens(cblib, name, k=heads(cblib, h=2, **far, **kw)) == I, kw


def decode(cblib, q=None, c=None, length=DATA, out=None, scale=0.125, cap=0.0, ws=DATA, size=1 << 40):
    q = heads(cblib, l=1, data=DATA + FAR) if q is None else q
    out = heads(cblib, l=1, data=DATA + 2 * FAR) if out is None else out
    c = cache(cblib) if c is None else c
    return cblib.load().cb_attention_decode4(r(q), r(c), length, None, scale, cap, None, r(out), ws, size, None)


def test_decode_refusals(cblib):
    I, q, o = cblib.ERR_INVALID_ARG, dict(l=1, data=DATA + FAR), dict(l=1, data=DATA + 2 * FAR)
    for kw in BAD_CACHES:
        assert decode(cblib, c=cache(cblib, **kw)) == I, kw
    assert decode(cblib, length=None) == I and decode(cblib, ws=None) == I
    assert decode(cblib, q=heads(cblib, l=2, data=DATA + FAR)) == I and decode(cblib, q=heads(cblib, d=32, **q)) == I
    assert decode(cblib, q=heads(cblib, h=3, **q)) == I and decode(cblib, q=heads(cblib, b=3, **q)) == I
    assert decode(cblib, out=heads(cblib, h=2, **o)) == I and decode(cblib, out=heads(cblib, l=1, data=DATA + FAR)) == I
    assert decode(cblib, out=heads(cblib, dtype=0, **o)) == I and decode(cblib, out=heads(cblib, sh=0, **o)) == I
    for part in range(4):
        assert decode(cblib, out=heads(cblib, l=1, data=DATA + part * (1 << 22) + 8)) == I
    assert decode(cblib, scale=0.0) == I and decode(cblib, cap=-1.0) == I
    assert decode(cblib, ws=DATA + 16) == cblib.ERR_ALIGNMENT
    assert decode(cblib, q=heads(cblib, l=1, data=DATA + FAR + 1)) == cblib.ERR_ALIGNMENT
    assert decode(cblib, c=cache(cblib, v_scale=DATA + 3 * (1 << 22) + 1)) == cblib.ERR_ALIGNMENT
    assert decode(cblib, q=heads(cblib, d=136, **q), c=cache(cblib, dk=136)) == cblib.ERR_UNSUPPORTED
    n, lib = ctypes.c_size_t(0), cblib.load()
    assert lib.cb_attention_decode4_workspace(None, None, r(n)) == I
    assert lib.cb_attention_decode4_workspace(r(heads(cblib, l=1)), r(cache(cblib)), None) == I


def test_packed_rule_has_the_structures_layout(cblib):
    import torch
    freq, axis = torch.zeros(16), torch.zeros(16, dtype=torch.int32)
    w, pos = torch.ones(64), torch.zeros(5, 3, 9, dtype=torch.int32)[1:3, :, 2:]
    with pytest.raises(ValueError):
        cblib.Rotation(freq, axis=axis, axes=2)  # host tensors

    class Claims(torch.Tensor):
        def get_device(self):
            return 0

    freq, axis, w, pos = (t.as_subclass(Claims) for t in (freq, axis, w, pos))
    rot = cblib.Rotation(freq, axis=axis, axes=2, adjacent=True, norm=True, eps=0.25, k_weight=w)
    packed = rot.view(3, 7, 64, pos, 0)
    for bad in ((3, 7, 32, pos, 0), (3, 7, 64, pos, 1), (3, 7, 64, None, 0), (3, 6, 64, pos, 0), (3, 7, 64, pos.long(), 0),
                (3, 7, 64, pos.transpose(1, 2).contiguous().transpose(1, 2), 0)):
        with pytest.raises(ValueError):
            rot.view(*bad)
    assert len(packed) == ctypes.sizeof(cblib.CbHeadRule)
    got = cblib.CbHeadRule.from_buffer_copy(packed)
    assert (got.norm, got.eps, got.q_weight, got.k_weight) == (1, 0.25, None, w.data_ptr())
    assert (got.rotary, got.adjacent, got.axes, got.freq, got.axis) == (32, 1, 2, freq.data_ptr(), axis.data_ptr())
    assert (got.pos, got.pos_stride_axis, got.pos_stride_b) == (pos.data_ptr(), 27, 9)


def test_binding_checks(cblib):
    import torch
    u8, bf, i32 = torch.uint8, torch.bfloat16, torch.int32
    with pytest.raises(ValueError):
        cblib.Rotation(q_weight=torch.ones(8))
    with pytest.raises(ValueError):
        cblib.Rotation(axis=torch.zeros(8, dtype=i32))
    codes, scales, table = torch.zeros(2, 4, 1, 32, dtype=u8), torch.zeros(2, 4, 1, 2, dtype=bf), torch.zeros(1, 1, dtype=i32)
    for bad in ((codes[..., :16], scales, codes, scales, table), (codes, scales[..., :1], codes, scales, table),
                (codes, scales, codes.to(torch.int8), scales, table), (codes, scales.float(), codes, scales, table),
                (codes, scales, codes[:1], scales, table), (codes, scales, codes, scales, table.long()),
                (codes, scales, codes.transpose(2, 3).contiguous().transpose(2, 3).expand(2, 4, 2, 32)[:, :, ::2, ::2], scales, table)):
        with pytest.raises(ValueError):
            cblib.PagedCache4(*bad)
    assert [cblib.scales_per_row(d) for d in (1, 32, 64, 65, 128)] == [2, 2, 2, 4, 4]


@pytest.mark.parametrize("device", [-1, 1], ids=["host", "another"])
def test_binding_checks_every_tensors_device(cblib, monkeypatch, device):
    import torch
    on = OnDevice(monkeypatch, cblib)
    s, B, h = on.stream, (2, 3, 4, 64), torch.bfloat16

    def refused(call, shapes):
        tensors = {n: on.make(*sh, dtype=dt) for n, (sh, dt) in shapes.items()}
        with pytest.raises(AssertionError, match="was called"):
            call(tensors)  # all on one device: the call goes on to the library
        for n, (sh, dt) in shapes.items():
            with pytest.raises(ValueError):
                call({**tensors, n: on.make(*sh, dtype=dt, device=device)})

    refused(lambda t: cblib.norm_rotate(t["q"], t["k"], t["pos"], cblib.Rotation(t["f"], axis=t["a"], axes=2, norm=True, q_weight=t["w"],
                                                                                 k_weight=t["x"]), t["qo"], t["ko"], stream=s),
            {"q": (B, h), "k": (B, h), "qo": (B, h), "ko": (B, h), "pos": ((2, 2, 3), on.i32), "f": ((32,), on.f32),
             "a": ((32,), on.i32), "w": ((64,), on.f32), "x": ((64,), on.f32)})
    u8 = torch.uint8
    pages = {"kc": ((5, 16, 4, 32), u8), "ks": ((5, 16, 4, 2), h), "vc": ((5, 16, 4, 32), u8), "vs": ((5, 16, 4, 2), h),
             "table": ((2, 3), on.i32)}

    def made(t):
        return cblib.PagedCache4(t["kc"], t["ks"], t["vc"], t["vs"], t["table"])

    refused(lambda t: cblib.cache4_append(t["k"], t["v"], made(t), t["pos"], count=t["count"], stream=s),
            {"k": (B, h), "v": (B, h), **pages, "pos": ((2,), on.i32), "count": ((2,), on.i32)})
    refused(lambda t: cblib.cache4_read(made(t), t["k"], t["v"], first=t["first"], count=t["count"], stream=s),
            {"k": (B, h), "v": (B, h), **pages, "first": ((2,), on.i32), "count": ((2,), on.i32)})
    refused(lambda t: cblib.attention_decode4(t["q"], made(t), t["n"], t["out"], t["ws"], 0.1, slopes=t["slopes"], first=t["first"], stream=s),
            {"q": ((2, 4, 64), h), **pages, "n": ((2,), on.i32), "out": ((2, 4, 64), h), "ws": ((4096,), u8), "slopes": ((4,), on.f32),
             "first": ((2,), on.i32)})


def test_stored_values_against_whole_numbers(cblib):
    """The tests' own reference against exact arithmetic: scales and codes of borders."""
    from fractions import Fraction as F

    import torch

    import cache4_ref as ref4
    g = torch.Generator().manual_seed(3)
    x = torch.randn(60, 32, generator=g)
    x[::2] = x[::2].to(torch.bfloat16).float()
    codes, scales = ref4.store(x)
    got = ref4.values(codes, scales, 32)
    for row, s, v in zip(x.tolist(), scales[:, 0].tolist(), got.tolist()):
        top, s = max(abs(F(e)) for e in row) / 7, F(s)
        unit = F(2) ** next(e for e in range(-40, 40) if s < F(2) ** (e + 8))  # s has 8 bits
        assert s % unit == 0 and abs(top - s) <= unit / 2
        for e, y in zip(row, v):
            c = F(y) / s
            assert c.denominator == 1 and abs(c) <= 7
            d = abs(F(e) / s - c)
            assert d < F(1, 2) or (d == F(1, 2) and c % 2 == 0) or abs(c) == 7


def test_binding_refuses_another_device_than_the_current_one(cblib, monkeypatch):
    import torch
    on = OnDevice(monkeypatch, cblib)
    cblib.heads(torch.zeros(1, 1, 1, 8))  # what the first call sets up
    monkeypatch.setattr(cblib, "_several", True)
    k, v = on.make(2, 3, 4, 64), on.make(2, 3, 4, 64)
    for current, wrong in ((0, AssertionError), (1, ValueError)):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
        with pytest.raises(wrong):
            cblib.norm_rotate(k, v, None, cblib.Rotation(norm=True), stream=on.stream)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
def test_heads_that_lie_between_anothers(cblib, dtype):
    """Queries, keys and values side by side for each head ([B, L, H, 3, D]): views that share no byte are no overlap.
    All data lies one byte off, which is refused after the overlaps: nothing is launched where there is a GPU."""
    e, I, A = 2 if dtype else 4, cblib.ERR_INVALID_ARG, cblib.ERR_ALIGNMENT

    def at(part, **kw):
        a = dict(h=4, data=DATA + part * 64 * e + 1, sh=3 * 64, sl=4 * 3 * 64, dtype=dtype)
        a.update(kw)
        return heads(cblib, **a)

    def in_place(q, k):
        return rotate(cblib, q=q, k=k, q_out=q, k_out=k)

    assert in_place(at(0), at(1)) == A
    assert in_place(at(0), at(1, data=DATA + 32 * e + 1)) == I  # half over the queries
    assert in_place(at(0), at(1, sh=2 * 64)) == I  # another step of heads
    gap = dict(sl=4 * 3 * 64 + 64)
    assert in_place(at(0, **gap), at(1, **gap)) == A
    out = dict(data=DATA + 2 * FAR + 1, dtype=dtype)
    for near in (dict(sl=3 * 3 * 64), dict(sb=64 * 3 * 64)):  # tokens, sequences into which the heads of others reach
        assert rotate(cblib, q=at(0, **near), k=at(1, **near), q_out=heads(cblib, **out), k_out=at(0, **near)) == I
    assert in_place(at(0), at(1, h=1)) == A


def test_views_that_are_taken_share_no_byte(cblib):
    """Small views at random strides: what is not refused as an overlap has no element twice.  All data lies one byte off, as
    above."""
    import random

    rng = random.Random(5)

    def drawn():
        d, h, ln, b = rng.choice((2, 4)), rng.randint(1, 3), rng.randint(1, 3), rng.randint(1, 2)
        pick = lambda low: rng.choice((low, low + 2, 2 * low, 3 * low, rng.randint(0, 60)))  # noqa: E731
        sh = pick(d)
        sl = pick(max(sh * h, 1))
        return dict(b=b, l=ln, h=h, d=d, sh=sh, sl=sl, sb=pick(max(sl * ln, 1)))

    def bytes_of(v, at):
        return [at + 4 * (b * v["sb"] + i * v["sl"] + h * v["sh"] + d) for b in range(v["b"]) for i in range(v["l"]) for h in range(v["h"])
                for d in range(v["d"])]

    taken = {True: 0, False: 0}
    for _ in range(6000):
        v = drawn()
        w = dict(drawn(), b=v["b"], l=v["l"], h=v["h"], d=v["d"]) if rng.random() < 0.3 else v
        at = DATA + 4 * rng.randint(0, 40)
        st = rotate(cblib, q=heads(cblib, dtype=0, data=DATA + 1, **v), q_out=heads(cblib, dtype=0, data=at + 1, **w), k=None, k_out=None,
                    rule=rule(cblib, rotary=0))
        assert st in (cblib.ERR_INVALID_ARG, cblib.ERR_ALIGNMENT)
        out = bytes_of(w, at)
        same = at == DATA and w == v
        free = len(set(out)) == len(out) and (same or not set(out) & set(bytes_of(v, DATA)))
        if st != cblib.ERR_INVALID_ARG:
            assert free, (v, w, at)
        taken[st != cblib.ERR_INVALID_ARG] += free
    assert taken[True] > 4 * taken[False] > 0  # most of those that could be taken are


def test_counts_of_heads_that_fit_the_kernels(cblib):
    """Heads are counted in 32 bits, with their dims and both kinds together: more than 65536 are refused, before anything
    is worked out from them."""
    U, big = cblib.ERR_UNSUPPORTED, 65537
    huge = 1 << 40
    for h in (big, (1 << 31) - 1):
        q, out = (heads(cblib, b=1, l=1, h=h, d=8, data=DATA + i * huge) for i in (0, 1))
        k, k_out = (heads(cblib, b=1, l=1, h=1, d=8, data=DATA + i * huge) for i in (2, 3))
        assert rotate(cblib, q=q, k=k, q_out=out, k_out=k_out, rule=rule(cblib, rotary=8)) == U
        assert rotate(cblib, q=k, k=q, q_out=k_out, k_out=out, rule=rule(cblib, rotary=8)) == U
        c = cblib.CbPagedCache4(DATA + 4 * huge, DATA + 5 * huge, DATA + 6 * huge, DATA + 7 * huge, 1, 1, h, 8, 8, h * 4, h * 4, 4, h * 4, h * 4,
                                4, h * 2, h * 2, 2, h * 2, h * 2, 2, DATA, 1, 1, 1)
        for name in ("append", "read"):
            assert tokens(cblib, name, k=q, v=out, c=c) == U
        assert decode(cblib, q=q, c=c, out=out) == U
        n = ctypes.c_size_t(0)
        assert cblib.load().cb_attention_decode4_workspace(r(q), r(c), r(n)) == U


def test_every_call_refuses_another_device_than_the_current_one(cblib, monkeypatch):
    """Attention, the caches and the rotation all launch on the current device; a stream does not change that."""
    import torch
    on = OnDevice(monkeypatch, cblib)
    cblib.heads(torch.zeros(1, 1, 1, 8))  # what the first call sets up
    monkeypatch.setattr(cblib, "_several", True)
    u8, bf, B = torch.uint8, torch.bfloat16, 2
    q, k, v, o = (on.make(B, 3, 4, 64) for _ in range(4))
    one, out, n = on.make(B, 4, 64), on.make(B, 4, 64), on.make(B, dtype=on.i32)
    ws, table = on.make(4096, dtype=u8), on.make(B, 3, dtype=on.i32)
    cache = cblib.PagedCache(on.make(5, 16, 4, 64), on.make(5, 16, 4, 64), table)
    codes, scales = on.make(5, 16, 4, 32, dtype=u8), on.make(5, 16, 4, 2, dtype=bf)
    cache4 = cblib.PagedCache4(codes, scales, codes, scales, table)
    for stream in (None, on.stream):
        if stream is None:
            monkeypatch.setattr(cblib, "_raw_stream", lambda device: 0)
        calls = [lambda: cblib.attention(q, k, v, o, cblib.Score(0.1), stream=stream),
                 lambda: cblib.cache_append(k, v, cache, n, stream=stream),
                 lambda: cblib.attention_decode(one, cache, n, out, ws, 0.1, stream=stream),
                 lambda: cblib.norm_rotate(q, k, None, cblib.Rotation(norm=True), stream=stream),
                 lambda: cblib.cache4_append(k, v, cache4, n, stream=stream),
                 lambda: cblib.cache4_read(cache4, k, v, stream=stream),
                 lambda: cblib.attention_decode4(one, cache4, n, out, ws, 0.1, stream=stream)]
        for call in calls:
            for current, wrong in ((0, AssertionError), (1, ValueError)):
                monkeypatch.setattr(torch.cuda, "current_device", lambda current=current: current)
                with pytest.raises(wrong):
                    call()
