"""Refusals of the attention entry points, on the host: nothing is launched (no GPU)."""
import ctypes

import pytest

DATA = 1 << 20  # never dereferenced


def heads(cblib, b=2, l=8, h=4, d=64, data=DATA, dtype=1, sb=None, sl=None, sh=None):
    sh = d if sh is None else sh
    sl = h * d if sl is None else sl
    return cblib.CbHeads(data, b, l, h, d, l * sl if sb is None else sb, sl, sh, dtype)


def score(cblib, scale=0.125, softcap=0.0, **kw):
    s = cblib.CbScore(scale, softcap)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def attention(cblib, **kw):
    far = 1 << 24
    a = {"q": heads(cblib), "k": heads(cblib, h=2, data=DATA + far), "v": heads(cblib, h=2, data=DATA + 2 * far),
         "out": heads(cblib, data=DATA + 3 * far), "score": score(cblib)}
    a.update(kw)
    r = ctypes.byref
    null = lambda x: r(x) if x is not None else None  # noqa: E731
    return cblib.load().cb_attention(null(a["q"]), null(a["k"]), null(a["v"]), null(a["score"]), null(a["out"]), None)


@pytest.mark.parametrize("name", ["q", "k", "v", "out", "score"])
def test_attention_null(cblib, name):
    assert attention(cblib, **{name: None}) == cblib.ERR_INVALID_ARG


def test_attention_shapes(cblib):
    far = 1 << 24
    bad = [{"k": heads(cblib, h=3, data=DATA + far), "v": heads(cblib, h=3, data=DATA + far)},  # 4 % 3
           {"k": heads(cblib, b=1, h=2, data=DATA + far)}, {"v": heads(cblib, l=7, h=2, data=DATA + far)},
           {"k": heads(cblib, h=2, d=32, data=DATA + far)}, {"out": heads(cblib, d=32, data=DATA + 3 * far)},
           {"out": heads(cblib, l=9, data=DATA + 3 * far)}, {"k": heads(cblib, h=2, dtype=0, data=DATA + far)},
           {"q": heads(cblib, dtype=7)}, {"q": heads(cblib, data=0)}, {"q": heads(cblib, sl=-1, sb=0)},
           {"q": heads(cblib, h=0)}, {"out": heads(cblib, data=DATA + 128)}]  # the last overlaps q
    for kw in bad:
        assert attention(cblib, **kw) == cblib.ERR_INVALID_ARG, kw


def test_attention_scores(cblib):
    inf, nan = float("inf"), float("nan")
    for kw in ({"scale": 0.0}, {"scale": -1.0}, {"scale": nan}, {"scale": inf}, {"softcap": -1.0}, {"softcap": nan},
               {"prefix_len": DATA}, {"doc_q": DATA}, {"doc_k": DATA}, {"q_offset": 1 << 30}):
        assert attention(cblib, score=score(cblib, **kw)) == cblib.ERR_INVALID_ARG, kw


def test_attention_unsupported_and_alignment(cblib):
    far = 1 << 24
    q, o = heads(cblib, d=136), heads(cblib, d=64, data=DATA + 3 * far)
    assert attention(cblib, q=q, k=heads(cblib, h=2, d=136, data=DATA + far), out=o) == cblib.ERR_UNSUPPORTED
    v, o = heads(cblib, h=2, d=129, data=DATA + far), heads(cblib, d=129, data=DATA + 3 * far)
    assert attention(cblib, v=v, out=o) == cblib.ERR_UNSUPPORTED
    assert attention(cblib, q=heads(cblib, data=DATA + 1)) == cblib.ERR_ALIGNMENT


def test_attention_nothing_to_do(cblib):
    e = {n: heads(cblib, b=0, h=2 if n in "kv" else 4, data=0) for n in ("q", "k", "v", "out")}
    assert attention(cblib, **e) == cblib.OK


def cache(cblib, P=10, page=16, H=2, dk=64, dv=64, batch=2, width=5, dtype=1, k=DATA, table=DATA, **kw):
    c = cblib.CbPagedCache(k, DATA + (1 << 24), P, page, H, dk, dv, page * H * dk, H * dk, dk, page * H * dv, H * dv, dv, table,
                           batch, width, width, dtype)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def append(cblib, k=None, v=None, pos=DATA, c=None):
    k = heads(cblib, h=2) if k is None else k
    v = heads(cblib, h=2) if v is None else v
    c = cache(cblib) if c is None else c
    return cblib.load().cb_cache_append(ctypes.byref(k), ctypes.byref(v), pos, None, ctypes.byref(c), None)


def test_append_refusals(cblib):
    I = cblib.ERR_INVALID_ARG
    assert append(cblib, pos=None) == I
    assert append(cblib, k=heads(cblib, h=4)) == I and append(cblib, v=heads(cblib, h=2, d=32)) == I
    assert append(cblib, k=heads(cblib, h=2, l=3)) == I and append(cblib, c=cache(cblib, batch=3)) == I
    assert append(cblib, c=cache(cblib, dtype=0)) == I and append(cblib, c=cache(cblib, page=0)) == I
    assert append(cblib, c=cache(cblib, k=0)) == I and append(cblib, c=cache(cblib, table=0)) == I
    assert append(cblib, c=cache(cblib, page=1 << 20, width=1 << 12)) == I
    assert append(cblib, c=cache(cblib, k_stride_page=-1)) == I
    assert append(cblib, c=cache(cblib, k=DATA + 1)) == cblib.ERR_ALIGNMENT
    lib = cblib.load()
    assert lib.cb_cache_append(None, None, DATA, None, None, None) == I
    empty = heads(cblib, h=2, l=0)
    assert append(cblib, k=empty, v=empty) == cblib.OK


def decode(cblib, q=None, c=None, length=DATA, out=None, scale=0.125, cap=0.0, ws=DATA, size=1 << 40):
    q = heads(cblib, l=1) if q is None else q
    out = heads(cblib, l=1, data=DATA + (1 << 25)) if out is None else out
    c = cache(cblib) if c is None else c
    return cblib.load().cb_attention_decode(ctypes.byref(q), ctypes.byref(c), length, None, scale, cap, None,
                                            ctypes.byref(out), ws, size, None)


def test_decode_refusals(cblib):
    I = cblib.ERR_INVALID_ARG
    assert decode(cblib, length=None) == I and decode(cblib, ws=None) == I
    assert decode(cblib, q=heads(cblib, l=2)) == I and decode(cblib, q=heads(cblib, l=1, d=32)) == I
    assert decode(cblib, q=heads(cblib, l=1, h=3)) == I and decode(cblib, q=heads(cblib, l=1, b=3)) == I
    assert decode(cblib, out=heads(cblib, l=1, h=2)) == I and decode(cblib, out=heads(cblib, l=1)) == I  # the last overlaps q
    assert decode(cblib, scale=0.0) == I and decode(cblib, cap=-1.0) == I
    assert decode(cblib, ws=DATA + 16) == cblib.ERR_ALIGNMENT
    assert decode(cblib, q=heads(cblib, l=1, data=DATA + 1)) == cblib.ERR_ALIGNMENT
    wide = dict(d=136, l=1)
    assert decode(cblib, q=heads(cblib, **wide), c=cache(cblib, dk=136)) == cblib.ERR_UNSUPPORTED
    n = ctypes.c_size_t(0)
    lib = cblib.load()
    assert lib.cb_attention_decode_workspace(None, None, ctypes.byref(n)) == I
    q, c = heads(cblib, l=1), cache(cblib)
    assert lib.cb_attention_decode_workspace(ctypes.byref(q), ctypes.byref(c), None) == I


def test_packed_views_have_the_structures_layout(cblib):
    import torch
    t = torch.zeros(3, 5, 4, 16, dtype=torch.bfloat16)[:, 1:, ::2, 8:]
    want = cblib.CbHeads(t.data_ptr(), 3, 4, 2, 8, *t.stride()[:3], cblib.DTYPE_BF16)
    got = cblib.CbHeads.from_buffer_copy(cblib.heads(t))
    assert all(getattr(got, n) == getattr(want, n) for n, _ in cblib.CbHeads._fields_)
    assert len(cblib.heads(t)) == ctypes.sizeof(cblib.CbHeads)
    packed = cblib.Score(0.5, 2.0, causal=True, q_offset=-3).view(1, 2, 3, 4)
    assert len(packed) == ctypes.sizeof(cblib.CbScore)
    got = cblib.CbScore.from_buffer_copy(packed)
    assert (got.scale, got.softcap, got.causal, got.q_offset, got.slopes, got.doc_k) == (0.5, 2.0, 1, -3, None, None)


def test_binding_checks_index_tensors(cblib):
    import torch
    s = cblib.Score(0.1, kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        s.view(2, 4, 4, 4)
    with pytest.raises(ValueError):
        cblib.heads(torch.zeros(1, 2, 3, 8).transpose(2, 3))
    with pytest.raises(ValueError):
        cblib.PagedCache(torch.zeros(2, 4, 1, 8), torch.zeros(2, 4, 2, 8), torch.zeros(1, 1, dtype=torch.int32))


class OnDevice:
    """Host tensors that say they lie on a CUDA device, and a library that must not be reached."""

    def __init__(self, monkeypatch, cblib):
        import torch

        class Claims(torch.Tensor):
            def get_device(self):
                return self.claimed

        def make(*shape, dtype=torch.bfloat16, device=0):
            t = torch.zeros(*shape, dtype=dtype).as_subclass(Claims)
            t.claimed = device
            return t

        class Library:
            def __getattr__(self, name):
                def called(*args):
                    raise AssertionError(f"{name} was called")
                return called

        class Stream:
            cuda_stream = 0

        self.make, self.i32, self.f32, self.stream = make, torch.int32, torch.float32, Stream()
        monkeypatch.setattr(cblib, "_lib", Library())


@pytest.mark.parametrize("device", [-1, 1], ids=["host", "another"])
def test_binding_checks_every_tensors_device(cblib, monkeypatch, device):
    """A tensor on the host, or on another device than the others, is refused before the library is called, also
    where a stream is given."""
    on = OnDevice(monkeypatch, cblib)
    s = on.stream

    def refused(call, shapes):
        tensors = {n: on.make(*sh, dtype=dt) for n, (sh, dt) in shapes.items()}
        with pytest.raises(AssertionError, match="was called"):
            call(tensors)  # all on one device: the call goes on to the library
        for n, (sh, dt) in shapes.items():
            with pytest.raises(ValueError):
                call({**tensors, n: on.make(*sh, dtype=dt, device=device)})

    import torch
    B, h = (2, 3, 4, 64), torch.bfloat16
    refused(lambda t: cblib.attention(t["q"], t["k"], t["v"], t["out"],
                                      cblib.Score(0.1, kv_len=t["kv"], slopes=t["slopes"]), stream=s),
            {"q": (B, h), "k": (B, h), "v": (B, h), "out": (B, h), "kv": ((2,), on.i32), "slopes": ((4,), on.f32)})
    pages, table = ((5, 16, 4, 64), h), ((2, 3), on.i32)
    refused(lambda t: cblib.cache_append(t["k"], t["v"], cblib.PagedCache(t["kp"], t["vp"], t["table"]), t["pos"],
                                         count=t["count"], stream=s),
            {"k": (B, h), "v": (B, h), "kp": pages, "vp": pages, "table": table, "pos": ((2,), on.i32), "count": ((2,), on.i32)})
    refused(lambda t: cblib.attention_decode(t["q"], cblib.PagedCache(t["kp"], t["vp"], t["table"]), t["n"], t["out"],
                                             t["ws"], 0.1, slopes=t["slopes"], first=t["first"], stream=s),
            {"q": ((2, 4, 64), h), "kp": pages, "vp": pages, "table": table, "n": ((2,), on.i32), "out": ((2, 4, 64), h),
             "ws": ((4096,), torch.uint8), "slopes": ((4,), on.f32), "first": ((2,), on.i32)})


def test_binding_wants_a_contiguous_workspace(cblib, monkeypatch):
    import torch
    on = OnDevice(monkeypatch, cblib)
    cache = cblib.PagedCache(on.make(5, 16, 4, 64), on.make(5, 16, 4, 64), on.make(2, 3, dtype=on.i32))
    q, n, ws = on.make(2, 4, 64), on.make(2, dtype=on.i32), on.make(4096, 2, dtype=torch.uint8)[:, 0]
    ws.claimed = 0
    with pytest.raises(ValueError):
        cblib.attention_decode(q, cache, n, on.make(2, 4, 64), ws, 0.1, stream=on.stream)


FAR, BYTES = 1 << 26, 10 * 16 * 2 * 64 * 2  # BYTES: of the cache's key or value pages


def test_append_refuses_tokens_that_lie_in_the_pages(cblib):
    k, v = heads(cblib, h=2, data=DATA + FAR), heads(cblib, h=2, data=DATA + 2 * FAR)
    for at in (DATA, DATA + BYTES - 2, DATA - 2, DATA + (1 << 24) + 4096):
        new = heads(cblib, h=2, data=at)
        assert append(cblib, k=new, v=v) == cblib.ERR_INVALID_ARG, at
        assert append(cblib, k=k, v=new) == cblib.ERR_INVALID_ARG, at


def test_decode_refuses_an_output_in_the_pages(cblib):
    """With no workspace: what is not refused for its place is refused for that, and nothing is launched."""
    page = 16 * 2 * 64  # elements of a page; strided ones have the next three pages' room free
    q, wide = heads(cblib, l=1, data=DATA + FAR), cache(cblib, k_stride_page=4 * page, v_stride_page=4 * page)
    wide.v = DATA + 2 * page
    behind = DATA + 2 * (5 * 4 * page + 2 * page)  # behind the values of page 5

    def status(at, c=None):
        return decode(cblib, q=q, c=c, out=heads(cblib, l=1, data=at), size=0)

    for at in (DATA, DATA + BYTES - 2, DATA + (1 << 24) + 4096):
        assert status(at) == cblib.ERR_INVALID_ARG, at
    assert status(behind - 2, wide) == cblib.ERR_INVALID_ARG
    assert status(DATA + BYTES) != cblib.ERR_INVALID_ARG and status(behind, wide) != cblib.ERR_INVALID_ARG
