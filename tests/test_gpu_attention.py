"""cb_attention on the GPU against the definition in 64 bits: head layouts, lengths from one token on, odd sizes,
strides, every mask, masks that leave a row empty, and what lies in masked places."""
import pytest
import torch

import attention_ref as ref
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# B, Lq, Lk, Hq, Hkv, Dk, Dv
SHAPES = [(1, 1, 1, 1, 1, 8, 8), (2, 49, 49, 3, 3, 64, 64), (1, 130, 257, 4, 2, 32, 64), (2, 128, 128, 2, 1, 128, 128),
          (1, 1, 1000, 8, 1, 128, 128), (1, 300, 300, 2, 2, 40, 72), (3, 127, 129, 5, 1, 96, 96), (1, 513, 640, 2, 2, 64, 128),
          (1, 260, 70, 2, 1, 128, 64), (2, 400, 400, 4, 4, 32, 64), (1, 16, 2049, 6, 2, 64, 64), (1, 5, 0, 2, 1, 64, 64)]
RULES = ["full", "causal", "prefix", "kv_len", "docs", "cap", "bias", "all"]


def make(shape, dtype, seed=0, spread=3.0, device="cuda"):
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    q = ref.randn(B, Lq, Hq, Dk, seed=seed, dtype=torch.float32, device=device) * spread
    return (q.to(dtype), ref.randn(B, Lk, Hkv, Dk, seed=seed + 1, dtype=dtype, device=device),
            ref.randn(B, Lk, Hkv, Dv, seed=seed + 2, dtype=dtype, device=device))


def rule(name, shape, device="cuda"):
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    kw = {"scale": Dk ** -0.5}
    every = name == "all"
    if name in ("causal", "prefix") or every:
        kw.update(causal=True, q_offset=Lk - Lq)
    if name == "prefix" or every:
        kw["prefix_len"] = torch.tensor([(Lk // 3 + 37 * b) for b in range(B)], dtype=torch.int32, device=device)
    if name == "kv_len" or every:  # the first sequence of several has no key at all
        kw["kv_len"] = torch.tensor([Lk * (b if B > 1 else 2) // max(B, 3) for b in range(B)], dtype=torch.int32, device=device)
    if name == "docs" or every:  # unsorted ids, padding, documents without a key
        g = torch.Generator().manual_seed(Lq + Lk)
        kw["doc_q"] = (torch.randint(-1, 4, (B, Lq), generator=g).repeat_interleave(37, 1)[:, :Lq]).to(torch.int32).to(device)
        kw["doc_k"] = (torch.randint(-1, 3, (B, Lk), generator=g).repeat_interleave(61, 1)[:, :Lk]).to(torch.int32).to(device)
        kw["doc_q"], kw["doc_k"] = kw["doc_q"].contiguous(), kw["doc_k"].contiguous()
    if name == "cap" or every:
        kw["softcap"] = 5.0
    if name == "bias" or every:
        kw["slopes"] = ref.alibi_slopes(Hq, device)
    return kw


def run(q, k, v, kw, out=None, stream=None):
    if out is None:
        out = torch.full((*q.shape[:3], v.shape[3]), float("nan"), dtype=q.dtype, device=q.device)
    cb.attention(q, k, v, out, cb.Score(**kw), stream=stream)
    return out


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_definition(gpu, shape, name, dtype):
    q, k, v = make(shape, dtype)
    kw = rule(name, shape)
    out = run(q, k, v, kw)
    sync_check()
    ref.check(out, ref.attention(q, k, v, **kw), v, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(7, 5), (64, 64), (1, 1), (33, 128)], ids=str)
def test_odd_dims_and_strides(gpu, dims, dtype):
    """Head-major storage, rows with gaps, data off 16-byte boundaries; what lies around the output stays."""
    B, Lq, Lk, Hq, Hkv = 2, 70, 131, 4, 2
    dk, dv = dims
    q, k, v = make((B, Lq, Lk, Hq, Hkv, dk, dv), dtype, seed=5)
    qs = torch.zeros(B, Hq, Lq + 1, dk + 3, dtype=dtype, device="cuda")[:, :, 1:, 1:dk + 1].transpose(1, 2)
    ks = torch.zeros(B, Hkv, Lk, dk + 1, dtype=dtype, device="cuda")[..., 1:].transpose(1, 2)
    vs = torch.zeros(B, Lk, Hkv, 2 * dv + 1, dtype=dtype, device="cuda")[..., dv + 1:]
    qs.copy_(q), ks.copy_(k), vs.copy_(v)
    buf = torch.full((B, Lq, Hq + 1, dv + 2), 77.0, dtype=dtype, device="cuda")
    out = buf[:, :, 1:, 1:dv + 1]
    kw = {"scale": dk ** -0.5, "causal": True, "q_offset": Lk - Lq}
    run(qs, ks, vs, kw, out=out)
    sync_check()
    ref.check(out, ref.attention(q, k, v, **kw), v, dtype)
    assert (buf[:, :, 0] == 77).all() and (buf[..., 0] == 77).all() and (buf[..., -1] == 77).all()


def test_slices_of_one_projection(gpu):
    """q, k, v as channel slices of a projection's output, the output a slice beside them."""
    B, L, Hq, Hkv, D = 2, 200, 8, 2, 64
    row = ref.randn(B, L, (2 * Hq + 2 * Hkv) * D, seed=3, dtype=BF16, device="cuda")
    q, k, v, o = (t.unflatten(-1, (-1, D)) for t in torch.split(row, [Hq * D, Hkv * D, Hkv * D, Hq * D], dim=-1))
    want = ref.attention(q, k, v, 0.125)
    cb.attention(q, k, v, o, cb.Score(0.125))
    sync_check()
    ref.check(o, want, v, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_masked_places_do_not_matter(gpu, poison, dtype):
    """Infinities and NaN in keys and values that a query does not see leave its row as it is: past kv_len,
    in the future, in another document, in padding."""
    shape = (2, 300, 300, 4, 2, 64, 64)
    q, k, v = make(shape, dtype, seed=9)
    doc = (torch.arange(300) // 90).to(torch.int32)
    doc[280:] = -1
    doc = doc[None].expand(2, 300).contiguous().cuda()
    kw = {"scale": 0.125, "causal": True, "doc_q": doc, "doc_k": doc,
          "kv_len": torch.tensor([300, 250], dtype=torch.int32, device="cuda")}
    clean = ref.attention(q, k, v, **kw)
    k[:, 285:] = poison
    v[:, 285:] = poison
    k[1, 250:] = poison
    v[1, 250:] = poison
    v[:, 150] = poison   # seen by queries 150..179 (its document, not before it) alone
    out = run(q, k, v, kw)
    sync_check()
    got = out.cpu().double()
    seen = torch.zeros(2, 300, dtype=torch.bool)
    seen[:, 150:180] = True
    assert torch.isfinite(got[~seen]).all()
    assert not torch.isfinite(got[seen]).any()
    got[seen] = clean[seen]
    ref.check(got, clean, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_large_scores_and_late_maximum(gpu, dtype):
    """Scores of hundreds, the largest among the last keys: the running maximum moves far, exponentials of
    the first tiles vanish, and nothing overflows."""
    B, L, H, D = 1, 1024, 2, 64
    q, k, v = make((B, L, L, H, H, D, D), dtype, seed=2, spread=1.0)
    k = (k.float() * torch.linspace(0.5, 30.0, L, device="cuda")[None, :, None, None]).to(dtype)
    out = run(q, k, v, {"scale": 1.0})
    sync_check()
    got, want = out.cpu().double(), ref.attention(q, k, v, 1.0)
    # scores up to ~1000: their fp32 rounding (2^-24 * 1000 a few times) moves a weight by ~1e-3 of itself
    err = (got - want).abs().max()
    assert float(err) <= (3e-3 if dtype == F32 else 3e-3 + 2.0 ** -7) * float(v.abs().max())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_same_bits_twice_and_on_another_stream(gpu, dtype):
    shape = (2, 333, 777, 4, 2, 128, 128)
    q, k, v = make(shape, dtype, seed=4)
    kw = rule("all", shape)
    a = run(q, k, v, kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = torch.empty_like(a)
    run(q, k, v, kw, out=b, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_graph_capture(gpu):
    shape = (1, 200, 200, 4, 4, 64, 64)
    q, k, v = make(shape, BF16, seed=8)
    kw = rule("causal", shape)
    out = torch.zeros(1, 200, 4, 64, dtype=BF16, device="cuda")
    run(q, k, v, kw, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(q, k, v, kw, out=out)
    q.copy_(ref.randn(*q.shape, seed=77, dtype=BF16, device="cuda"))
    out.zero_()
    g.replay()
    sync_check()
    ref.check(out, ref.attention(q, k, v, **kw), v, BF16)


@pytest.mark.parametrize("name", RULES)
def test_more_items_than_sms(gpu, name):
    """Several rounds of work per CTA: lists, rings and accumulators pass from item to item."""
    shape = (41, 300, 300, 6, 3, 64, 64)
    q, k, v = make(shape, BF16, seed=12)
    kw = rule(name, shape)
    out = run(q, k, v, kw)
    sync_check()
    pick = [0, 1, 17, 40]
    part = {n: (t[pick] if n in ("prefix_len", "kv_len", "doc_q", "doc_k") else t) for n, t in kw.items()}
    ref.check(out[pick], ref.attention(q[pick], k[pick], v[pick], **part), v, BF16)


def test_empty_batch_and_rows(gpu):
    for shape in ((0, 4, 4, 2, 2, 64, 64), (2, 0, 4, 2, 2, 64, 64)):
        q, k, v = make(shape, BF16)
        assert run(q, k, v, {"scale": 1.0}).numel() == 0
    sync_check()


def test_wide_offsets(gpu):
    """Rows of one sequence more than 2^31 elements apart from the data pointer."""
    stride = (1 << 30) + 64
    flat = torch.empty(3 * stride + 4096, dtype=BF16, device="cuda")
    k = flat.as_strided((1, 4, 1, 64), (0, stride, 64, 1))
    v = flat.as_strided((1, 4, 1, 64), (0, stride, 64, 1), 64)
    q, k0, v0 = make((1, 4, 4, 1, 1, 64, 64), BF16, seed=1)
    k.copy_(k0), v.copy_(v0)
    out = run(q, k, v, {"scale": 0.125})
    sync_check()
    ref.check(out, ref.attention(q, k0, v0, 0.125), v0, BF16)


@pytest.mark.parametrize("poison", [False, True], ids=["clean", "poison"])
@pytest.mark.parametrize("name", ["full", "all"])
@pytest.mark.parametrize("shape", [(40, 70, 83, 10, 10, 64, 64), (24, 66, 90, 20, 4, 72, 96), (5, 201, 190, 40, 8, 128, 128),
                                   (40, 33, 40, 24, 8, 96, 128), (9, 300, 300, 12, 4, 40, 72), (3, 700, 700, 8, 8, 124, 100)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fp32_tiles(gpu, shape, name, poison):
    """Enough work that fp32 takes the tiled kernel: rows of 32, 64 and 128, heads that share a key head in one
    tile, 64, 96 and 128 values; with NaN and infinities among the values that lie past the sequences' ends."""
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    q, k, v = make(shape, F32, seed=8, spread=1.0)
    kw = rule(name, shape)
    kv = torch.tensor([Lk - 7 * b % Lk for b in range(B)], dtype=torch.int32, device="cuda")
    kw["kv_len"] = kv
    past = torch.arange(Lk, device="cuda")[None, :] >= kv[:, None]
    if poison:
        k[past], v[past] = float("nan"), float("inf")
    out = run(q, k, v, kw)
    sync_check()
    kd, vd = (t.double().masked_fill(past[..., None, None], 0.).repeat_interleave(Hq // Hkv, 2) for t in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q.double(), kd) * kw["scale"]
    at, j = torch.arange(Lq, device="cuda")[:, None] + kw.get("q_offset", 0), torch.arange(Lk, device="cuda")[None, :]
    if name == "all":
        s = 5.0 * torch.tanh(s / 5.0) - kw["slopes"].double()[None, :, None, None] * (at - j).abs()
    keep = ~past[:, None, None, :]
    if name == "all":
        keep = keep & ((j <= at) | (j < kw["prefix_len"][:, None, None]))[:, None]
        keep = keep & ((kw["doc_q"][:, :, None] == kw["doc_k"][:, None, :]) & (kw["doc_q"] >= 0)[:, :, None])[:, None]
    w = torch.exp((s - s.masked_fill(~keep, -1e30).amax(-1, keepdim=True)).masked_fill(~keep, float("-inf")))
    want = torch.einsum("bhij,bjhd->bihd", w / w.sum(-1, keepdim=True).clamp(min=1e-300), vd).cpu()
    ref.check(out, want, vd, F32)


@pytest.mark.parametrize("docs", [False, True], ids=["odd_tiles", "padded_tiles"])
def test_items_whose_second_tile_sees_nothing(gpu, docs):
    """Pairs of query tiles of which one has no key to visit, over one or two key tiles and many rounds: its
    queries' load is waited for before the next one is issued.  The same bits every time."""
    shape = (100, 300, 100, 4, 4, 64, 64) if not docs else (30, 500, 500, 8, 8, 64, 64)
    q, k, v = make(shape, BF16, seed=4)
    kw = {"scale": 0.125}
    if docs:
        d = torch.arange(500, device="cuda") // 130
        d[384:] = -1
        kw["doc_q"] = kw["doc_k"] = d.to(torch.int32).expand(shape[0], 500).contiguous()
    first = run(q, k, v, kw)
    for _ in range(100):
        assert torch.equal(run(q, k, v, kw).view(torch.int16), first.view(torch.int16))
    sync_check()
    pick = [0, 1, shape[0] - 1]
    part = {n: (t[pick] if n in ("doc_q", "doc_k") else t) for n, t in kw.items()}
    ref.check(first[pick], ref.attention(q[pick], k[pick], v[pick], **part), v, BF16)


LONG = [(1, 4096, 4096, 4, 2, 64, 64), (1, 1500, 2000, 2, 1, 128, 128), (3, 2, 3000, 4, 2, 64, 96), (1, 700, 900, 2, 2, 20, 36)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_visible_infinities_and_nan_stay_in_their_rows_and_dims(gpu, shape, where, poison, dtype):
    """A key that is not finite makes every row that sees it NaN; a value that is not finite only its own
    dimension, in the rows that see it. Rows that share a tile with them are as ever."""
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    q, k, v = make(shape, dtype, seed=41, spread=1.0)
    at, off, d = Lk - Lq + Lq // 3, Lk - Lq, 3
    s = torch.einsum("bihd,bjhd->bhij", q.double(), k.double().repeat_interleave(Hq // Hkv, 2)) * Dk ** -0.5
    i, j = torch.arange(Lq, device="cuda")[:, None] + off, torch.arange(Lk, device="cuda")[None, :]
    w = torch.softmax(s.masked_fill(j > i, float("-inf")), -1)
    want = torch.einsum("bhij,bjhd->bihd", w, v.double().repeat_interleave(Hq // Hkv, 2)).cpu()
    hit = torch.zeros(B, Lq, Hq, Dv, dtype=torch.bool)
    if where == "key":
        k[:, at] = poison  # with queries of both signs in every dimension: a score of NaN
        hit[:, at - off:] = True
    else:
        v[:, at, :, d] = poison
        hit[:, at - off:, :, d] = True
    got = run(q, k, v, {"scale": Dk ** -0.5, "causal": True, "q_offset": off}).cpu().double()
    sync_check()
    assert torch.isfinite(got[~hit]).all() and not torch.isfinite(got[hit]).any()
    clean = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    ref.check(torch.where(hit, want, got), want, clean, dtype)


@pytest.mark.parametrize("where", ["key", "value"])
def test_one_nan_holds_up_no_bounded_wait(gpu, where):
    """16384 queries that all see one NaN, with waits bounded at 50 ms."""
    shape = (1, 16384, 16384, 4, 1, 128, 128)
    q, k, v = make(shape, BF16, seed=42)
    kw = {"scale": 128 ** -0.5, "causal": True}
    clean = run(q, k, v, kw)
    (k if where == "key" else v)[:, 0, :, 5] = float("nan")
    with cb.tuning("CB_TIMEOUT_MS", "50"):
        got = run(q, k, v, kw)
        sync_check()
    if where == "key":
        assert torch.isnan(got).all()
    else:
        assert torch.isnan(got[..., 5]).all()
        rest = torch.arange(128, device="cuda") != 5
        assert torch.equal(got[..., rest], clean[..., rest])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_padding_with_nan_in_every_tile(gpu, dtype):
    """Padding tokens that hold NaN among every 32 keys: no row's tiled sum stands, and each comes out right."""
    shape = (1, 600, 600, 2, 1, 64, 64)
    q, k, v = make(shape, dtype, seed=43)
    doc = (torch.arange(600, device="cuda") // 200).to(torch.int32)
    doc[::32] = -1
    doc = doc[None].contiguous()
    kw = {"scale": 0.125, "doc_q": doc, "doc_k": doc}
    want = ref.attention(q, k, v, **kw)
    k[:, ::32], v[:, ::32] = float("nan"), float("nan")
    out = run(q, k, v, kw)
    sync_check()
    ref.check(out, want, torch.where(torch.isfinite(v), v, torch.zeros_like(v)), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("nan", [False, True], ids=["finite", "one_nan"])
def test_large_values_under_rising_scores(gpu, nan, dtype):
    """Scores that rise by 2^40 from the first tiles to the last, over values of 1e30: sums relative to the first
    tiles' maximum would overflow. With a visible NaN in one dimension the others stay finite all the same."""
    L, D = 1024, 64
    q = torch.zeros(1, L, 1, D, device="cuda", dtype=dtype)
    k = torch.zeros(1, L, 1, D, device="cuda", dtype=dtype)
    q[..., 0] = 8
    k[..., 0] = (torch.linspace(0, 28, L, device="cuda") / 8)[None, :, None].to(dtype)
    v = (ref.randn(1, L, 1, D, seed=44, dtype=F32, device="cuda") * 1e30).to(dtype)
    want = ref.attention(q, k, v, 1.0)
    big = v.clone()
    if nan:
        v[0, 900, 0, 7] = float("nan")
    got = run(q, k, v, {"scale": 1.0}).cpu().double()
    sync_check()
    if nan:
        assert torch.isnan(got[..., 7]).all()
        got[..., 7] = want[..., 7]
    ref.check(got, want, big, dtype)


@pytest.mark.parametrize("sorted_ids", [True, False], ids=["sorted", "mixed"])
def test_documents_over_more_keys_than_kept_ranges(gpu, sorted_ids):
    """70000 keys: more key tiles than whose document ranges are kept at once."""
    B, Lq, Lk, H, D = 1, 300, 70000, 2, 64
    q, k, v = make((B, Lq, Lk, H, 1, D, D), BF16, seed=6, spread=1.0)
    j = torch.arange(Lk, device="cuda")
    doc_k = j // 997 if sorted_ids else (j // 128 * 7919) % 71
    doc_k = torch.where(j % 1009 == 5, -1, doc_k).to(torch.int32)[None].contiguous()
    doc_q = (torch.arange(Lq, device="cuda") // 50 * 11).to(torch.int32)[None].contiguous()
    doc_q[0, 120:130] = -1
    kw = {"scale": 0.125, "doc_q": doc_q, "doc_k": doc_k, "kv_len": torch.tensor([69990], dtype=torch.int32, device="cuda")}
    out = run(q, k, v, kw)
    sync_check()
    s = torch.einsum("ihd,jd->hij", q[0].double(), k[0, :, 0].double()) * 0.125
    keep = (doc_q[0][:, None] == doc_k[0][None, :]) & (doc_q[0] >= 0)[:, None] & (j < 69990)[None, :]
    w = torch.exp(s - s.masked_fill(~keep, -1e30).amax(-1, keepdim=True)).masked_fill(~keep, 0.0)
    want = torch.einsum("hij,jd->ihd", w / w.sum(-1, keepdim=True).clamp(min=1e-300), v[0, :, 0].double())
    ref.check(out[0], want.cpu(), v, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 400, 400, 4, 2, 64, 64), (2, 3, 500, 4, 2, 64, 128), (4, 260, 300, 4, 1, 128, 128)],
                         ids=lambda s: "x".join(map(str, s)))
def test_orders_and_broadcast_inputs(gpu, shape, dtype):
    """Whole 16-byte pieces in other orders than [B, L, H, D]: head-major, sequence-major, keys and values that
    all sequences or all key heads share (strides of zero)."""
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    q, k, v = make(shape, dtype, seed=31)
    kw = {"scale": Dk ** -0.5, "causal": True, "q_offset": Lk - Lq}
    want = run(q, k, v, kw)
    heads_first = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    out = torch.full((B, Hq, Lq, Dv), float("nan"), dtype=dtype, device="cuda").transpose(1, 2)
    assert torch.equal(run(*heads_first, kw, out=out), want)
    rows_first = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    out = torch.full((Lq, B, Hq, Dv), float("nan"), dtype=dtype, device="cuda").transpose(0, 1)
    assert torch.equal(run(*rows_first, kw, out=out), want)
    for wide, narrow in (((B, Lk, Hkv), (1, Lk, Hkv)), ((B, Lk, Hkv), (B, Lk, 1))):
        ke, ve = (t[:narrow[0], :, :narrow[2]].expand(*wide, -1) for t in (k, v))
        assert torch.equal(run(q, ke, ve, kw), run(q, ke.contiguous(), ve.contiguous(), kw))
    sync_check()


@pytest.mark.parametrize("Lk", [1, 130, 400])
@pytest.mark.parametrize("case", ["offset", "lengths", "documents"])
def test_runs_of_items_without_a_key(gpu, case, Lk):
    """Many rounds of work per CTA in which most items see no key, several in a row: the next item's keys are not
    waited for while the last one's output is still to come."""
    shape = (45, 450, Lk, 16, 2, 64, 64)
    B, Lq, _, Hq, Hkv, D, _ = shape
    q, k, v = make(shape, BF16, seed=51)
    kw = {"scale": 0.125}
    i, j = torch.arange(Lq, device="cuda")[:, None], torch.arange(Lk, device="cuda")[None, :]
    if case == "offset":  # the last queries alone see keys
        kw.update(causal=True, q_offset=-(Lq - 3))
        keep = (j <= i + kw["q_offset"]).expand(B, Lq, Lk)
    elif case == "lengths":
        kw["kv_len"] = torch.tensor([Lk if b % 7 in (0, 3) else 0 for b in range(B)], dtype=torch.int32, device="cuda")
        keep = (j < kw["kv_len"][:, None, None]).expand(B, Lq, Lk)
    else:
        b = torch.arange(B, device="cuda")[:, None]
        kw["doc_q"] = ((i[:, 0] // 150)[None] + 10 * b).to(torch.int32).contiguous()
        kw["doc_k"] = torch.where(b % 5 == 2, 10 * b + j // 100, -1).to(torch.int32).contiguous()
        keep = kw["doc_q"][:, :, None] == kw["doc_k"][:, None, :]
    out = run(q, k, v, kw)
    sync_check()
    s = torch.einsum("bihd,bjhd->bhij", q.double(), k.double().repeat_interleave(Hq // Hkv, 2)) * 0.125
    w = torch.exp(s - s.amax(-1, keepdim=True)).masked_fill(~keep[:, None], 0.0)
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    ref.check(out, torch.einsum("bhij,bjhd->bihd", w, v.double().repeat_interleave(Hq // Hkv, 2)).cpu(), v, BF16)


THREADS = """
import sys, threading
sys.path.insert(0, {root!r})
import torch
from conv_bn_activation_gb300 import binding as cb

cb.load()
q = torch.randn(1, 256, 2, 64, device="cuda").to(torch.bfloat16)
sizes = [1000, 30000, 60000, 120000, 90000, 45000, 200000, 150000]
kv = [torch.randn(1, n, 2, 64, device="cuda").to(torch.bfloat16) for n in sizes]
out = [torch.empty_like(q) for n in sizes]
start = threading.Barrier(len(sizes))
failed = []

def call(i):
    start.wait()
    for x in (i, *range(len(sizes))):
        try:
            cb.attention(q, kv[x], kv[x], out[x] if x == i else torch.empty_like(q), cb.Score(0.125))
        except cb.CbError as e:
            failed.append((i, x, str(e)))

threads = [threading.Thread(target=call, args=(i,)) for i in range(len(sizes))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
assert cb.get_device_error() == cb.OK
"""


def test_first_calls_of_many_threads(gpu):
    """Calls that need different amounts of shared memory, the first ones of a process at the same time."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", THREADS.format(root=root)], capture_output=True, text=True, timeout=240)
        assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("offset", [20000, 250000, -250000])
def test_bias_over_long_distances(gpu, offset, dtype):
    """Keys that all lie far from their queries: what a bias differs by from key to key is small beside it."""
    shape = (2, 300, 384, 8, 8, 64, 64)
    q, k, v = make(shape, dtype, seed=81)
    kw = {"scale": 0.125, "slopes": ref.alibi_slopes(8, "cuda"), "q_offset": offset}
    out = run(q, k, v, kw)
    sync_check()
    s = torch.einsum("bihd,bjhd->bhij", q.double(), k.double()) * 0.125
    i, j = torch.arange(300, device="cuda")[:, None] + offset, torch.arange(384, device="cuda")[None, :]
    w = torch.softmax(s - kw["slopes"].double()[None, :, None, None] * (i - j).abs(), -1)
    want = torch.einsum("bhij,bjhd->bihd", w, v.double()).cpu()
    # scores of up to 125000 hold no more than 2^-7 of themselves: the weights carry that, rounded once, at worst
    worst = 2.0 ** -24 * 0.5 * abs(offset) * 1.4427
    err = (out.cpu().double() - want).abs().max()
    assert float(err) <= worst * float(v.abs().max()) + float(ref.bound(want, v.cpu().double(), dtype).max())
