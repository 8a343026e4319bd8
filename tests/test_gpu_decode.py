"""The paged cache on the GPU: cb_cache_append bit for bit, cb_attention_decode against the definition in 64 bits."""
import pytest
import torch

import attention_ref as ref
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def paged(lens, page, Hkv, dk, dv, dtype, seed=0, spare=2, poison=float("nan")):
    """A cache with each sequence's tokens at scattered pages; every other slot holds `poison`, every other
    table entry -1."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    count = sum(need) + spare
    order = torch.randperm(count, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
    k = torch.full((count, page, Hkv, dk), poison)
    v = torch.full((count, page, Hkv, dv), poison)
    for b, n in enumerate(lens):
        for p in range(need[b]):
            at = order.pop()
            table[b, p] = at
            m = min(page, n - p * page)
            k[at, :m] = torch.randn(m, Hkv, dk, generator=g)
            v[at, :m] = torch.randn(m, Hkv, dv, generator=g)
    return k.to("cuda", dtype), v.to("cuda", dtype), table.cuda()


def run(q, k, v, table, lens, out=None, stream=None, **kw):
    cache = cb.PagedCache(k, v, table)
    ws = torch.empty(cb.attention_decode_workspace(q, cache), dtype=torch.uint8, device="cuda").fill_(255)
    if out is None:
        out = torch.full((*q.shape[:2], v.shape[3]), float("nan"), dtype=q.dtype, device="cuda")
    cb.attention_decode(q, cache, lens, out, ws, stream=stream, **kw)
    return out


def finite(v):
    return torch.where(torch.isfinite(v), v, torch.zeros_like(v))


CASES = [  # lens, page, Hq, Hkv, dk, dv
    ([1], 16, 1, 1, 64, 64), ([421], 16, 8, 2, 64, 64), ([0, 5, 64, 65, 63, 0], 16, 4, 4, 128, 128),
    ([1000, 1, 333], 20, 8, 1, 128, 128), ([100] * 5, 7, 10, 2, 96, 96), ([5000], 64, 16, 1, 64, 128),
    ([300, 200], 1, 6, 6, 32, 64), ([130] * 33, 128, 4, 2, 40, 72), ([20000, 3], 32, 4, 1, 128, 128),
    ([77, 78, 79], 24, 40, 2, 64, 64), ([0, 0], 16, 2, 2, 64, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", ["plain", "cap", "bias", "first", "all"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_definition(gpu, case, name, dtype):
    lens, page, Hq, Hkv, dk, dv = CASES[case]
    k, v, table = paged(lens, page, Hkv, dk, dv, dtype, seed=case)
    B = len(lens)
    q = (ref.randn(B, Hq, dk, seed=case + 50, dtype=F32, device="cuda") * 3).to(dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = {"scale": dk ** -0.5}
    if name in ("cap", "all"):
        kw["softcap"] = 5.0
    if name in ("bias", "all"):
        kw["slopes"] = ref.alibi_slopes(Hq, "cuda")
    if name in ("first", "all"):  # the last sequence starts past its end
        kw["first"] = torch.tensor([x // 3 if b + 1 < B or B == 1 else x + 1 for b, x in enumerate(lens)],
                                   dtype=torch.int32, device="cuda")
    out = run(q, k, v, table, n, **kw)
    sync_check()
    ref.check(out, ref.decode(q, k, v, table, n, **kw), finite(v), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(7, 5), (33, 128), (64, 64)], ids=str)
def test_odd_dims_and_strides(gpu, dims, dtype):
    """Head-major pages, gaps between slots, data off 16-byte boundaries."""
    dk, dv = dims
    lens, page, Hq, Hkv = [90, 17], 20, 6, 3
    k, v, table = paged(lens, page, Hkv, dk, dv, dtype, seed=3)
    ks = torch.zeros(k.shape[0], Hkv, page, dk + 3, dtype=dtype, device="cuda")[..., 1:dk + 1].transpose(1, 2)
    vs = torch.zeros(k.shape[0], page, Hkv, dv + 1, dtype=dtype, device="cuda")[..., 1:]
    ks.copy_(k), vs.copy_(v)
    q = ref.randn(2, Hq, dk + 2, seed=5, dtype=dtype, device="cuda")[..., 1:dk + 1]
    buf = torch.full((2, Hq + 2, dv + 1), 77.0, dtype=dtype, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    run(q, ks, vs, table, n, out=buf[:, 1:-1, 1:], scale=dk ** -0.5)
    sync_check()
    ref.check(buf[:, 1:-1, 1:], ref.decode(q, k, v, table, n, dk ** -0.5), finite(v), dtype)
    assert (buf[:, 0] == 77).all() and (buf[:, -1] == 77).all() and (buf[..., 0] == 77).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_same_bits_twice(gpu, dtype):
    lens = [9000, 10, 4000]
    k, v, table = paged(lens, 16, 2, 64, 64, dtype, seed=1)
    q = ref.randn(3, 8, 64, seed=2, dtype=dtype, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    a = run(q, k, v, table, n, scale=0.125)
    torch.cuda.synchronize()
    b = run(q, k, v, table, n, scale=0.125, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_bad_pages_are_reported_not_followed(gpu):
    lens = [100, 100]
    k, v, table = paged(lens, 16, 2, 64, 64, BF16, seed=4)
    q = ref.randn(2, 4, 64, seed=2, dtype=BF16, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    good = run(q, k, v, table, n, scale=0.125)
    assert cb.get_device_error() == cb.OK
    table[0, 2] = k.shape[0] + 5
    out = run(q, k, v, table, n, scale=0.125)
    assert cb.get_device_error() == cb.ERR_INVALID_ARG
    assert cb.get_device_error() == cb.OK
    assert torch.equal(out[1], good[1]) and torch.isfinite(out.float()).all()
    keep = torch.tensor([j for j in range(100) if not 32 <= j < 48])
    rows = table[0].cpu().long()[keep // 16]
    kk, vv = k.cpu()[rows, keep % 16].double(), v.cpu()[rows, keep % 16].double()
    want = torch.stack([torch.softmax(kk[:, h // 2] @ q[0, h].cpu().double() * 0.125, 0) @ vv[:, h // 2] for h in range(4)])
    ref.check(out[0], want, finite(v), BF16)


def test_lengths_past_the_table_are_clamped(gpu):
    k, v, table = paged([48], 16, 1, 64, 64, F32, seed=6)
    q = ref.randn(1, 2, 64, seed=2, dtype=F32, device="cuda")
    table = table[:, :3].contiguous()
    got = run(q, k, v, table, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"), scale=0.125)
    sync_check()
    ref.check(got, ref.decode(q, k, v, table, [48], 0.125), finite(v), F32)


def test_wide_offsets(gpu):
    """Pages more than 2^31 elements past the first."""
    page, H, D = 16, 2, 64
    stride = (1 << 30) + 4096
    flat = torch.empty(3 * stride + page * H * 2 * D, dtype=BF16, device="cuda")
    kw = flat.as_strided((4, page, H, D), (stride, H * 2 * D, 2 * D, 1))
    vw = flat.as_strided((4, page, H, D), (stride, H * 2 * D, 2 * D, 1), D)
    k, v, table = paged([55], page, H, D, D, BF16, seed=6, spare=0)
    q = ref.randn(1, 4, D, seed=2, dtype=BF16, device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.arange(55)
    rows = table[0].cpu().long()[at // page].cuda()
    cb.cache_append(k[rows, (at % page).cuda()][None].contiguous(), v[rows, (at % page).cuda()][None].contiguous(),
                    cb.PagedCache(kw, vw, table), pos)
    n = torch.tensor([55], dtype=torch.int32, device="cuda")
    out = run(q, kw, vw, table, n, scale=0.125)
    sync_check()
    ref.check(out, ref.decode(q, k, v, table, n, 0.125), finite(v), BF16)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 1, 16, 1, 64, 64, 0), (3, 50, 16, 2, 64, 128, 7), (5, 77, 20, 4, 32, 64, 13),
                                  (2, 33, 1, 3, 7, 5, 0), (40, 1, 64, 8, 128, 128, 63), (1, 700, 128, 2, 40, 72, 100)], ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_append(gpu, case, ragged, dtype):
    """Bit for bit, from slices of a projection's output; every other slot keeps its bits."""
    B, T, page, H, dk, dv, past = case
    width = (past + T + page - 1) // page
    g = torch.Generator().manual_seed(T)
    table = torch.randperm(B * width + 3, generator=g)[:B * width].reshape(B, width).to(torch.int32).cuda()
    k = ref.randn(B * width + 3, page, H, dk, seed=1, dtype=dtype, device="cuda")
    v = ref.randn(B * width + 3, page, H, dv, seed=2, dtype=dtype, device="cuda")
    row = ref.randn(B, T, H * (dk + dv), seed=3, dtype=dtype, device="cuda")
    row[0, 0, 0] = float("nan")
    kn, vn = torch.split(row, [H * dk, H * dv], dim=-1)
    kn, vn = kn.unflatten(-1, (H, dk)), vn.unflatten(-1, (H, dv))
    counts = [(b * 11) % (T + 1) for b in range(B)] if ragged else [T] * B
    pos = torch.tensor([past - b % 2 if past else 0 for b in range(B)], dtype=torch.int32, device="cuda")
    want_k, want_v = k.clone(), v.clone()
    for b in range(B):
        for t in range(counts[b]):
            at = int(pos[b]) + t
            want_k[int(table[b, at // page]), at % page] = kn[b, t]
            want_v[int(table[b, at // page]), at % page] = vn[b, t]
    cb.cache_append(kn, vn, cb.PagedCache(k, v, table), pos,
                    count=torch.tensor(counts, dtype=torch.int32, device="cuda") if ragged else None)
    sync_check()
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(k.view(bits), want_k.view(bits)) and torch.equal(v.view(bits), want_v.view(bits))


def test_append_refuses_bad_places(gpu):
    k, v, table = paged([40], 16, 1, 64, 64, F32, seed=1, poison=0.0)
    before = k.clone()
    new = torch.ones(1, 2, 1, 64, device="cuda")
    for at in (-1, 16 * table.shape[1] - 1):
        cb.cache_append(new, new, cb.PagedCache(k, v, table), torch.tensor([at], dtype=torch.int32, device="cuda"))
        assert cb.get_device_error() == cb.ERR_INVALID_ARG
    changed = (k != before).any(-1).any(-1).nonzero().tolist()
    assert changed == [[int(table[0, 0]), 0]]  # position -1 + 1 is token 0; the table's last page is -1
    assert cb.get_device_error() == cb.OK


@pytest.mark.parametrize("lens", [[40, 0, 129], [3000, 1, 2100, 777]], ids=["whole", "runs"])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (20, 2)], ids=["one_head", "ten_heads"])
@pytest.mark.parametrize("dk,dv", [(96, 96), (72, 96), (88, 80), (96, 128), (128, 72), (96, 64)])
def test_dims_between_64_and_128(gpu, dk, dv, Hq, Hkv, lens):
    """The pads of rows shorter than the kernel's are zeros, whatever the pages hold beyond a sequence."""
    k, v, table = paged(lens, 16, Hkv, dk, dv, BF16, seed=dk + dv)
    if len(lens) == 4:  # a table that could name far more: too many tiles for whole items
        table = torch.cat([table, torch.full((4, 3000), -1, dtype=torch.int32, device="cuda")], 1)
    q = (ref.randn(len(lens), Hq, dk, seed=5, dtype=F32, device="cuda") * 2).to(BF16)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = run(q, k, v, table, n, scale=dk ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k, v, table, n, dk ** -0.5), finite(v), BF16)


def test_append_from_another_layers_pages(gpu):
    """Two layers' pages in turn in one buffer: one layer's tokens, as a view with the pages' strides, are appended
    to the other's."""
    P, page, H, D = 6, 16, 2, 64
    g = torch.Generator().manual_seed(1)
    buf = torch.randn(P, 4, page, H, D, generator=g).to("cuda", BF16)  # k and v of layer 0, then of layer 1
    want = buf.clone()
    want[[3, 1], :2] = buf[[0, 1], 2:]
    table = torch.tensor([[3], [1]], dtype=torch.int32, device="cuda")
    cb.cache_append(buf[:2, 2], buf[:2, 3], cb.PagedCache(buf[:, 0], buf[:, 1], table),
                    torch.zeros(2, dtype=torch.int32, device="cuda"))
    sync_check()
    assert torch.equal(buf, want)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (7, 5)], ids=str)
def test_lengths_near_the_largest_int(gpu, dims, dtype):
    """A table of 2^31 - 2 tokens (one page, named everywhere), of which the query sees the last hundred."""
    page, pages = 99962, 21483
    room = page * pages
    assert room == 2 ** 31 - 2
    k = ref.randn(1, page, 1, dims[0], seed=1, dtype=dtype, device="cuda")
    v = ref.randn(1, page, 1, dims[1], seed=2, dtype=dtype, device="cuda")
    table = torch.zeros(1, pages, dtype=torch.int32, device="cuda")
    q = ref.randn(1, 4, dims[0], seed=3, dtype=dtype, device="cuda")
    kw = {"scale": dims[0] ** -0.5, "slopes": ref.alibi_slopes(4, "cuda")}
    n = torch.tensor([room], dtype=torch.int32, device="cuda")
    got = run(q, k, v, table, n, first=n - 100, **kw)
    sync_check()
    last = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    want = ref.decode(q, k[:, -100:], v[:, -100:], last, torch.tensor([100]), **kw)
    ref.check(got, want, v, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (7, 5)], ids=str)
@pytest.mark.parametrize("wide", [False, True], ids=["tight_table", "wide_table"])
@pytest.mark.parametrize("B", [129, 300, 1000])
def test_more_sequences_than_threads(gpu, B, wide, dims, dtype):
    """Several sequences per thread where the prefix over the lengths is taken; empty ones among them."""
    lens = [(37 * b) % 150 if b % 5 else 0 for b in range(B)]
    k, v, table = paged(lens, 16, 1, *dims, dtype, seed=7)
    if wide:
        table = torch.cat([table, torch.full((B, 3000), -1, dtype=torch.int32, device="cuda")], 1)
    q = ref.randn(B, 2, dims[0], seed=8, dtype=dtype, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = run(q, k, v, table, n, scale=dims[0] ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k.cpu(), v.cpu(), table.cpu(), lens, dims[0] ** -0.5), finite(v), dtype)


@pytest.mark.parametrize("lens", [[40, 0, 129], [3000, 1, 2100, 777]], ids=["whole", "runs"])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2), (20, 2)], ids=["one_head", "three_heads", "ten_heads"])
@pytest.mark.parametrize("dk,dv", [(96, 96), (72, 100), (36, 40), (128, 72), (96, 64)])
def test_fp32_dims_between_the_kernels(gpu, dk, dv, Hq, Hkv, lens):
    """test_dims_between_64_and_128 for fp32, and for fewer than 64."""
    k, v, table = paged(lens, 16, Hkv, dk, dv, F32, seed=dk + dv)
    if len(lens) == 4:
        table = torch.cat([table, torch.full((4, 3000), -1, dtype=torch.int32, device="cuda")], 1)
    q = ref.randn(len(lens), Hq, dk, seed=5, dtype=F32, device="cuda") * 2
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = run(q, k, v, table, n, scale=dk ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k, v, table, n, dk ** -0.5), finite(v), F32)
