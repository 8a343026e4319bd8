"""The 4-bit cache on the GPU: tokens stored bit for bit and read back, attention over it against the definition in
64 bits."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def pages4(count, page, H, dk, dv, tokens_first=False):
    """Pages whose rows nothing has stored: codes of ones, scales NaN."""
    out = []
    for dim in (dk, dv):
        for width, dtype, fill in (((dim + 1) // 2, torch.uint8, 255), (ref4.scales_per_row(dim), BF16, float("nan"))):
            shape = (count, page, H, width) if tokens_first else (count, H, page, width)
            t = torch.full(shape, fill, dtype=dtype, device="cuda")
            out.append(t if tokens_first else t.transpose(1, 2))
    return out


def filled(lens, page, H, dk, dv, seed=0, spare=2, tokens_first=False, wide=0):
    """A cache with each sequence's tokens at scattered pages; every other slot is as pages4 leaves it, every other
    table entry -1.  Also the values [pages, page, H, dim] (0 elsewhere)."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    count = sum(need) + spare
    order = torch.randperm(count, generator=g).tolist()
    table = torch.full((len(lens), max(need + [1]) + 1 + wide), -1, dtype=torch.int32)
    parts = pages4(count, page, H, dk, dv, tokens_first)
    host = [t.cpu() for t in parts]
    for b, n in enumerate(lens):
        for p in range(need[b]):
            at = order.pop()
            table[b, p] = at
            m = min(page, n - p * page)
            for i, dim in enumerate((dk, dv)):
                host[2 * i][at, :m], host[2 * i + 1][at, :m] = ref4.store(torch.randn(m, H, dim, generator=g).to(BF16))
    for t, h in zip(parts, host):
        t.copy_(h)
    k, v = (torch.nan_to_num(ref4.values(host[2 * i], host[2 * i + 1], dim)) for i, dim in enumerate((dk, dv)))
    return cb.PagedCache4(*parts, table.cuda(), dim_k=dk, dim_v=dv), k, v


def run(q, cache, lens, out=None, stream=None, **kw):
    ws = torch.empty(cb.attention_decode4_workspace(q, cache), dtype=torch.uint8, device="cuda").fill_(255)
    if out is None:
        out = torch.full((*q.shape[:2], cache.view.dim_v), float("nan"), dtype=q.dtype, device="cuda")
    cb.attention_decode4(q, cache, lens, out, ws, stream=stream, **kw)
    return out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append
@DTYPES
@pytest.mark.parametrize("tokens_first", [False, True], ids=["head_major", "token_major"])
@pytest.mark.parametrize("ragged", [False, True], ids=["all", "ragged"])
@pytest.mark.parametrize("case", [(1, 1, 16, 1, 64, 64, 0), (3, 50, 16, 2, 64, 128, 7), (5, 77, 20, 4, 32, 64, 13), (2, 33, 1, 3, 7, 5, 0),
                                  (40, 1, 64, 8, 128, 128, 63), (1, 700, 128, 2, 40, 72, 100), (2, 90, 7, 2, 96, 33, 3),
                                  (1, 5, 16, 2, 1, 128, 0), (3, 11, 32, 1, 80, 112, 31)], ids=str)
def test_append_and_read(gpu, case, ragged, tokens_first, dtype):
    """Bit for bit, from slices of a projection's output; every other row keeps its bits; what is read back is what
    was stored, and rows behind the counts keep what they hold."""
    B, T, page, H, dk, dv, past = case
    width = (past + T + page - 1) // page
    g = torch.Generator().manual_seed(T)
    table = torch.randperm(B * width + 3, generator=g)[:B * width].reshape(B, width).to(torch.int32)
    parts = pages4(B * width + 3, page, H, dk, dv, tokens_first)
    row = ref.randn(B, T, H * (dk + dv), seed=3, dtype=F32, device="cuda") * torch.logspace(-3, 3, T, device="cuda")[None, :, None]
    row = row.to(dtype)
    row[0, 0, 0], row[-1, -1, -1] = float("nan"), float("-inf")
    kn, vn = torch.split(row, [H * dk, H * dv], dim=-1)
    kn, vn = kn.unflatten(-1, (H, dk)), vn.unflatten(-1, (H, dv))
    counts = [(b * 11) % (T + 1) for b in range(B)] if ragged else [T] * B
    pos = [past - b % 2 if past else 0 for b in range(B)]
    want = [t.cpu().clone() for t in parts]
    for i, x in enumerate((kn, vn)):
        codes, scales = ref4.store(x)
        for b in range(B):
            for t in range(counts[b]):
                page_at, slot = int(table[b, (pos[b] + t) // page]), (pos[b] + t) % page
                want[2 * i][page_at, slot], want[2 * i + 1][page_at, slot] = codes[b, t], scales[b, t]
    cache = cb.PagedCache4(*parts, table.cuda(), dim_k=dk, dim_v=dv)
    count = ints(counts) if ragged else None
    cb.cache4_append(kn, vn, cache, ints(pos), count=count)
    sync_check()
    for got, w in zip(parts, want):
        bits = torch.uint8 if got.dtype == torch.uint8 else torch.int16
        assert torch.equal(got.cpu().contiguous().view(bits), w.contiguous().view(bits))
    for out_type in (F32, BF16):
        out = [torch.full((B, T, H, d), 7.0, dtype=out_type, device="cuda") for d in (dk, dv)]
        cb.cache4_read(cache, *out, first=ints(pos), count=count)
        sync_check()
        for got, x in zip(out, (kn, vn)):
            stored = ref4.values(*ref4.store(x), x.shape[-1]).to(out_type)
            for b in range(B):
                assert torch.equal(torch.nan_to_num(got[b, :counts[b]].cpu().float(), 99.0), torch.nan_to_num(stored[b, :counts[b]].float(), 99.0))
                assert (got[b, counts[b]:] == 7).all()


@DTYPES
def test_borders_of_the_codes(gpu, dtype):
    """Elements at and next to the borders of two codes, maxima at and next to the borders of two scales, the smallest
    and the largest numbers, zeros of either sign."""
    g = torch.Generator().manual_seed(1)
    H, dim = 1, 128
    rows = []
    for e in (-149, -140, -134, -133, -132, -128, -126, -120, -70, -64, -63, -20, 0, 3, 60, 120):
        s = torch.ldexp(torch.tensor(1.0 + int(torch.randint(0, 128, (1,), generator=g)) / 128, dtype=torch.float64), torch.tensor(e))
        k = torch.randint(-7, 7, (dim,), generator=g).double() + 0.5
        x = k * s
        x[::32] = 7 * s  # the scale is s
        for step in (0, 1, -1):  # at the border, and one step of fp32 beside it
            y = x.float()
            bits = y.view(torch.int32) + step * ((torch.arange(dim) % 32 != 0) & (y != 0)).int()
            rows.append(bits.view(F32))
    for top in (7.0, 7 * 1.00390625, 7 * 1.01171875, 3.0, 1.0, 6.999999, 7.027344):  # 7 (1 + odd / 256): ties of the scale
        for step in (-1, 0, 1):
            y = torch.randn(dim, generator=g).clamp(-0.9, 0.9)
            y[5::32] = (torch.tensor([top]).view(torch.int32) + step).view(F32)
            rows.append(y)
    rows += [torch.zeros(dim), -torch.zeros(dim), torch.full((dim,), 3.3e38), torch.full((dim,), -1e-45)]
    x = torch.stack(rows)[:, None, None].to(dtype).cuda()  # a sequence per row, one token
    B = x.shape[0]
    cache = cb.PagedCache4(*pages4(B, 1, H, dim, dim), ints([[b] for b in range(B)]))
    cb.cache4_append(x, x, cache, ints([0] * B))
    sync_check()
    codes, scales = ref4.store(x)
    for got_c, got_s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert torch.equal(got_s.cpu().contiguous().view(torch.int16), scales[:, :, :].contiguous().view(torch.int16))
        assert torch.equal(got_c.cpu().contiguous(), codes)


def test_many_values_bit_for_bit(gpu):
    """fp32 values at large, through the kernel for whole pieces and through the other one."""
    B, T, H, dim = 4, 500, 4, 128
    x = ref.randn(B, T, H, dim, seed=5, dtype=F32, device="cuda")
    codes, scales = ref4.store(x)
    for shift in (0, 1):
        src = torch.empty(B, T, H, dim + 4, device="cuda")[..., shift:shift + dim]
        src.copy_(x)
        cache = cb.PagedCache4(*pages4(B * 5, 100, H, dim, dim), torch.arange(B * 5, dtype=torch.int32, device="cuda").view(B, 5))
        cb.cache4_append(src, src, cache, ints([0] * B))
        sync_check()
        for got, want in ((cache.k_codes, codes), (cache.k_scales, scales), (cache.v_codes, codes), (cache.v_scales, scales)):
            assert torch.equal(got.cpu().reshape(want.shape).contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def test_bad_places_are_reported_not_followed(gpu):
    cache, k, v = filled([40], 16, 1, 64, 64, seed=1)
    before = cache.k_codes.clone()
    new = torch.ones(1, 2, 1, 64, device="cuda")
    for at in (-1, 16 * cache.table.shape[1] - 1):
        cb.cache4_append(new, new, cache, ints([at]))
        assert cb.get_device_error() == cb.ERR_INVALID_ARG
    changed = (cache.k_codes != before).any(-1).any(-1).nonzero().tolist()
    assert changed == [[int(cache.table[0, 0]), 0]]  # position -1 + 1 is token 0; the table's last page is -1
    out = torch.full((1, 60, 1, 64), 5.0, device="cuda")
    cb.cache4_read(cache, out, out.clone(), first=ints([-10]))
    assert cb.get_device_error() == cb.ERR_INVALID_ARG and cb.get_device_error() == cb.OK
    assert (out[0, :10] == 0).all() and (out[0, 58:] == 0).all()
    assert torch.equal(out[0, 11:26].cpu(), k[int(cache.table[0, 0]), 1:])


def test_lengths_near_the_largest_int(gpu):
    """Tokens near 2^31 - 2 of a table that names one page everywhere."""
    page, pages = 99962, 21483
    parts = pages4(1, page, 1, 64, 64)
    cache = cb.PagedCache4(*parts, torch.zeros(1, pages, dtype=torch.int32, device="cuda"))
    x = ref.randn(1, 100, 1, 64, seed=1, dtype=BF16, device="cuda")
    last = page * pages - 100
    cb.cache4_append(x, x, cache, ints([last]))
    out = torch.zeros_like(x)
    cb.cache4_read(cache, out, torch.zeros_like(x), first=ints([last]))
    q = ref.randn(1, 4, 64, seed=3, dtype=BF16, device="cuda")
    got = run(q, cache, ints([last + 100]), scale=0.125, first=ints([last]), slopes=ref.alibi_slopes(4, "cuda"))
    sync_check()
    k = ref4.values(*ref4.store(x), 64)
    assert torch.equal(out.cpu(), k.to(BF16))
    ref.check(got, ref.decode(q, k, k, torch.zeros(1, 1, dtype=torch.int32), [100], 0.125, slopes=ref.alibi_slopes(4)), k, BF16)


def test_wide_offsets(gpu):
    """Pages more than 2^31 bytes past the first."""
    page, H, D = 16, 2, 64
    stride = (1 << 31) + 4096
    flat = torch.empty(2 * stride + (1 << 20), dtype=torch.uint8, device="cuda")
    wide = [flat.as_strided((3, page, H, 32), (stride, 32, page * 32, 1), i * 8192) for i in range(2)]
    scales = [flat.view(BF16).as_strided((3, page, H, 2), (stride // 2, 2, page * 2, 1), (32768 + i * 8192) // 2) for i in range(2)]
    cache = cb.PagedCache4(wide[0], scales[0], wide[1], scales[1], ints([[2, 0, 1]]))
    x, y = (ref.randn(1, 45, H, D, seed=i, dtype=BF16, device="cuda") for i in range(2))
    cb.cache4_append(x, y, cache, ints([0]))
    out = torch.zeros(1, 45, H, D, device="cuda"), torch.zeros(1, 45, H, D, device="cuda")
    cb.cache4_read(cache, *out)
    q = ref.randn(1, 4, D, seed=2, dtype=BF16, device="cuda")
    got = run(q, cache, ints([45]), scale=0.125)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D) for t in (x, y))
    assert torch.equal(out[0].cpu(), k) and torch.equal(out[1].cpu(), v)
    ref.check(got, ref.decode(q, k, v, torch.zeros(1, 1, dtype=torch.int32), [45], 0.125), v, BF16)


# ------------------------------------------------------------------ decode
CASES = [  # lens, page, Hq, Hkv, dk, dv
    ([1], 16, 1, 1, 64, 64), ([421], 16, 8, 2, 64, 64), ([0, 5, 64, 65, 63, 0], 16, 4, 4, 128, 128), ([1000, 1, 333], 20, 8, 1, 128, 128),
    ([100] * 5, 7, 10, 2, 96, 96), ([5000], 64, 16, 1, 64, 128), ([300, 200], 1, 6, 6, 32, 64), ([130] * 33, 128, 4, 2, 40, 72),
    ([9000, 3], 32, 4, 1, 128, 128), ([77, 78, 79], 24, 40, 2, 64, 64), ([0, 0], 16, 2, 2, 64, 64), ([90, 17], 20, 6, 3, 33, 7)]


@DTYPES
@pytest.mark.parametrize("name", ["plain", "cap", "bias", "first", "all"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_definition(gpu, case, name, dtype):
    lens, page, Hq, Hkv, dk, dv = CASES[case]
    # every other case: a table that could name far more (another way to deal the tokens), and token-major pages
    cache, k, v = filled(lens, page, Hkv, dk, dv, seed=case, wide=3000 * (case % 2), tokens_first=case % 4 == 1)
    B = len(lens)
    q = (ref.randn(B, Hq, dk, seed=case + 50, dtype=F32, device="cuda") * 3).to(dtype)
    n = ints(lens)
    kw = {"scale": dk ** -0.5}
    if name in ("cap", "all"):
        kw["softcap"] = 5.0
    if name in ("bias", "all"):
        kw["slopes"] = ref.alibi_slopes(Hq, "cuda")
    if name in ("first", "all"):  # the last sequence starts past its end
        kw["first"] = ints([x // 3 if b + 1 < B or B == 1 else x + 1 for b, x in enumerate(lens)])
    out = run(q, cache, n, **kw)
    sync_check()
    ref.check(out, ref.decode(q, k, v, cache.table, n, **kw), v, dtype)


@DTYPES
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2), (20, 2), (16, 1)], ids=str)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (32, 96), (96, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens", [[40, 0, 129], [3000, 1, 2100, 777]], ids=["whole", "runs"])
def test_head_counts_and_dims(gpu, lens, dk, dv, Hq, Hkv, dtype):
    cache, k, v = filled(lens, 16, Hkv, dk, dv, seed=dk + dv, wide=3000 * (len(lens) == 4))
    q = (ref.randn(len(lens), Hq, dk, seed=5, dtype=F32, device="cuda") * 2).to(dtype)
    n = ints(lens)
    got = run(q, cache, n, scale=dk ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k, v, cache.table, n, dk ** -0.5), v, dtype)


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
@pytest.mark.parametrize("sizes", [(1e-30, 1e30), (1e30, 1e-30), (1e36, 1e36), (1e-37, 1e-38), (1.0, 1.0)], ids=str)
def test_sizes_far_from_one(gpu, sizes, wide, dtype):
    """Keys and values of any size; queries that bring the scores back to ordinary size; values whose size changes by
    2^40 along the sequence."""
    lens, D, H = [700, 45], 64, 2
    size_k, size_v = sizes
    parts = pages4(60, 16, H, D, D)
    table = torch.full((2, 50 + wide), -1, dtype=torch.int32)
    table[0, :44], table[1, :3] = torch.randperm(44), torch.arange(44, 47)
    cache = cb.PagedCache4(*parts, table.cuda())
    x, y = (ref.randn(2, 700, H, D, seed=i, dtype=F32, device="cuda") for i in range(2))
    along = torch.logspace(-12, 0, 700, device="cuda").view(1, 700, 1, 1) if size_v == 1.0 else 1.0
    x, y = (x * size_k).to(BF16), (y * size_v * along).to(BF16)
    cb.cache4_append(x, y, cache, ints([0, 0]), count=ints(lens))
    q = (ref.randn(2, 4, D, seed=9, dtype=F32, device="cuda") * min(3 / size_k, 1e37)).to(dtype)
    got = run(q, cache, ints(lens), scale=0.125)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x, y))  # pages of one token
    place = torch.arange(1400).view(2, 700)
    ref.check(got, ref.decode(q, k, v, place, lens, 0.125), v, dtype)


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
def test_even_weights_over_long_sequences(gpu, wide, dtype):
    """Queries of zeros: the mean of the values, small beside them, over tens of thousands of tokens; and single
    tokens whose values are far above the others'."""
    n, D = 40000, 64
    cache, k, v = filled([n, 100], 64, 1, D, D, seed=2, wide=wide)
    q = torch.zeros(2, 8, D, dtype=dtype, device="cuda")
    got = run(q, cache, ints([n, 100]), scale=0.125)
    sync_check()
    want = ref.decode(q, k, v, cache.table, [n, 100], 0.125)
    # the mean of n values c s: weights 2^-24 n ... their sum's roundings, relative to the result, and the output's own
    bound = torch.finfo(dtype).eps / 2 * want.abs() + 2e-6 * float(v.abs().max()) + (2.0 ** -10 * want.abs() if dtype == BF16 else 0)
    assert ((got.cpu().double() - want).abs() <= bound).all()


@DTYPES
def test_nan_reaches_only_who_sees_it(gpu, dtype):
    """A group with a NaN or an infinity: NaN where it is seen, nothing where it is behind the length or before the
    first key, or another head's."""
    lens, D, H = [50, 50, 50, 50], 64, 2
    x, y = (ref.randn(4, 50, H, D, seed=i, dtype=BF16, device="cuda") for i in range(2))
    x0, y0 = x.clone(), y.clone()
    x[0, 10, 0, 3], y[1, 20, 1, 40] = float("nan"), float("inf")
    x[2, 45, 0, 0], y[2, 49, 1, 1] = float("nan"), float("nan")  # behind the length
    x[3, 2, 1, 0], y[3, 0, 0, 1] = float("inf"), float("nan")  # before the first key
    cache = cb.PagedCache4(*pages4(16, 16, H, D, D), torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4))
    cb.cache4_append(x, y, cache, ints([0] * 4))
    q = ref.randn(4, 4, D, seed=5, dtype=dtype, device="cuda")
    n, first = ints([50, 50, 45, 50]), ints([0, 0, 0, 3])
    got = run(q, cache, n, scale=0.125, first=first)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x0, y0))
    want = ref.decode(q, k, v, torch.arange(200).view(4, 50), n, 0.125, first=first)
    bad = torch.zeros(4, 4, D, dtype=torch.bool)
    bad[0, :2], bad[1, 2:, 32:] = True, True
    assert torch.equal(torch.isnan(got.float()).cpu(), bad)
    ref.check(torch.where(bad.cuda(), torch.zeros_like(got), got), torch.where(bad, torch.zeros_like(want), want), v, dtype)


@DTYPES
def test_same_bits_twice(gpu, dtype):
    lens = [9000, 10, 4000]
    cache, k, v = filled(lens, 16, 2, 64, 64, seed=1)
    q = ref.randn(3, 8, 64, seed=2, dtype=dtype, device="cuda")
    a = run(q, cache, ints(lens), scale=0.125)
    torch.cuda.synchronize()
    b = run(q, cache, ints(lens), scale=0.125, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
def test_bad_pages_count_as_absent(gpu, wide, dtype):
    lens = [100, 100]
    cache, k, v = filled(lens, 16, 2, 64, 64, seed=4, wide=wide)
    q = ref.randn(2, 4, 64, seed=2, dtype=dtype, device="cuda")
    good = run(q, cache, ints(lens), scale=0.125)
    assert cb.get_device_error() == cb.OK
    rows = cache.table[0].cpu().long()
    cache.table[0, 2] = k.shape[0] + 5
    out = run(q, cache, ints(lens), scale=0.125)
    assert cb.get_device_error() == cb.ERR_INVALID_ARG and cb.get_device_error() == cb.OK
    keep = torch.tensor([j for j in range(100) if not 32 <= j < 48])
    kk, vv = k[rows[keep // 16], keep % 16].double(), v[rows[keep // 16], keep % 16].double()
    want = torch.stack([torch.softmax(kk[:, h // 2] @ q[0, h].cpu().double() * 0.125, 0) @ vv[:, h // 2] for h in range(4)])
    assert torch.equal(out[1], good[1])
    ref.check(out[0], want, v, dtype)


@DTYPES
def test_strides_and_clamped_lengths(gpu, dtype):
    """A slice of wider queries into a slice of a wider output; lengths past the table."""
    cache, k, v = filled([48, 48], 16, 3, 64, 64, seed=6, spare=0)
    cache = cb.PagedCache4(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.table[:, :3])
    q = ref.randn(2, 6, 66, seed=5, dtype=dtype, device="cuda")[..., 1:65]
    buf = torch.full((2, 8, 65), 77.0, dtype=dtype, device="cuda")
    run(q, cache, ints([1 << 30, 48]), out=buf[:, 1:-1, 1:], scale=0.125)
    sync_check()
    ref.check(buf[:, 1:-1, 1:], ref.decode(q, k, v, cache.table, [48, 48], 0.125), v, dtype)
    assert (buf[:, 0] == 77).all() and (buf[:, -1] == 77).all() and (buf[..., 0] == 77).all()


@DTYPES
@pytest.mark.parametrize("dims", [(64, 64), (7, 5)], ids=str)
@pytest.mark.parametrize("B", [129, 1000])
def test_more_sequences_than_threads(gpu, B, dims, dtype):
    lens = [(37 * b) % 50 if b % 5 else 0 for b in range(B)]
    cache, k, v = filled(lens, 16, 1, *dims, seed=7, wide=3000 * (B > 500))
    q = ref.randn(B, 2, dims[0], seed=8, dtype=dtype, device="cuda")
    got = run(q, cache, ints(lens), scale=dims[0] ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k, v, cache.table, lens, dims[0] ** -0.5), v, dtype)


@DTYPES
def test_two_captured_steps_share_a_workspace(gpu, dtype):
    """Append and decode captured in a graph, replayed in turn with another graph on the same workspace."""
    B, H, D = 3, 2, 64
    caches = [cb.PagedCache4(*pages4(12, 16, H, D, D), torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)) for _ in range(2)]
    q, x = ref.randn(B, 8, D, seed=1, dtype=dtype, device="cuda"), ref.randn(B, 1, H, D, seed=2, dtype=dtype, device="cuda")
    past = [ref.randn(B, 40, H, D, seed=3 + i, dtype=dtype, device="cuda") for i in range(2)]
    pos, n = ints([40] * B), ints([41] * B)
    ws = torch.empty(cb.attention_decode4_workspace(q, caches[0]), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty(B, 8, D, dtype=dtype, device="cuda") for _ in range(2)], []
    for c, p, o in zip(caches, past, outs):
        cb.cache4_append(p, p, c, ints([0] * B))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cb.cache4_append(x, x, c, pos)
            cb.attention_decode4(q, c, n, o, ws, scale=0.125)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    sync_check()
    for p, o in zip(past, outs):
        k = ref4.values(*ref4.store(torch.cat([p, x], 1)), D)
        ref.check(o, ref.decode(q, k.flatten(0, 1)[:, None], k.flatten(0, 1)[:, None], torch.arange(B * 41).view(B, 41), [41] * B, 0.125), k, dtype)


@DTYPES
def test_rotated_cached_and_attended(gpu, dtype):
    """A prompt and three tokens through all of them: rotate, append, decode; then the cached prompt read back for a
    further prompt's attention."""
    B, L, Hq, H, D = 2, 37, 8, 2, 64
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device="cuda")
    rule = cb.Rotation(freq, axis=torch.arange(32, dtype=torch.int32, device="cuda") % 3, axes=3, norm=True)
    cache = cb.PagedCache4.empty(B * 3, 16, H, D, D, torch.arange(B * 3, dtype=torch.int32, device="cuda").view(B, 3))
    keys, vals = [], []
    at = 0
    for step, T in enumerate((L, 1, 1, 1)):
        row = ref.randn(B, T, (Hq + 2 * H) * D, seed=step, dtype=dtype, device="cuda").unflatten(-1, (-1, D))
        q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + H], row[:, :, Hq + H:]
        pos = torch.arange(at, at + T, dtype=torch.int32, device="cuda").expand(3, B, T).contiguous()
        cb.norm_rotate(q, k, pos, rule)
        cb.cache4_append(k, v, cache, ints([at] * B))
        keys.append(ref4.values(*ref4.store(k), D)), vals.append(ref4.values(*ref4.store(v), D))
        at += T
        if T == 1:
            kk, vv = torch.cat(keys, 1), torch.cat(vals, 1)
            got = run(q[:, 0], cache, ints([at] * B), scale=0.125)
            sync_check()
            ref.check(got, ref.decode(q[:, 0], kk.flatten(0, 1)[:, None], vv.flatten(0, 1)[:, None], torch.arange(B * at).view(B, at),
                                      [at] * B, 0.125), vv, dtype)
    kc, vc = (torch.empty(B, at, H, D, dtype=dtype, device="cuda") for _ in range(2))
    cb.cache4_read(cache, kc, vc)
    q = ref.randn(B, 5, Hq, D, seed=20, dtype=dtype, device="cuda")
    out = torch.empty(B, 5, Hq, D, dtype=dtype, device="cuda")
    cb.attention(q, kc, vc, out, cb.Score(0.125))
    sync_check()
    assert torch.equal(kc.cpu(), torch.cat(keys, 1).to(dtype)) and torch.equal(vc.cpu(), torch.cat(vals, 1).to(dtype))
    ref.check(out, ref.attention(q, kc, vc, 0.125), vc, dtype)


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
@pytest.mark.parametrize("at", [0, 5, 150], ids=lambda x: f"token{x}")
def test_a_large_value_of_no_weight(gpu, at, wide, dtype):
    """One token's values are 2^40 times the others', and its weight e^-100 of theirs; the second half of the dims is
    2^-24 of the first.  Each half is as exact as without the token."""
    n, D = 300, 64
    x, y = (ref.randn(2, n, 1, D, seed=i, dtype=F32, device="cuda") for i in range(2))
    y[..., 32:] *= 2.0 ** -24
    x[0, at, 0, 0], y[0, at] = -100.0, y[0, at] * 2.0 ** 40
    x, y = x.to(BF16), y.to(BF16)
    table = torch.full((2, 19 + wide), -1, dtype=torch.int32)
    table[:, :19] = torch.arange(38).view(2, 19)
    cache = cb.PagedCache4(*pages4(38, 16, 1, D, D), table.cuda())
    cb.cache4_append(x, y, cache, ints([0, 0]))
    q = torch.zeros(2, 4, D, dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([8.0, 7.0, 8.5, 9.0], dtype=dtype, device="cuda")
    got = run(q, cache, ints([n, n]), scale=0.125)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x, y))
    want = ref.decode(q, k, v, torch.arange(2 * n).view(2, n), [n, n], 0.125)
    v[at] = 0
    for half in (slice(0, 32), slice(32, 64)):
        ref.check(got[..., half], want[..., half], v[..., half], dtype)


def walked(q, x, y, wide, want, v, dtype, parts):
    """300 sequences that share two sequences' tokens x, y [2, n, 1, D]: a warp walks several steps of one."""
    n, D = x.shape[1], x.shape[3]
    per = (n + 15) // 16
    table = torch.full((2, per + wide), -1, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.arange(2 * per, device="cuda").view(2, per)
    pages = pages4(2 * per, 16, 1, D, D)
    cb.cache4_append(x, y, cb.PagedCache4(*pages, table), ints([0, 0]))
    got = run(q.repeat(150, 1, 1), cb.PagedCache4(*pages, table.repeat(150, 1)), ints([n] * 300), scale=0.125)
    sync_check()
    for part in parts:
        ref.check(got[..., part], want.repeat(150, 1, 1)[..., part], v[..., part], dtype)


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
@pytest.mark.parametrize("early,late", [(-123, 14), (-100, 60), (-126, -126), (100, 30)], ids=str)
def test_values_that_grow_or_shrink_by_many_powers(gpu, early, late, wide, dtype):
    """Values of 2^early, then of 2^late; the first ones have no weight where they are the larger ones."""
    n, D = 500, 64
    x, y = (ref.randn(2, n, 1, D, seed=i, dtype=F32, device="cuda") for i in range(2))
    y[:, :200] *= 2.0 ** early
    y[:, 200:] *= 2.0 ** late
    x[..., 0] = 0.0
    if early > late:  # e^-100 and less
        x[:, :200, 0, 0] = -100.0
    x, y = x.to(BF16), y.to(BF16)
    q = torch.zeros(2, 4, D, dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([8.0, 9.0, 10.0, 8.5], dtype=dtype, device="cuda")
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x, y))  # pages of one token
    want = ref.decode(q, k, v, torch.arange(2 * n).view(2, n), [n, n], 0.125)
    if early > late:  # 2^100 e^-100 is 2^-44: beside 2^30 nothing
        v.view(2, n, D)[:, :200] = 0
    walked(q, x, y, wide, want, v, dtype, [slice(None)])


@DTYPES
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
@pytest.mark.parametrize("at", [0, 5, 150, 499], ids=lambda x: f"token{x}")
def test_a_large_value_of_no_weight_in_a_long_walk(gpu, at, wide, dtype):
    """As above, where a warp has other tokens before and behind that one."""
    n, D = 500, 64
    x, y = (ref.randn(2, n, 1, D, seed=i, dtype=F32, device="cuda") for i in range(2))
    y[..., 32:] *= 2.0 ** -24
    x[:, at, 0, 0], y[:, at] = -100.0, y[:, at] * 2.0 ** 40
    x, y = x.to(BF16), y.to(BF16)
    q = torch.zeros(2, 4, D, dtype=dtype, device="cuda")
    q[..., 0] = torch.tensor([8.0, 7.0, 8.5, 9.0], dtype=dtype, device="cuda")
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x, y))
    want = ref.decode(q, k, v, torch.arange(2 * n).view(2, n), [n, n], 0.125)
    v.view(2, n, D)[:, at] = 0
    walked(q, x, y, wide, want, v, dtype, [slice(0, 32), slice(32, 64)])


@DTYPES
def test_values_that_begin_with_zeros(gpu, dtype):
    """Tokens, and groups, of zeros before the first others."""
    n, D = 200, 64
    x, y = (ref.randn(1, n, 1, D, seed=i, dtype=BF16, device="cuda") for i in range(2))
    y[0, :70] = 0
    y[0, :, 0, 32:] = 0
    y[0, 199, 0, 40] = 3.0
    cache = cb.PagedCache4(*pages4(13, 16, 1, D, D), torch.arange(13, dtype=torch.int32, device="cuda").view(1, 13))
    cb.cache4_append(x, y, cache, ints([0]))
    q = ref.randn(1, 8, D, seed=9, dtype=dtype, device="cuda")
    got = run(q, cache, ints([n]), scale=0.125)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D).flatten(0, 1)[:, None] for t in (x, y))
    ref.check(got, ref.decode(q, k, v, torch.arange(n).view(1, n), [n], 0.125), v, dtype)


@DTYPES
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (12, 2), (10, 1)], ids=str)
@pytest.mark.parametrize("dk,dv", [(40, 72), (72, 40), (8, 120), (104, 8)])
@pytest.mark.parametrize("lens", [[40, 0, 129], [3000, 1, 2100, 777]], ids=["whole", "runs"])
def test_dims_of_whole_words(gpu, lens, dk, dv, Hq, Hkv, dtype):
    """Rows that are multiples of 4 bytes, not of 16; a last group of 8, 16 or 24 dims."""
    cache, k, v = filled(lens, 16, Hkv, dk, dv, seed=dk + dv, wide=3000 * (len(lens) == 4))
    q = (ref.randn(len(lens), Hq, dk, seed=5, dtype=F32, device="cuda") * 2).to(dtype)
    got = run(q, cache, ints(lens), scale=dk ** -0.5)
    sync_check()
    ref.check(got, ref.decode(q, k, v, cache.table, lens, dk ** -0.5), v, dtype)


@DTYPES
@pytest.mark.parametrize("gap,shift", [(4, 0), (16, 4), (3, 1), (32, 16)], ids=str)
@pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])
def test_gaps_between_rows(gpu, wide, gap, shift, dtype):
    """Codes that lie at any byte, scales at any bf16: append, read and decode choose by that."""
    lens, H, D, page = [300, 45, 0], 2, 64, 32
    count = 13
    table = torch.full((3, 11 + wide), -1, dtype=torch.int32)
    table[0, :10], table[1, :2] = torch.randperm(10, generator=torch.Generator().manual_seed(1)), torch.tensor([10, 12])
    parts = []
    for _ in range(2):
        codes = torch.full((count, H, page, 32 + gap), 255, dtype=torch.uint8, device="cuda")
        scales = torch.full((count, H, page, 2 + gap % 4), float("nan"), dtype=BF16, device="cuda")
        parts += [codes, scales]
    cut = [parts[i][..., shift:shift + 32].transpose(1, 2) if i % 2 == 0 else parts[i][..., :2].transpose(1, 2) for i in range(4)]
    cache = cb.PagedCache4(*cut, table.cuda())
    x, y = (ref.randn(3, 300, H, D, seed=i, dtype=dtype, device="cuda") for i in range(2))
    cb.cache4_append(x, y, cache, ints([0] * 3), count=ints(lens))
    out = [torch.zeros(3, 300, H, D, dtype=dtype, device="cuda") for _ in range(2)]
    cb.cache4_read(cache, *out, count=ints(lens))
    q = ref.randn(3, 4, D, seed=9, dtype=dtype, device="cuda")
    got = run(q, cache, ints(lens), scale=0.125)
    sync_check()
    k, v = (ref4.values(*ref4.store(t), D) for t in (x, y))
    for t, w in zip(out, (k, v)):
        for b, n in enumerate(lens):
            assert torch.equal(t[b, :n].cpu(), w[b, :n].to(dtype)) and (t[b, n:] == 0).all()
    flat = [t.flatten(0, 1)[:, None] for t in (k, v)]
    ref.check(got, ref.decode(q, *flat, torch.arange(900).view(3, 300), lens, 0.125), v, dtype)
    for i in (0, 2):  # the gaps
        assert (parts[i][..., :shift] == 255).all() and (parts[i][..., shift + 32:] == 255).all()


def test_no_pages(gpu):
    """A cache without a page: every token is absent, and said to be."""
    cache = cb.PagedCache4.empty(0, 16, 2, 64, 64, torch.zeros(2, 3, dtype=torch.int32, device="cuda"))
    q = ref.randn(2, 4, 64, seed=1, dtype=BF16, device="cuda")
    got = run(q, cache, ints([5, 0]), scale=0.125)
    assert cb.get_device_error() == cb.ERR_INVALID_ARG and cb.get_device_error() == cb.OK
    assert (got == 0).all()
