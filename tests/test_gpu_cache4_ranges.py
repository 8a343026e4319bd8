"""Attention over a 4-bit cache where sizes differ by many powers of two, between tokens, groups of dims and heads,
against the definition in 64 bits; and how far its roundings go."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check
from test_gpu_cache4 import BF16, DTYPES, F32, ints, pages4, run

pytestmark = pytest.mark.gpu
WAYS = pytest.mark.parametrize("wide", [0, 3000], ids=["whole", "runs"])


def stored(x, y, copies=1, wide=0, page=16):
    """A cache of sequences with tokens x [B, n, H, dk] and y [B, n, H, dv], `copies` times over the same pages, and the
    stored values as pages of one token with the table that names them."""
    B, n, H, dk = x.shape
    per = (n + page - 1) // page
    table = torch.full((B, per + wide), -1, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.arange(B * per, device="cuda").view(B, per)
    parts = pages4(B * per, page, H, dk, y.shape[3])
    cb.cache4_append(x, y, cb.PagedCache4(*parts, table, dim_k=dk, dim_v=y.shape[3]), ints([0] * B))
    cache = cb.PagedCache4(*parts, table.repeat(copies, 1), dim_k=dk, dim_v=y.shape[3])
    k, v = (ref4.values(*ref4.store(t), t.shape[3]).flatten(0, 1)[:, None] for t in (x, y))
    return cache, k, v, torch.arange(B * n).view(B, n)


def scored(n, D, at, low, seed):
    """Keys whose first dim alone is asked for: ordinary ones, and token `at` of weight e^-1000 where low."""
    x = ref.randn(2, n, 1, D, seed=seed, dtype=F32, device="cuda")
    x[..., 0] = 0.0
    if low:
        x[:, at, 0, 0] = -1000.0
    return x


def asking(Hq, D, dtype, copies):
    q = torch.zeros(2, Hq, D, dtype=dtype, device="cuda")
    q[..., 0] = torch.linspace(8.0, 10.0, Hq).to(dtype)
    return q, q.repeat(copies, 1, 1)


# ------------------------------------------------------------------ values
@DTYPES
@WAYS
@pytest.mark.parametrize("copies", [1, 150], ids=["alone", "walk"])
@pytest.mark.parametrize("low", [False, True], ids=["weighted", "unweighted"])
@pytest.mark.parametrize("early,late", [(-100, 70), (-123, 100), (-126, 122)], ids=str)
def test_finite_values_stay_finite(gpu, early, late, low, copies, wide, dtype):
    """Values of 2^early and one token of 2^late, up to 2^248 times the others."""
    n, D, at = 500, 64, 300
    x, y = scored(n, D, at, low, 0), ref.randn(2, n, 1, D, seed=1, dtype=F32, device="cuda").clamp(-3, 3)
    large = y[:, at] * 2.0 ** late
    y *= 2.0 ** early
    y[:, at] = large
    x, y = x.to(BF16), y.to(BF16)
    cache, k, v, place = stored(x, y, copies, wide)
    q, many = asking(4, D, dtype, copies)
    want = ref.decode(q, k, v, place, [n, n], 0.125)
    got = run(many, cache, ints([n] * 2 * copies), scale=0.125)
    sync_check()
    if low:
        v.view(2, n, D)[:, at] = 0
    ref.check(got, want.repeat(copies, 1, 1), v, dtype)


@DTYPES
@WAYS
@pytest.mark.parametrize("copies", [1, 150], ids=["alone", "walk"])
@pytest.mark.parametrize("early,late", [(-61, 69), (-20, 115), (-20, 15), (-60, 60)], ids=str)
def test_values_far_below_one_of_no_weight(gpu, early, late, copies, wide, dtype):
    """The same where the large value has no weight, and f16, or the least scale beside it, would take the others'."""
    test_finite_values_stay_finite(gpu, early, late, True, copies, wide, dtype)


@DTYPES
@WAYS
@pytest.mark.parametrize("copies", [1, 150], ids=["alone", "walk"])
@pytest.mark.parametrize("low", [False, True], ids=["weighted", "unweighted"])
@pytest.mark.parametrize("at", [0, 5, 40, 130], ids=lambda x: f"token{x}")
@pytest.mark.parametrize("power", [6, 13, 24, 32, 40, 100], ids=lambda p: f"2^{p}")
def test_an_outlier_in_one_group(gpu, power, at, low, copies, wide, dtype):
    """One token's first 32 values are 2^power times the others': each group of dims is as exact as its own values
    ask for, whatever the token's weight."""
    n, D = 140, 96
    x, y = scored(n, D, at, low, 2), ref.randn(2, n, 1, D, seed=3, dtype=F32, device="cuda").abs() + 0.5
    y[:, at, :, :32] *= 2.0 ** power
    y[..., 64:] *= 2.0 ** -30
    x, y = x.to(BF16), y.to(BF16)
    cache, k, v, place = stored(x, y, copies, wide)
    q, many = asking(5, D, dtype, copies)
    want = ref.decode(q, k, v, place, [n, n], 0.125).repeat(copies, 1, 1)
    got = run(many, cache, ints([n] * 2 * copies), scale=0.125)
    sync_check()
    if low:
        v.view(2, n, D)[:, at] = 0
    for group in (slice(0, 32), slice(32, 64), slice(64, 96)):
        ref.check(got[..., group], want[..., group], v[..., group], dtype)


# ------------------------------------------------------------------ scores
@DTYPES
@WAYS
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("size", [100, 40, 0, -100], ids=lambda e: f"keys2^{e}")
def test_heads_of_different_sizes(gpu, size, cap, wide, dtype):
    """A head whose scores go to 2^120 beside heads of ordinary scores, whatever the keys' size.  Queries of one dim of
    8 bits, so that scores are exact: of the large ones one token's is the largest."""
    n, D = 120, 64
    x, y = ref.randn(2, n, 1, D, seed=4, dtype=F32, device="cuda") * 2.0 ** size, ref.randn(2, n, 1, D, seed=5, dtype=BF16, device="cuda")
    cache, k, v, place = stored(x.to(BF16), y, 1, wide)
    q = torch.zeros(2, 4, D, dtype=F32, device="cuda")
    for h, power in enumerate((118 - size if size >= 0 else 126, 3 - size, 1 - size, -size)):
        q[:, h, 17 + h] = 1.375 * 2.0 ** power
    q = q.to(dtype)
    got = run(q, cache, ints([n, n]), scale=0.125, softcap=cap)
    sync_check()
    ref.check(got, ref.decode(q, k, v, place, [n, n], 0.125, softcap=cap), v, dtype)


@DTYPES
@WAYS
@pytest.mark.parametrize("copies", [1, 150], ids=["alone", "walk"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("power", [4, 12, 19, 20, 21, 24, 31, 33, 40, 80, 119], ids=lambda e: f"2^{e}")
def test_scores_of_any_size(gpu, power, sign, copies, wide, dtype):
    """Scores of up to 2^power, exact as above, all of one sign: the largest one's token is the result, or tokens of equal scores
    are."""
    n, D = 300, 64
    x, y = (ref.randn(2, n, 1, D, seed=s, dtype=F32, device="cuda") for s in (6, 7))
    x = (x.abs() + 0.5) * sign
    cache, k, v, place = stored(x.to(BF16), y.to(BF16), copies, wide)
    q = torch.zeros(2, 4, D, dtype=F32, device="cuda")
    for h in range(4):
        q[:, h, 17 + h] = 1.375 * 2.0 ** power
    q = q.to(dtype)
    want = ref.decode(q, k, v, place, [n, n], 0.125).repeat(copies, 1, 1)
    got = run(q.repeat(copies, 1, 1), cache, ints([n] * 2 * copies), scale=0.125)
    sync_check()
    ref.check(got, want, v, dtype)


@DTYPES
@WAYS
@pytest.mark.parametrize("power", [3, 8, 14, 20, 28, 40, 60], ids=lambda e: f"2^{e}")
def test_queries_small_where_keys_are_large(gpu, power, wide, dtype):
    """A group of dims whose queries are 2^-power of the others' and whose keys 2^power: it has as much to say in a score."""
    n, D = 200, 96
    x, y = (ref.randn(2, n, 1, D, seed=s, dtype=F32, device="cuda") for s in (8, 9))
    q = ref.randn(2, 5, D, seed=10, dtype=F32, device="cuda")
    x[..., 32:64] *= 2.0 ** power
    q[..., 32:64] *= 2.0 ** -power
    q[:, 2, 64:] = 0
    x, y, q = x.to(BF16), y.to(BF16), q.to(dtype)
    cache, k, v, place = stored(x, y, 1, wide)
    got = run(q, cache, ints([n, n]), scale=0.3)
    sync_check()
    ref.check(got, ref.decode(q, k, v, place, [n, n], 0.3), v, dtype)


@DTYPES
@WAYS
@pytest.mark.parametrize("top", [127, -100], ids=lambda e: f"2^{e}")
def test_small_groups_of_queries_at_the_ends_of_the_range(gpu, top, wide, dtype):
    """Queries up to 2^127, or of 2^-100, with a group far below them and keys that bring both to ordinary scores."""
    n, D = 100, 64
    x, y = (ref.randn(2, n, 1, D, seed=s, dtype=F32, device="cuda").clamp(-3, 3) for s in (11, 12))
    q = ref.randn(2, 5, D, seed=13, dtype=F32, device="cuda").clamp(-0.99, 0.99)
    low = max(top - 60, -125)
    x[..., :32] *= 2.0 ** min(-top, 120) if top < 0 else 2.0 ** -63
    x[..., :32] *= 1.0 if top < 0 else 2.0 ** -64
    x[..., 32:] *= 2.0 ** -low
    q = torch.cat([q[..., :32] * 2.0 ** (top - 20) * 2.0 ** 20, q[..., 32:] * 2.0 ** low], -1)
    x, y, q = x.to(BF16), y.to(BF16), q.to(dtype)
    cache, k, v, place = stored(x, y, 1, wide)
    got = run(q, cache, ints([n, n]), scale=0.3)
    sync_check()
    assert torch.isfinite(q).all() and (q[..., :32].abs().amax() > 2.0 ** (top - 1))
    ref.check(got, ref.decode(q, k, v, place, [n, n], 0.3), v, dtype)
