"""How far the roundings of attention over a 4-bit cache go, against bounds that count them.

bf16 (include/cb.h, csrc/decode4.cuh): a weight times its token's largest scale is rounded to f16 (half a step: 2^-11 of
it), so is a group's scale beside that, and their product: three roundings where a token has several groups, one where it
has one.  A step's MMA adds up to 17 terms, each cut off at 2^-14 of the largest weight in it times one code (25 bits below
the largest product, whose code counts as 2^-14 where it is code 2^-24), twice (codes, offset), in rows for two dims of
which one is a difference: 4 terms cut for each token, and for the sum so far.  Then the output's rounding, 2^-8 of it at most.
fp32: weights to 22 bits (two f16 numbers, 2^-22), exponentials and scores to a few 2^-22 for the scores here, sums of
fp32: 2^-18 in all of the sum of |weight value|."""
import math

import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from gpu_util import sync_check
from test_gpu_cache4 import BF16, DTYPES, F32, ints, run
from test_gpu_cache4_ranges import WAYS, stored

pytestmark = pytest.mark.gpu


def sums(q, k, v, n, scale):
    """float64 [B, Hq, Dv]: the result; the sum of |weight value|; 4 2^-14 of the steps' largest weight times scale, for every
    token and once more for a step.  k, v [B, n, D]."""
    B, Hq, _ = q.shape
    p = torch.softmax(torch.einsum("bhd,bnd->bhn", q.cpu().double(), k.double()) * scale, -1)
    v = v.double()
    size = v.abs().unflatten(-1, (-1, 32)).amax(-1) / 7 * 1.01  # scales, bf16's rounding up
    cut = torch.zeros(B, Hq, v.shape[-1], dtype=torch.float64)
    for lo in range(0, n, 16):
        most = torch.einsum("bhn,bng->bhng", p[..., lo:lo + 16], size[:, lo:lo + 16]).amax(2)
        cut += (min(n - lo, 16) + 1) * 4 * 2.0 ** -14 * most.repeat_interleave(32, -1)
    return torch.einsum("bhn,bnd->bhd", p, v), torch.einsum("bhn,bnd->bhd", p, v.abs()), cut


def check(got, want, total, cut, dtype, roundings, score_error=0.0):
    got = got.cpu().double()
    scores = math.expm1(2 * score_error) * (total + want.abs())
    if dtype == F32:
        bound = 2.0 ** -18 * total + 2.0 ** -24 * want.abs() + scores
    else:
        bound = (1 + score_error) * (roundings * 2.0 ** -11 * 1.02 * total + cut) + 2.0 ** -8 * want.abs() + scores
    over = float(((got - want).abs() / bound.clamp(min=1e-30)).max())
    assert torch.isfinite(got).all() and over <= 1.0, over


@DTYPES
@WAYS
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("n", [2, 4, 6])
def test_weights_keep_their_bits(gpu, n, D, wide, dtype):
    """Few tokens whose values nearly cancel: what is left of the sum shows the weights' roundings, and the output's own
    is small.  Scores are exact: one dim of the query has a value."""
    B = 300
    x, y = (ref.randn(B, n, 1, D, seed=s, dtype=F32, device="cuda") for s in (20, 21))
    for t in range(1, n, 2):
        y[:, t] = -y[:, t - 1]
        x[:, t] = x[:, t - 1] * 0.97
    cache, k, v, _ = stored(x.to(BF16), y.to(BF16), 1, wide)
    q = torch.zeros(B, 8, D, dtype=dtype, device="cuda")
    for h in range(8):
        q[:, h, h] = 0.5 + h / 4
    got = run(q, cache, ints([n] * B), scale=0.125)
    sync_check()
    check(got, *sums(q, k.view(B, n, D), v.view(B, n, D), n, 0.125), dtype, 1 if D == 32 else 3)


@DTYPES
@WAYS
@pytest.mark.parametrize("power", [0, 4, 8])
def test_queries_with_one_large_dim(gpu, power, wide, dtype):
    """bf16: a score's products are cut off at 2^-14 of a group's largest query times its keys' scale, 17 of them in each of
    two MMAs."""
    B, n, D = 20, 40, 64
    x, y = (ref.randn(B, n, 1, D, seed=s, dtype=F32, device="cuda") for s in (22, 23))
    q = ref.randn(B, 4, D, seed=24, dtype=F32, device="cuda") * 2.0 ** -power
    q[..., 5] *= 2.0 ** power
    q = q.to(dtype)
    cache, k, v, _ = stored(x.to(BF16), y.to(BF16), 1, wide)
    got = run(q, cache, ints([n] * B), scale=0.125)
    sync_check()
    k = k.view(B, n, D)
    large = q.cpu().double().abs().unflatten(-1, (-1, 32)).amax(-1).amax((0, 1))  # of each group
    scales = k.double().abs().unflatten(-1, (-1, 32)).amax(-1).amax((0, 1)) / 7 * 1.01
    error = 0.125 * (34 * 2.0 ** -14 if dtype == BF16 else 32 * 15 * 2.0 ** -24) * float((large * scales).sum()) + 2.0 ** -19
    check(got, *sums(q, k, v.view(B, n, D), n, 0.125), dtype, 3, error)


@DTYPES
@WAYS
@pytest.mark.parametrize("power", [10, 20])
@pytest.mark.parametrize("groups", [1, 2], ids=["one_group", "all_groups"])
def test_weighted_tokens_far_above_others_in_a_long_walk(gpu, groups, power, wide, dtype):
    """Tokens of ordinary weight whose values are 2^power times the others', among tens of thousands: each group against
    its own sums."""
    n, D = 40000, 64
    x, y = (ref.randn(1, n, 1, D, seed=s, dtype=F32, device="cuda") for s in (25, 26))
    y[:, torch.tensor([7, 9000, 20011, 39990], device="cuda"), :, :32 * groups] *= 2.0 ** power
    cache, k, v, _ = stored(x.to(BF16), y.to(BF16), 1, wide)
    q = torch.zeros(1, 8, D, dtype=dtype, device="cuda")
    got = run(q, cache, ints([n]), scale=0.125)
    sync_check()
    want, total, cut = sums(q, k.view(1, n, D), v.view(1, n, D), n, 0.125)
    check(got, want, total, cut, dtype, 3)
