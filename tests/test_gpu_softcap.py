"""Capped scores on every attention kernel, at caps far above, near and far below the scores, against the
definition in 64 bits: scale, cap tanh(s / cap), softmax."""
import pytest
import torch

import attention_ref as ref
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check
from test_gpu_decode import finite, paged, run as run_decode

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def definition(q, k, v, scale, softcap, slopes=None, causal=False):
    """attention_ref.attention for whole rows, on the GPU in 64 bits."""
    group = q.shape[2] // k.shape[2]
    q, k, v = q.double(), k.double().repeat_interleave(group, 2), v.double().repeat_interleave(group, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * scale
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    i, j = torch.arange(s.shape[2], device="cuda")[:, None], torch.arange(s.shape[3], device="cuda")[None, :]
    i = i + (s.shape[3] - s.shape[2] if causal else 0)
    if slopes is not None:
        s = s - slopes.double()[None, :, None, None] * (i - j).abs()
    if causal:
        s = s.masked_fill(j > i, float("-inf"))
    return torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), v).cpu()


def tokens(shape, dtype, seed, spread=3.0):
    B, Lq, Lk, Hq, Hkv, Dk, Dv = shape
    return ((ref.randn(B, Lq, Hq, Dk, seed=seed, dtype=F32, device="cuda") * spread).to(dtype),
            ref.randn(B, Lk, Hkv, Dk, seed=seed + 1, dtype=dtype, device="cuda"),
            ref.randn(B, Lk, Hkv, Dv, seed=seed + 2, dtype=dtype, device="cuda"))


def attend(q, k, v, **kw):
    out = torch.full((*q.shape[:3], v.shape[3]), float("nan"), dtype=q.dtype, device="cuda")
    if kw.get("causal"):
        kw["q_offset"] = k.shape[1] - q.shape[1]
    cb.attention(q, k, v, out, cb.Score(**kw))
    sync_check()
    return out


# few queries per key head (the streaming kernel), then tiles (tensor cores; fp32 on the CUDA cores), then bf16
# rows that are not whole 16-byte pieces
ROWS = [(1, 1, 1000, 8, 1, 128, 128), (8, 2, 700, 6, 2, 64, 64), (4, 1, 300, 4, 4, 96, 64)]
TILES = [(2, 400, 400, 4, 4, 32, 64), (16, 300, 300, 8, 2, 128, 128), (2, 150, 150, 2, 2, 33, 31)]
CAPS = pytest.mark.parametrize("softcap", [50.0, 1e3, 1e6, 1e30], ids=str)


@TYPES
@CAPS
@pytest.mark.parametrize("shape", ROWS + TILES, ids=lambda s: "x".join(map(str, s)))
def test_attention_keeps_scores_far_below_their_cap(gpu, shape, softcap, dtype):
    q, k, v = tokens(shape, dtype, seed=3)
    kw = {"scale": shape[5] ** -0.5, "softcap": softcap}
    ref.check(attend(q, k, v, **kw), definition(q, k, v, **kw), v, dtype)


@TYPES
@CAPS
@pytest.mark.parametrize("dims", [(64, 64), (96, 128), (33, 31)], ids=str)
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (16, 2)], ids=["one_head", "eight_heads"])
@pytest.mark.parametrize("lens", [[421, 77], [3000, 1, 2100]], ids=["whole", "runs"])
def test_decode_keeps_scores_far_below_their_cap(gpu, lens, Hq, Hkv, dims, softcap, dtype):
    dk, dv = dims
    k, v, table = paged(lens, 16, Hkv, dk, dv, dtype, seed=2)
    if len(lens) == 3:  # a table that could name far more: too many tiles for whole items
        table = torch.cat([table, torch.full((3, 3000), -1, dtype=torch.int32, device="cuda")], 1)
    q = (ref.randn(len(lens), Hq, dk, seed=5, dtype=F32, device="cuda") * 3).to(dtype)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = {"scale": dk ** -0.5, "softcap": softcap}
    got = run_decode(q, k, v, table, n, **kw)
    sync_check()
    ref.check(got, ref.decode(q, k, v, table, n, **kw), finite(v), dtype)


ENDS = pytest.mark.parametrize("softcap", [1e-45, 1e-40, 1e-30, 1e-9, 2e38, 3.4e38], ids=str)


@TYPES
@ENDS
@pytest.mark.parametrize("shape", ROWS[:1] + TILES, ids=lambda s: "x".join(map(str, s)))
def test_attention_with_caps_at_the_ends_of_fp32(gpu, shape, softcap, dtype):
    """A cap as small as fp32 holds leaves the mean of the values, one as large caps nothing; a score of exactly
    zero is neither's NaN."""
    q, k, v = tokens(shape, dtype, seed=6)
    q[:, 0] = 0
    kw = {"scale": shape[5] ** -0.5, "softcap": softcap}
    ref.check(attend(q, k, v, **kw), definition(q, k, v, **kw), v, dtype)


@TYPES
@ENDS
@pytest.mark.parametrize("dims", [(64, 64), (33, 31)], ids=str)
def test_decode_with_caps_at_the_ends_of_fp32(gpu, dims, softcap, dtype):
    lens = [421, 77]
    k, v, table = paged(lens, 16, 2, *dims, dtype, seed=2)
    q = (ref.randn(2, 4, dims[0], seed=5, dtype=F32, device="cuda") * 3).to(dtype)
    q[0, 0] = 0
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = {"scale": dims[0] ** -0.5, "softcap": softcap}
    got = run_decode(q, k, v, table, n, **kw)
    sync_check()
    ref.check(got, ref.decode(q, k, v, table, n, **kw), finite(v), dtype)


@pytest.mark.parametrize("softcap", [30.0, 50.0])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("bias", [False, True], ids=["flat", "bias"])
@pytest.mark.parametrize("shape", [(1, 384, 640, 2, 1, 64, 64), (2, 512, 512, 4, 2, 128, 128), (1, 700, 700, 2, 2, 32, 128),
                                   (1, 256, 900, 4, 4, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_whole_tiles_of_ordinary_caps(gpu, shape, bias, causal, softcap):
    """Scores of standard deviation 3 under caps of 30 and 50: unmasked tiles of 128 keys in which every score is
    far enough from the cap for the tensor-core kernel's polynomial, with and without a bias."""
    q, k, v = tokens(shape, BF16, seed=11)
    kw = {"scale": shape[5] ** -0.5, "softcap": softcap, "causal": causal}
    if bias:
        kw["slopes"] = ref.alibi_slopes(shape[3], "cuda")
    ref.check(attend(q, k, v, **kw), definition(q, k, v, **kw), v, BF16)


@pytest.mark.parametrize("bias", [False, True], ids=["flat", "bias"])
@pytest.mark.parametrize("lead", [False, True], ids=["near_first", "far_first"])
def test_rows_that_meet_both_forms_of_the_cap(gpu, lead, bias):
    """Key tiles whose scores all stay below 0.8 of the cap beside tiles whose scores pass it."""
    shape = (1, 256, 768, 2, 1, 64, 64)
    q, k, v = tokens(shape, BF16, seed=21, spread=1.5)
    big = torch.arange(768, device="cuda") // 128 % 2 == int(lead)
    k[:, big] *= 4
    kw = {"scale": 0.125, "softcap": 12.0}
    y = torch.einsum("bihd,bjhd->bhij", q.double(), k.double().repeat_interleave(2, 2)).abs() * 0.125 / 12.0
    assert float(y[..., ~big].max()) < 0.79 and float(y[..., big].max()) > 1.0
    if bias:
        kw["slopes"] = ref.alibi_slopes(2, "cuda") * 0.02
    ref.check(attend(q, k, v, **kw), definition(q, k, v, **kw), v, BF16)


@TYPES
@pytest.mark.parametrize("softcap,scale", [(1e-40, 0.125), (1e-9, 0.125), (1e-6, 0.125), (1e-3, 1e3), (0.5, 1e6)], ids=str)
@pytest.mark.parametrize("shape", ROWS[:1] + TILES, ids=lambda s: "x".join(map(str, s)))
def test_scores_of_zero_under_any_cap(gpu, shape, softcap, scale, dtype):
    """Queries of zeros see the mean of the values, however large scale / softcap is; so do, nearly, queries whose
    scores stay a little below or above the cap."""
    q, k, v = tokens(shape, dtype, seed=61)
    kw = {"scale": scale, "softcap": softcap}
    for factor in (0.0, softcap / scale * 0.05, softcap / scale * 0.5):
        x = (q.float() * factor).to(dtype)
        ref.check(attend(x, k, v, **kw), definition(x, k, v, **kw), v, dtype)


@pytest.mark.parametrize("softcap", [1e4, 1e5, 1e6])
@pytest.mark.parametrize("shape", [(1, 384, 384, 2, 2, 64, 64), (2, 300, 520, 4, 2, 128, 128)], ids=lambda s: "x".join(map(str, s)))
def test_small_scores_beside_rows_at_their_cap(gpu, shape, softcap):
    """Every other query's scores lie far above a large cap, its neighbours' far below: those keep their precision."""
    q, k, v = tokens(shape, BF16, seed=71)
    q[:, 1::2] = (q[:, 1::2].float() * softcap).to(BF16)
    kw = {"scale": shape[5] ** -0.5, "softcap": softcap}
    got, want = attend(q, k, v, **kw), definition(q, k, v, **kw)
    assert torch.isfinite(got.float()).all()
    ref.check(got[:, ::2], want[:, ::2], v, BF16)
