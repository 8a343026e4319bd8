"""Attention over a 4-bit cache at drawn sizes, rules and spreads of scales, against the definition in 64 bits and the bounds
of test_gpu_cache4_rounding (steps of 16 tokens in full), with the definition's sums on the GPU."""
import math
import random

import pytest
import torch

from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check
from test_gpu_cache4 import BF16, DTYPES, F32, ints, pages4

pytestmark = pytest.mark.gpu


def groups(x, dim):
    """[..., dim] -> [..., groups]: each group's largest."""
    return torch.nn.functional.pad(x.abs(), (0, -dim % 32)).unflatten(-1, (-1, 32)).amax(-1)


@DTYPES
@pytest.mark.parametrize("seed", range(150))
def test_drawn(gpu, seed, dtype):
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    dk, dv = rng.choice(((32, 64), (64, 64), (96, 96), (128, 128), (40, 72), (64, 128), (8, 120), (128, 32)))
    H, G, B = rng.choice((1, 2, 4)), rng.choice((1, 2, 4, 5, 8, 12)), rng.choice((1, 2, 3, 8, 40))
    page, n = rng.choice((16, 20, 32, 64, 128)), int(math.exp(rng.uniform(0, math.log(10000 if B < 4 else 2000))))
    lens = [min(n, int(n * rng.random() ** 0.5) + rng.randint(0, 2)) for _ in range(B)]
    tokens_first, wide = rng.random() < 0.3, rng.choice((0, 3000))
    per = (n + page - 1) // page

    def tokens(dim, by_group, by_token, rare):
        e = randn(B, n, H, (dim + 31) // 32) * by_group
        if rare:
            e = e * (torch.rand(e.shape, generator=g, device="cuda") < 0.02)
        e = (e + randn(B, n, H, 1) * by_token).clamp(-100, 100)
        return randn(B, n, H, dim) * torch.exp2(e).repeat_interleave(32, -1)[..., :dim]

    x = tokens(dk, rng.choice((0.0, 1.0, 3.0)), rng.choice((0.0, 1.0)), False)
    y = tokens(dv, rng.choice((0.0, 0.0, 1.0, 4.0, 20.0)), rng.choice((0.0, 2.0, 20.0)), rng.random() < 0.5)
    if rng.random() < 0.2:
        y[..., :32] = 0
    if rng.random() < 0.2:
        y[:, :n // 2] = 0
    table = torch.full((B, per + wide), -1, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.randperm(B * per + 1, generator=g, device="cuda")[:B * per].view(B, per).int()
    cache = cb.PagedCache4(*pages4(B * per + 1, page, H, dk, dv, tokens_first), table, dim_k=dk, dim_v=dv)
    cb.cache4_append(x.to(BF16), y.to(BF16), cache, ints([0] * B))
    k, v = torch.empty(B, n, H, dk, device="cuda"), torch.empty(B, n, H, dv, device="cuda")
    cb.cache4_read(cache, k, v)
    q = randn(B, H * G, dk) * rng.choice((0.0, 1.0, 3.0, 10.0))
    if rng.random() < 0.3:
        q = q * torch.exp2(randn(B, H * G, (dk + 31) // 32) * rng.choice((2.0, 8.0))).repeat_interleave(32, -1)[..., :dk]
    q = q.to(dtype)
    scale, cap = dk ** -0.5, rng.choice((0.0, 0.0, 30.0, 3.0))
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / (H * G)) for h in range(H * G)], device="cuda") if rng.random() < 0.3 else None
    first = ints([rng.randint(0, max(m, 1)) // rng.choice((1, 3, 50)) for m in lens]) if rng.random() < 0.4 else None
    ws = torch.empty(cb.attention_decode4_workspace(q, cache), dtype=torch.uint8, device="cuda")
    out = [torch.full((B, H * G, dv), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    for o in out:
        cb.attention_decode4(q, cache, ints(lens), o, ws, scale=scale, softcap=cap, slopes=slopes, first=first)
    sync_check()
    assert torch.equal(out[0], out[1])  # NaN is no number's equal

    k, v, q, j = k.double(), v.double(), q.double().view(B, H, G, dk), torch.arange(n, device="cuda")
    s = torch.einsum("bhgd,bnhd->bhgn", q, k) * scale
    s = cap * torch.tanh(s / cap) if cap else s
    if slopes is not None:
        s = s - slopes.double().view(1, H, G, 1) * (ints(lens).view(B, 1, 1, 1) - 1 - j).double()
    keep = j.view(1, n) < ints(lens).view(B, 1)
    if first is not None:
        keep &= j.view(1, n) >= first.view(B, 1)
    p = torch.nan_to_num(torch.softmax(s.masked_fill(~keep[:, None, None], -math.inf), -1), 0.0)
    want, total = torch.einsum("bhgn,bnhd->bhgd", p, v), torch.einsum("bhgn,bnhd->bhgd", p, v.abs())
    size = groups(v, dv) * (1.01 / 7)  # scales, bf16's rounding up
    cut = torch.zeros(B, H, G, size.shape[-1], dtype=torch.float64, device="cuda")
    for lo in range(0, n, 16):
        cut += torch.einsum("bhgn,bnhe->bhgne", p[..., lo:lo + 16], size[:, lo:lo + 16]).amax(3)

    def dims(t):
        return t.repeat_interleave(32, -1)[..., :dv]

    # of a score: its products' cuts (fp32: roundings), the bias's and the cap's roundings
    error = scale * torch.einsum("bhge,bhe->bhg", groups(q, dk), groups(k, dk).amax(1) * (1.01 / 7))
    error = error * (34 * 2.0 ** -14 if dtype == BF16 else 32 * 15 * 2.0 ** -24) + 2.0 ** -18
    error = error + (2.0 ** -22 * n if slopes is not None else 0.0) + (1e-5 if cap else 0.0)
    off = torch.expm1(2 * error.clamp(max=30))[..., None]  # finite: times sums of 0 it is 0
    # a weight of less than 2^-80 of the largest is none
    bound = off * (total + want.abs()) + 2.0 ** -80 * dims(size.amax(1)[:, :, None]) + 1e-37
    if dtype == F32:  # products below 2^-24 of a group's largest
        bound = bound + 2.0 ** -17 * total + 2.0 ** -23 * want.abs() + dims(cut) * 17 * 4 * 2.0 ** -26
    else:
        bound = bound + (1 + off) * (3 * 2.0 ** -11 * 1.02 * total + dims(cut) * 17 * 4 * 2.0 ** -14) + 2.0 ** -8 * want.abs()
    over = float(((out[0].double().view(B, H, G, dv) - want).abs() / bound).max())
    assert over <= 1.0, over
