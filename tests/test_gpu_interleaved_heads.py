"""Views whose heads lie between each other's: queries, keys and values of a head side by side in a token."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check
from test_gpu_cache4 import DTYPES, ints, pages4

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("D,shift", [(64, 0), (64, 1), (40, 0), (6, 0), (128, 0)], ids=str)
def test_in_place_among_values(gpu, D, shift, dtype):
    """[B, L, H, 3, D]: queries and keys turn in place, the values keep their bits; then both go into a cache and come
    back into such a buffer, and attention reads it in place."""
    B, L, H = 2, 37, 4
    flat = ref.randn(B * L * H * 3 * D + 8, seed=1, dtype=dtype, device="cuda")
    row = flat[shift:shift + B * L * H * 3 * D].view(B, L, H, 3, D)
    q, k, v = row.unbind(3)
    was = [t.clone() for t in (q, k, v)]
    half = D // 2
    freq = torch.tensor([100.0 ** (-i / half) for i in range(half)], device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda").expand(1, B, L).contiguous()
    cb.norm_rotate(q, k, pos, cb.Rotation(freq, norm=True))
    sync_check()
    assert torch.equal(v, was[2])
    for got, x in ((q, was[0]), (k, was[1])):
        want, size = ref4.norm_rotate(x, pos, freq, torch.zeros(half, dtype=torch.int32), norm=True)
        ref4.check_rotate(got, want, size)
    cache = cb.PagedCache4(*pages4(B * 3, 16, H, D, D), torch.arange(B * 3, dtype=torch.int32, device="cuda").view(B, 3), dim_k=D, dim_v=D)
    cb.cache4_append(k, v, cache, ints([0] * B))
    back = torch.full((B, L, H, 3, D), 7.0, dtype=dtype, device="cuda")
    cb.cache4_read(cache, back[:, :, :, 0], back[:, :, :, 2])
    sync_check()
    assert (back[:, :, :, 1] == 7).all()
    for got, x in ((back[:, :, :, 0], k), (back[:, :, :, 2], v)):
        assert torch.equal(got.cpu(), ref4.values(*ref4.store(x), D).to(dtype))
    cb.attention(q, k, v, back[:, :, :, 1], cb.Score(D ** -0.5))
    sync_check()
    ref.check(back[:, :, :, 1], ref.attention(q, k, v, D ** -0.5), v, dtype)
