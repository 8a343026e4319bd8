"""Norms of heads and weights whose product would leave fp32's range although the result does not."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check
from test_gpu_cache4 import DTYPES

pytestmark = pytest.mark.gpu


@DTYPES
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("D", [128, 40, 6])
@pytest.mark.parametrize("power,weight", [(60, 70), (58, 120), (-55, -90), (-58, -110), (40, -120), (-40, 120)], ids=str)
def test_large_heads_and_large_weights(gpu, power, weight, D, adjacent, dtype):
    """Heads of size 2^power, weights of 2^weight: results of 2^weight."""
    x = (ref.randn(2, 9, 3, D, seed=1, dtype=torch.float32, device="cuda") * 2.0 ** power).to(dtype)
    w = (ref.randn(D, seed=2, dtype=torch.float32, device="cuda").abs() + 0.5) * 2.0 ** weight
    half = D // 2
    freq = torch.tensor([100.0 ** (-i / half) for i in range(half)], device="cuda")
    pos = torch.arange(18, dtype=torch.int32, device="cuda").view(1, 2, 9)
    out = torch.empty_like(x)
    cb.norm_rotate(x, None, pos, cb.Rotation(freq, norm=True, eps=0.0, q_weight=w, adjacent=adjacent), out)
    sync_check()
    want, size = ref4.norm_rotate(x, pos, freq, torch.zeros(half, dtype=torch.int32), adjacent=adjacent, norm=True, eps=0.0, weight=w)
    ref4.check_rotate(out, want, size)
