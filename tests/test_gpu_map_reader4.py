"""MapReader with norms and rotary positions of its heads, and with a cache in 4 bits, against the definitions in 64
bits; each part is fed the GPU's own input."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb, synthetic
from conv_bn_activation_gb300.nets import MapReader
from gpu_util import sync_check

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def places(axes, hw, step=None):
    """Positions [axes, 1, L] of the map's tokens, or of the step-th token after it."""
    H, W = hw
    if axes == 0:
        return None
    if step is not None:
        return torch.full((axes, 1, 1), step + (max(hw) if axes > 1 else H * W))
    if axes == 1:
        return torch.arange(H * W).view(1, 1, -1)
    at = torch.tensor([[0, y, x] for y in range(H) for x in range(W)]).T
    return at[3 - axes:].reshape(axes, 1, -1)


@DTYPES
@pytest.mark.parametrize("bits", [None, 4])
@pytest.mark.parametrize("hw,heads,kv_heads,dim,axes,norm,adjacent", [
    ((5, 7), 8, 2, 32, 3, True, False), ((9, 4), 4, 4, 64, 2, False, True), ((3, 3), 4, 1, 128, 1, True, True), ((4, 6), 2, 2, 40, 0, True, False),
    ((2, 2), 8, 2, 32, 0, False, False)], ids=str)
def test_parts_against_definition(gpu, hw, heads, kv_heads, dim, axes, norm, adjacent, bits, dtype):
    B, C, steps = 2, 64, 3
    p = synthetic.map_reader_params(C, heads, kv_heads, dim, axes=axes, norm=norm, adjacent=adjacent)
    plain = {k: v for k, v in p.items() if k not in ("rope", "q_norm", "k_norm")}
    net, raw = MapReader(p, B, hw, steps, dtype=dtype, cache_bits=bits), MapReader(plain, B, hw, steps, dtype=dtype)

    def turned(x, name, pos):
        rope = p.get("rope")
        kw = {} if rope is None else {"pos": pos.expand(axes, B, -1), "freq": torch.tensor(rope["freq"]), "axis": torch.tensor(rope["axis"]),
                                      "adjacent": adjacent}
        return ref4.norm_rotate(x, norm=norm, weight=torch.tensor(p[name]) if norm else None, **kw)

    def seen(k, v):  # as the cache holds them
        return [ref4.values(*ref4.store(t), dim) if bits == 4 else t.float().cpu() for t in (k, v)]

    for _ in range(2):  # a second map starts over
        x = ref.randn(B, *hw, C, seed=1, dtype=dtype, device="cuda")
        net.read(x), raw.read(x)
        sync_check()
        q, k, v = (t.clone() for t in net._split(net.map_qkv))
        for got, was, name in zip((q, k), raw._split(raw.map_qkv), ("q_norm", "k_norm")):
            ref4.check_rotate(got, *turned(was, name, places(axes, hw)))
        assert torch.equal(v, raw._split(raw.map_qkv)[2])
        ref.check(net.map_ctx.view(*q.shape), ref.attention(q, k, v, dim ** -0.5), v, dtype)
        ks, vs = ([t] for t in seen(k, v))
        for i in range(steps):
            tok = ref.randn(B, C, seed=30 + i, dtype=dtype, device="cuda")
            net.step(tok), raw.step(tok)
            sync_check()
            q, k, v = net._split(net.tok_qkv)
            for got, was, name in zip((q, k), raw._split(raw.tok_qkv), ("q_norm", "k_norm")):
                ref4.check_rotate(got, *turned(was, name, places(axes, hw, i)))
            for kept, t in zip((ks, vs), seen(k, v)):
                kept.append(t)
            kk, vv = torch.cat(ks, 1), torch.cat(vs, 1)
            ref.check(net.tok_ctx.view(B, 1, heads, dim), ref.attention(q, kk, vv, dim ** -0.5), vv, dtype)


@DTYPES
def test_captured_steps_match_eager(gpu, dtype):
    B, hw, C = 2, (9, 11), 64
    p = synthetic.map_reader_params(C, axes=3, norm=True)
    x = ref.randn(B, *hw, C, seed=2, dtype=dtype, device="cuda")
    eager, net = (MapReader(p, B, hw, 8, dtype=dtype, cache_bits=4) for _ in range(2))
    toks = [ref.randn(B, C, seed=30 + i, dtype=dtype, device="cuda") for i in range(4)]
    want = [eager.read(x).clone()] + [eager.step(t).clone() for t in toks]
    tok = toks[0].clone()
    net.read(x)
    net.step(tok)  # once outside the graph
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        net.step(tok)
    got = [net.read(x).clone()]
    for t in toks:
        tok.copy_(t)
        g.replay()
        got.append(net.tok_out.view(B, C).clone())
    sync_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_step_past_the_room_is_refused(gpu):
    net = MapReader(synthetic.map_reader_params(axes=2), 2, (4, 4), 1, page=16, dtype=BF16, cache_bits=4)
    x, tok = ref.randn(2, 4, 4, 64, seed=1, dtype=BF16, device="cuda"), ref.randn(2, 64, seed=2, dtype=BF16, device="cuda")
    net.read(x)
    for _ in range(16):
        net.step(tok)
    with pytest.raises(ValueError):
        net.step(tok)
    sync_check()
    with pytest.raises(ValueError):
        MapReader(synthetic.map_reader_params(), 2, (4, 4), 1, cache_bits=8)
    with pytest.raises(ValueError):
        MapReader(synthetic.map_reader_params(axes=4), 2, (4, 4), 1)
    assert cb.get_device_error() == cb.OK
