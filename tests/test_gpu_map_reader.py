"""MapReader: attention over a feature map, its cache, and steps that read it, against the oracle's convs and
the definition of attention in 64 bits.  Each layer is fed the GPU's own input, so its own tolerance holds."""
import pytest
import torch

import attention_ref as ref
from conv_bn_activation_gb300 import synthetic
from conv_bn_activation_gb300.nets import MapReader
from gpu_util import TOL_BF16, TOL_TF32, rel_err, sync_check

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.detach().float().cpu().numpy()


def tokens(net, batch, channels, count, dtype):
    return [ref.randn(batch, channels, seed=30 + i, dtype=dtype, device="cuda") for i in range(count)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("batch,hw,heads,kv_heads,dim", [(3, (5, 7), 8, 2, 32), (2, (20, 20), 4, 4, 64), (1, (1, 1), 8, 1, 32)])
def test_layers_against_definition(gpu, orc, dtype, batch, hw, heads, kv_heads, dim):
    C, steps = 64, 3
    p = synthetic.map_reader_params(C, heads, kv_heads, dim)
    net = MapReader(p, batch, hw, steps, dtype=dtype)
    tol = TOL_BF16 if dtype == BF16 else TOL_TF32
    x = ref.randn(batch, *hw, C, seed=1, dtype=dtype, device="cuda")
    y = net.read(x)
    sync_check()

    def conv(a, name, residual=None):
        more = {} if residual is None else dict(residual=host(residual), res_mode=orc.RES_POST_ACT)
        return orc.conv_bn_act(host(a), p[name + "_w"], p[name + "_bn"], stride=1, pad=0, act=orc.ACT_NONE, **more)

    assert rel_err(host(net.map_qkv), conv(x, "qkv")) <= tol
    q, k, v = (t.clone() for t in net._split(net.map_qkv))
    ref.check(net.map_ctx.view(*q.shape), ref.attention(q, k, v, dim ** -0.5), v, dtype)
    assert rel_err(host(y), conv(net.map_ctx, "out", x)) <= tol
    for i, tok in enumerate(tokens(net, batch, C, steps, dtype)):
        z = net.step(tok)
        sync_check()
        assert net.length.tolist() == [hw[0] * hw[1] + i + 1] * batch
        t = tok.view(batch, 1, 1, C)
        assert rel_err(host(net.tok_qkv), conv(t, "qkv")) <= tol
        qt, kt, vt = net._split(net.tok_qkv)
        k, v = torch.cat([k, kt], 1), torch.cat([v, vt], 1)
        # the step sees all keys so far: the attention of its query over the contiguous rows
        ref.check(net.tok_ctx.view(batch, 1, heads, dim), ref.attention(qt, k, v, dim ** -0.5), v, dtype)
        assert rel_err(host(z).reshape(batch, 1, 1, C), conv(net.tok_ctx, "out", t)) <= tol


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_graph_and_stream_match_eager(gpu, dtype):
    """A captured step replayed, and a run on another stream, give the eager run's bits."""
    B, hw, C = 2, (9, 11), 64
    p = synthetic.map_reader_params(C)
    x = ref.randn(B, *hw, C, seed=2, dtype=dtype, device="cuda")
    nets = [MapReader(p, B, hw, 8, dtype=dtype) for _ in range(3)]
    toks = tokens(nets[0], B, C, 4, dtype)
    want = [nets[0].read(x).clone()] + [nets[0].step(t).clone() for t in toks]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    read = nets[1].read(x, stream=s)
    with torch.cuda.stream(s):
        got = [read.clone()]
    for t in toks:
        z = nets[1].step(t, stream=s)
        with torch.cuda.stream(s):
            got.append(z.clone())
    s.synchronize()
    sync_check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    net, tok = nets[2], toks[0].clone()
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


@pytest.mark.parametrize("hw,steps,page", [((4, 4), 0, 16), ((3, 3), 3, 4), ((5, 7), 2, 16)], ids=str)
def test_a_step_past_the_room_is_refused(gpu, hw, steps, page):
    """As many steps as the pages hold, then ValueError and nothing changed; a new map starts over."""
    net = MapReader(synthetic.map_reader_params(), 2, hw, steps, page=page, dtype=BF16)
    x, tok = ref.randn(2, *hw, 64, seed=1, dtype=BF16, device="cuda"), ref.randn(2, 64, seed=2, dtype=BF16, device="cuda")
    n = hw[0] * hw[1]
    room = -(-(n + steps) // page) * page - n
    assert room >= steps
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        net.read(x, stream=stream)
        for _ in range(room):
            net.step(tok, stream=stream)
        torch.cuda.synchronize()
        before = net.tok_out.clone()
        with pytest.raises(ValueError):
            net.step(tok, stream=stream)
        sync_check()
        assert net.length.tolist() == [n + room] * 2 and torch.equal(net.tok_out, before)


def test_the_room_leaves_captured_calls_alone(gpu):
    """Capturing a step takes no room; after a captured read, whose replays start over, no step is refused."""
    hw, page = (4, 4), 16
    net = MapReader(synthetic.map_reader_params(), 2, hw, 16, page=page, dtype=BF16)
    x, tok = ref.randn(2, *hw, 64, seed=1, dtype=BF16, device="cuda"), ref.randn(2, 64, seed=2, dtype=BF16, device="cuda")
    net.read(x)
    net.step(tok)
    for _ in range(20):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            net.step(tok)
    for _ in range(15):
        net.step(tok)
    with pytest.raises(ValueError):
        net.step(tok)
    read = torch.cuda.CUDAGraph()
    with torch.cuda.graph(read):
        net.read(x)
    for _ in range(3):
        read.replay()
        for _ in range(16):
            net.step(tok)
    sync_check()
    assert net.length.tolist() == [32, 32]
