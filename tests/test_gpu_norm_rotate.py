"""cb_norm_rotate on the GPU against its definition in 64 bits."""
import pytest
import torch

import attention_ref as ref
import cache4_ref as ref4
from conv_bn_activation_gb300 import binding as cb
from gpu_util import sync_check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


def freqs(n, base=10000.0, device="cuda"):
    return torch.tensor([base ** (-i / max(n, 1)) for i in range(n)], dtype=F32, device=device)


def positions(axes, B, L, seed=0, top=5000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-50, top, (axes, B, L), generator=g).to(torch.int32).cuda()


def both(q, k, pos, rule, q_out=None, k_out=None):
    """Runs the call and checks both results; the inputs are those before it."""
    q0, k0 = q.clone(), None if k is None else k.clone()
    got = cb.norm_rotate(q, k, pos, rule, q_out, k_out)
    sync_check()
    for y, x, w in ((got[0], q0, rule.q_weight), (got[1], k0, rule.k_weight)):
        if x is not None:
            ref4.check_rotate(y, *ref4.norm_rotate(x, pos, rule.freq, rule.axis, rule.adjacent, rule.norm, rule.eps, w))


CASES = [  # B, L, Hq, Hkv, dim, pairs, axes
    (1, 1, 1, 1, 128, 64, 1), (64, 1, 32, 8, 128, 64, 3), (2, 400, 8, 2, 32, 16, 2), (3, 7, 5, 1, 64, 16, 3), (1, 33, 4, 4, 96, 48, 2),
    (2, 5, 3, 3, 128, 32, 1), (1, 9, 2, 1, 40, 20, 2), (2, 3, 10, 2, 72, 18, 3), (1, 4, 2, 2, 7, 2, 1), (5, 2, 1, 1, 2, 1, 1),
    (1, 6, 3, 1, 16, 8, 8), (2, 300, 40, 8, 64, 0, 1), (1, 2, 2, 1, 1, 0, 1), (1, 1031, 16, 16, 80, 24, 3)]


@DTYPES
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_definition(gpu, case, norm, adjacent, dtype):
    B, L, Hq, Hkv, dim, n, axes = CASES[case]
    row = ref.randn(B, L, (Hq + 2 * Hkv) * dim, seed=case, dtype=dtype, device="cuda") * 3
    q, k, _ = torch.split(row, [Hq * dim, Hkv * dim, Hkv * dim], dim=-1)  # slices of a projection's output
    q, k = q.unflatten(-1, (Hq, dim)), k.unflatten(-1, (Hkv, dim))
    w = [ref.randn(dim, seed=case + i, dtype=F32, device="cuda") for i in range(2)] if norm else [None, None]
    axis = torch.tensor([(i * 5) % axes for i in range(n)], dtype=torch.int32, device="cuda") if axes > 1 else None
    rule = cb.Rotation(freqs(n) if n else None, axis=axis, axes=axes, adjacent=adjacent, norm=norm, eps=1e-6, q_weight=w[0], k_weight=w[1])
    pos = positions(axes, B, L, case) if n else None
    out = [torch.full((B, L, h, dim), float("nan"), dtype=dtype, device="cuda") for h in (Hq, Hkv)]
    both(q, k, pos, rule, *out)
    rest = row[..., (Hq + Hkv) * dim:].clone()
    both(q, k, pos, rule)  # in place
    assert torch.equal(row[..., (Hq + Hkv) * dim:], rest) and torch.equal(q, out[0]) and torch.equal(k, out[1])


@DTYPES
def test_queries_alone_and_weight_of_one(gpu, dtype):
    q = ref.randn(2, 5, 3, 64, seed=1, dtype=dtype, device="cuda")
    both(q, None, positions(1, 2, 5), cb.Rotation(freqs(32), norm=True, k_weight=torch.zeros(64, device="cuda")))
    k = ref.randn(2, 5, 1, 64, seed=2, dtype=dtype, device="cuda")
    both(q, k, None, cb.Rotation(norm=True, eps=0.5, k_weight=ref.randn(64, seed=3, dtype=F32, device="cuda")))


@pytest.mark.parametrize("dim", [128, 36])
def test_far_positions(gpu, dim):
    """The farthest positions, either sign; frequencies up to 1, some of them tiny or negative."""
    n = dim // 2
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -777777777, 131071, 0, 1, -1], dtype=torch.int32, device="cuda").view(1, 1, 8)
    freq = freqs(n)
    freq[3], freq[4], freq[5], freq[6] = -0.7, 0.0, 1e-42, 1e-10
    q, k = (ref.randn(1, 8, h, dim, seed=h, dtype=F32, device="cuda") for h in (3, 1))
    both(q, k, pos, cb.Rotation(freq))


def test_large_frequencies(gpu):
    """Frequencies of many turns per position: off by |pos| freq 2^-65 turns."""
    freq = torch.tensor([3.25, 1000.5, 65535.0, 2.0 ** 23], dtype=F32, device="cuda")
    pos = torch.tensor([1, 2, 3, -7, 1000], dtype=torch.int32, device="cuda").view(1, 1, 5)
    q = ref.randn(1, 5, 2, 8, seed=1, dtype=F32, device="cuda")
    both(q, None, pos, cb.Rotation(freq))


@DTYPES
def test_strides_and_broadcasts(gpu, dtype):
    """Head-major heads, a query row that every sequence shares, positions of one row for all, odd offsets."""
    B, L, H, D = 3, 6, 4, 64
    q = ref.randn(B, H, L, D + 3, seed=1, dtype=dtype, device="cuda")[..., 1:D + 1].transpose(1, 2)
    k = ref.randn(1, L, 2, D, seed=2, dtype=dtype, device="cuda").expand(B, L, 2, D)
    buf = torch.full((B, L + 1, H + 2, D + 1), 7.0, dtype=dtype, device="cuda")
    pos = positions(2, 1, L).expand(2, B, L)
    rule = cb.Rotation(freqs(32), axis=torch.arange(32, device="cuda", dtype=torch.int32) % 2, axes=2, norm=True)
    k_out = torch.empty(B, L, 2, D, dtype=dtype, device="cuda")
    both(q, k, pos, rule, buf[:, 1:, 1:-1, 1:], k_out)
    assert (buf[:, 0] == 7).all() and (buf[:, :, 0] == 7).all() and (buf[:, :, -1] == 7).all() and (buf[..., 0] == 7).all()


@DTYPES
def test_rows_of_zeros_and_of_large_values(gpu, dtype):
    q = torch.zeros(1, 3, 2, 64, dtype=dtype, device="cuda")
    q[0, 1] = 2.0 ** 50
    q[0, 2] = 2.0 ** -60
    both(q, None, positions(1, 1, 3), cb.Rotation(freqs(32), norm=True, eps=1e-6))
    assert (q[0, 0] == 0).all()


@DTYPES
def test_infinities_and_nan_stay_in_their_row(gpu, dtype):
    q = ref.randn(2, 4, 2, 128, seed=1, dtype=dtype, device="cuda")
    q[0, 1, 0, 5], q[1, 2, 1, 9] = float("nan"), float("inf")
    rule = cb.Rotation(freqs(64), norm=True)
    pos = positions(1, 2, 4)
    out = torch.empty_like(q)
    cb.norm_rotate(q, None, pos, rule, out)
    sync_check()
    bad = torch.zeros(2, 4, 2, dtype=torch.bool)
    bad[0, 1, 0] = bad[1, 2, 1] = True
    assert torch.equal(~torch.isfinite(out.float()).all(-1).cpu(), bad)
    good = torch.where(torch.isfinite(q), q, torch.zeros_like(q))
    want, size = ref4.norm_rotate(good, pos, rule.freq, None, norm=True)
    ref4.check_rotate(out.cpu()[~bad], want[~bad], size[~bad])


@DTYPES
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("dim,rotary", [(128, 64), (128, 0), (96, 32), (40, 20), (36, 12), (7, 4)], ids=str)
def test_infinities_behind_what_turns_touch_no_other_dim(gpu, dim, rotary, norm, adjacent, dtype):
    """Dims behind the turning ones stay y, and y of a row with an infinity is 0 but there."""
    q = ref.randn(1, 3, 4, dim, seed=1, dtype=dtype, device="cuda")
    far = [d for d in (rotary, rotary + 2, dim - 1) if d < dim]
    odd = q.clone()
    for d, x in zip(far, (float("inf"), -float("inf"), float("inf") if norm else float("nan"))):
        odd[0, 1, 2, d] = x
    rule = cb.Rotation(freqs(rotary // 2) if rotary else None, adjacent=adjacent, norm=norm)
    pos = positions(1, 1, 3) if rotary else None
    out = torch.empty_like(q)
    cb.norm_rotate(odd, None, pos, rule, out)
    sync_check()
    rest = [d for d in range(dim) if d not in far]
    row = out[0, 1, 2].clone()
    if norm:
        assert torch.isnan(row[far]).all() and (row[rest] == 0).all()
        out[0, 1, 2] = odd[0, 1, 2] = 0
    else:
        assert torch.equal(row[far].nan_to_num(7.0, 8.0, 9.0), odd[0, 1, 2, far].nan_to_num(7.0, 8.0, 9.0))
        out[0, 1, 2, far] = odd[0, 1, 2, far] = 0
    ref4.check_rotate(out, *ref4.norm_rotate(odd, pos, rule.freq, None, adjacent, norm))


@DTYPES
@pytest.mark.parametrize("dim", [64, 7])
def test_weights_are_the_norms_alone(gpu, dim, dtype):
    """The C struct may hold weights that norm = 0 does not ask for."""
    q = ref.randn(2, 3, 4, dim, seed=1, dtype=dtype, device="cuda")
    w = torch.full((dim,), 3.0, device="cuda")
    rule = cb.Rotation(norm=True, q_weight=w)
    packed = bytes(4) + rule.view(2, 3, dim, None, q.get_device())[4:]
    out = torch.empty_like(q)
    assert cb.load().cb_norm_rotate(cb.heads(q), None, packed, cb.heads(out), None, torch.cuda.current_stream().cuda_stream) == cb.OK
    sync_check()
    assert torch.equal(out, q)


def test_bad_pairs_do_not_turn_and_are_reported(gpu):
    q = ref.randn(1, 3, 2, 64, seed=1, dtype=F32, device="cuda")
    freq, pos = freqs(32), positions(2, 1, 3)
    axis = torch.arange(32, device="cuda", dtype=torch.int32) % 2
    axis[4], axis[40 - 32] = 2, -1
    freq[9], freq[10] = float("nan"), float("inf")
    out = torch.empty_like(q)
    cb.norm_rotate(q, None, pos, cb.Rotation(freq, axis=axis, axes=2), out)
    assert cb.get_device_error() == cb.ERR_INVALID_ARG and cb.get_device_error() == cb.OK
    still = [4, 8, 9, 10]
    freq[still], axis[still] = 0.0, 0
    ref4.check_rotate(out, *ref4.norm_rotate(q, pos, freq, axis))
    assert torch.equal(out[..., still], q[..., still])


def test_no_tokens(gpu):
    rule = cb.Rotation(freqs(32))
    for B, L in ((0, 4), (3, 0)):
        q = torch.empty(B, L, 2, 64, device="cuda")
        cb.norm_rotate(q, q[:, :, :1].clone(), torch.empty(1, B, L, dtype=torch.int32, device="cuda"), rule)
    sync_check()


def test_wide_offsets(gpu):
    """Sequences more than 2^31 elements apart."""
    stride = (1 << 31) + 4096
    flat = torch.empty(stride + 4096, dtype=BF16, device="cuda")
    q = flat.as_strided((2, 3, 2, 64), (stride, 128, 64, 1))
    q.copy_(ref.randn(2, 3, 2, 64, seed=1, dtype=BF16, device="cuda"))
    both(q, None, positions(1, 2, 3), cb.Rotation(freqs(32), norm=True))


def test_same_result_alone_and_among_others(gpu):
    """A token's result depends on nothing else of the call, whichever kernel and split its size selects."""
    q = ref.randn(1, 2000, 32, 128, seed=1, dtype=BF16, device="cuda")
    pos = positions(1, 1, 2000)
    rule = cb.Rotation(freqs(64), norm=True)
    whole, one = torch.empty_like(q), torch.empty_like(q[:, :1])
    cb.norm_rotate(q, None, pos, rule, whole)
    for t in (0, 7, 1999):
        cb.norm_rotate(q[:, t:t + 1], None, pos[:, :, t:t + 1], rule, one)
        sync_check()
        assert torch.equal(one[:, 0], whole[:, t])


def test_captured_and_on_another_stream(gpu):
    q, k = (ref.randn(4, 1, h, 64, seed=h, dtype=BF16, device="cuda") for h in (8, 2))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pos, rule = positions(1, 4, 1), cb.Rotation(freqs(32), norm=True)
    s = torch.cuda.Stream()
    cb.norm_rotate(q, k, pos, rule, qo, ko, stream=s)
    s.synchronize()
    want = qo.clone(), ko.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cb.norm_rotate(q, k, pos, rule, qo, ko)
    for shift in (0, 3):
        pos.add_(shift)
        qo.zero_(), ko.zero_()
        g.replay()
        sync_check()
        ref4.check_rotate(qo, *ref4.norm_rotate(q, pos, rule.freq, None, norm=True))
        if shift == 0:
            assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


@DTYPES
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("dim,rotary", [(128, 128), (96, 32), (64, 64), (40, 40), (24, 12), (36, 20), (12, 4)], ids=str)
@pytest.mark.parametrize("shift", [0, 2, 4, 1])
def test_pieces_of_every_size(gpu, shift, dim, rotary, adjacent, dtype):
    """Rows at 16, 8, 4 and 2 bytes, and dims that halve into pieces of those."""
    B, L, H = 2, 19, 3
    buf = ref.randn(B, L, 2 * H, dim + 4, seed=1, dtype=dtype, device="cuda")
    q, k = buf[:, :, :H, shift:dim + shift] if shift else buf[:, :, :H, :dim], buf[:, :, H:, shift:dim + shift]
    w = [ref.randn(dim, seed=i, dtype=F32, device="cuda") for i in range(2)]
    rule = cb.Rotation(freqs(rotary // 2), adjacent=adjacent, norm=True, q_weight=w[0], k_weight=w[1])
    rest = [buf[..., :shift].clone(), buf[..., dim + shift:].clone()]
    both(q, k, positions(1, B, L), rule)
    assert torch.equal(buf[..., :shift], rest[0]) and torch.equal(buf[..., dim + shift:], rest[1])
