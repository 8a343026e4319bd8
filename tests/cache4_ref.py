"""The 4-bit cache and the head rotations from their definitions, in 64 bits or exactly on the CPU: the reference of
their tests."""
import numpy as np
import torch

GROUP = 32


def scales_per_row(dim):
    return 2 * ((dim + 63) // 64)


def store(x):
    """Codes' bytes [..., (dim + 1) // 2] and scales [..., scales_per_row(dim)] of rows x [..., dim]."""
    x = x.detach().cpu().double()
    dim = x.shape[-1]
    codes = torch.zeros(*x.shape[:-1], dim + dim % 2, dtype=torch.int64)
    scales = torch.zeros(*x.shape[:-1], scales_per_row(dim), dtype=torch.float64)
    for g in range((dim + GROUP - 1) // GROUP):
        y = x[..., g * GROUP:(g + 1) * GROUP]
        top = y.abs().amax(-1) / 7
        # bf16: 8 significant bits, and no finer than 2^-133
        _, e = torch.frexp(top)
        unit = torch.from_numpy(np.ldexp(1.0, (e.clamp(min=-125) - 8).numpy()))
        s = torch.round(top / unit) * unit  # torch.round takes ties to even
        bad = ~torch.isfinite(y).all(-1)
        some = (s > 0) & ~bad
        c = torch.round(y / torch.where(some, s, torch.ones_like(s))[..., None]).clamp(-7, 7)
        codes[..., g * GROUP:g * GROUP + y.shape[-1]] = torch.where(some[..., None], c, torch.zeros_like(c)).long()
        scales[..., g] = torch.where(bad, torch.full_like(s, float("nan")), s)
    nibble = codes + 8
    return (nibble[..., 0::2] | (nibble[..., 1::2] << 4)).to(torch.uint8), scales.float().to(torch.bfloat16)


def values(codes, scales, dim):
    """float32 (exact: 11 bits) values of stored rows."""
    codes, scales = codes.cpu(), scales.cpu().float()
    nibble = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)[..., :dim].float() - 8
    return nibble * scales.repeat_interleave(GROUP, dim=-1)[..., :dim]


def angles(pos, freq, axis):
    """pos int [axes, B, L], freq fp32 [n], axis int [n] -> float64 [B, L, n], whole turns taken off.  The product
    has 55 bits: more than a double's 53, fewer than a long double's 64."""
    at = pos.cpu()[axis.cpu().long()].permute(1, 2, 0).numpy().astype(np.longdouble)
    turn = np.longdouble("6.283185307179586476925286766559005768")
    a = at * freq.cpu().numpy().astype(np.longdouble)
    return torch.from_numpy(np.asarray(a - np.rint(a / turn) * turn, dtype=np.float64))


def norm_rotate(x, pos=None, freq=None, axis=None, adjacent=False, norm=False, eps=1e-6, weight=None):
    """float64 result, and per element |y1| + |y2| of the pair (|y| of what does not turn)."""
    y = x.detach().cpu().double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.cpu().double()
    out, size = y.clone(), y.abs().clone()
    if freq is not None:
        n = freq.shape[0]
        ang = angles(pos, freq, torch.zeros(n) if axis is None else axis)[:, :, None]
        i = torch.arange(n)
        d1, d2 = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        y1, y2, co, si = y[..., d1], y[..., d2], torch.cos(ang), torch.sin(ang)
        out[..., d1], out[..., d2] = y1 * co - y2 * si, y2 * co + y1 * si
        size[..., d1] = size[..., d2] = y1.abs() + y2.abs()
    return out, size


# Roundings of a normed and turned element, in units of 2^-24 of |y1| + |y2|: the mean of squares, at most 128 terms in
# 32 lanes' sums of 4 to 16 and 5 levels of a tree, with its division and eps, 23 and half of that under the root; rsqrtf
# 4; the two products 2; the angle's conversion to 24 bits in half turns, pi / 2, and sincospif 2; the turn 3.
ROTATE_STEPS = 25


def check_rotate(got, ref, size):
    got = got.detach()
    dtype, got = got.dtype, got.cpu().double()
    bound = ROTATE_STEPS * 2.0 ** -24 * size + torch.finfo(dtype).eps / 2 * ref.abs() * 1.01 + 1e-37
    assert got.shape == ref.shape and torch.isfinite(got).all()
    over = float(((got - ref).abs() / bound).max()) if got.numel() else 0.0
    assert over <= 1.0, over
