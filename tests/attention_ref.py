"""Attention from its definition, in 64 bits on the CPU: the reference of the attention tests."""
import torch


def softmax_rows(s, keep, v):
    """Rows of softmax(s over keep) @ v; a row that keeps nothing is zero.  Dropped keys take no part."""
    out = torch.zeros(s.shape[0], v.shape[1], dtype=torch.float64)
    for i in range(s.shape[0]):
        idx = keep[i].nonzero()[:, 0]
        if idx.numel():
            p = torch.softmax(s[i, idx], dim=0)
            out[i] = p @ v[idx]
    return out


def attention(q, k, v, scale, softcap=0.0, slopes=None, causal=False, q_offset=0, prefix_len=None, kv_len=None,
              doc_q=None, doc_k=None):
    """q [B, Lq, Hq, Dk], k [B, Lk, Hkv, Dk], v [B, Lk, Hkv, Dv] (any device and dtype) -> float64 CPU."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    (B, Lq, Hq, _), (_, Lk, Hkv, Dv) = q.shape, v.shape
    out = torch.zeros(B, Lq, Hq, Dv, dtype=torch.float64)
    i = torch.arange(Lq)[:, None] + q_offset
    j = torch.arange(Lk)[None, :]
    for b in range(B):
        keep = torch.ones(Lq, Lk, dtype=torch.bool)
        if causal:
            keep = (j <= i) | (j < (int(prefix_len[b]) if prefix_len is not None else 0))
        if kv_len is not None:
            keep = keep & (j < int(kv_len[b]))
        if doc_q is not None:
            dq, dk = doc_q[b].cpu()[:, None], doc_k[b].cpu()[None, :]
            keep = keep & (dq == dk) & (dq >= 0)
        for h in range(Hq):
            s = q[b, :, h] @ k[b, :, h // (Hq // Hkv)].T * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * (i - j).abs()
            out[b, :, h] = softmax_rows(s, keep, v[b, :, h // (Hq // Hkv)])
    return out


def decode(q, k_pages, v_pages, table, length, scale, softcap=0.0, slopes=None, first=None):
    """q [B, Hq, Dk] over paged tokens -> float64 CPU [B, Hq, Dv]."""
    B, Hq, _ = q.shape
    page, Hkv, Dv = v_pages.shape[1], v_pages.shape[2], v_pages.shape[3]
    out = torch.zeros(B, Hq, Dv, dtype=torch.float64)
    for b in range(B):
        n, lo = int(length[b]), int(first[b]) if first is not None else 0
        if n <= lo:
            continue
        at = torch.arange(lo, n)
        pages = table[b].cpu().long()[at // page].to(k_pages.device)
        k = k_pages[pages, (at % page).to(k_pages.device)].cpu().double()
        v = v_pages[pages, (at % page).to(k_pages.device)].cpu().double()
        for h in range(Hq):
            s = k[:, h // (Hq // Hkv)] @ q[b, h].cpu().double() * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            if slopes is not None:
                s = s - float(slopes[h]) * (n - 1 - at)
            out[b, h] = torch.softmax(s, dim=0) @ v[:, h // (Hq // Hkv)]
    return out


def bound(ref, v, dtype):
    """Largest allowed |got - ref| per element.  An output is a weighted mean of v.  fp32: the weights carry
    the rounding of scores of size ~20 (a few 2^-24 * 20), under 1e-5 of max|v|.  bf16: besides that, the
    output is rounded once (2^-8 of it) and the weights may be rounded to bf16 before the product
    (2^-8 of each, so at most 2^-8 max|v| of their mean)."""
    big = float(v[torch.isfinite(v)].abs().max()) if v.numel() else 0.0
    if dtype == torch.float32:
        return torch.full_like(ref, 1e-5 * big)
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 1e-5) * big


def check(got, ref, v, dtype):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    over = (got - ref).abs() / bound(ref, v.detach().cpu().double(), dtype).clamp(min=1e-30)
    assert float(over.max()) <= 1.0, float(over.max())


def alibi_slopes(n, device="cpu"):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n) for h in range(n)], dtype=torch.float32, device=device)


def randn(*shape, seed, dtype, device):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(device=device, dtype=dtype)
