"""64-bit plain forms of the attention-path operators (query/key norm with
rotary positions, paged cache, paged attention), and the rounding bounds the
tests hold the kernels to."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


def inv_freq(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Radians per position, term by term from the definition."""
    out = []
    for j in range(rot // 2):
        b = base
        if scaling == "ntk" and rot > 2:
            b = base * factor ** (rot / (rot - 2))
        f = b ** (-2.0 * j / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            g = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f *= (1 - g) / factor + g
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def positions_of(segs, starts=None):
    starts = [0] * len(segs) if starts is None else starts
    parts = [torch.arange(s, s + n) for s, n in zip(starts, segs)]
    return torch.cat(parts) if parts else torch.zeros(0, dtype=torch.int64)


def columns(rot, interleaved):
    if interleaved:
        return torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    return torch.arange(rot // 2), torch.arange(rot // 2, rot)


def rope(x, pos, freq, gamma=None, eps=1e-6, interleaved=False, scale=1.0):
    """(output, the magnitude its rounding errors are relative to), fp64."""
    y = x.double()
    if gamma is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma.double()
    mag = y.abs()
    out = y.clone()
    if freq is not None and freq.numel():
        t = pos.double()[:, None, None] * freq
        c, s = torch.cos(t) * scale, torch.sin(t) * scale
        ia, ib = columns(2 * freq.numel(), interleaved)
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
        both = (a.abs() + b.abs()) * abs(scale)
        mag = mag.clone()
        mag[..., ia], mag[..., ib] = both, both
    return out, mag


def paged_kv(pool, table_row, n):
    """Keys (or values) of one sequence, (n, H_kv, d) in fp64."""
    ps = pool.shape[2]
    rows = [pool[int(table_row[x // ps]), :, x % ps] for x in range(n)]
    return torch.stack(rows).double() if rows else torch.zeros(0, pool.shape[1], pool.shape[3], dtype=torch.float64)


def paged_attn(k_pages, v_pages, q, table, lengths, scale=None):
    """(o, lse [H, B], sum_j p_j |v_j|, max_j sum_c |q_c k_jc| scale) in fp64."""
    B, H, d = q.shape
    Hk = k_pages.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros(B, H, d, dtype=torch.float64)
    mag = torch.zeros(B, H, d, dtype=torch.float64)
    cond = torch.zeros(B, H, 1, dtype=torch.float64)
    lse = torch.full((H, B), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(lengths[b])
        if n == 0:
            continue
        k, v = paged_kv(k_pages, table[b], n), paged_kv(v_pages, table[b], n)
        for h in range(H):
            g = h // (H // Hk)
            qh = q[b, h].double()
            s = k[:, g] @ qh * scale
            p = torch.softmax(s, 0)
            o[b, h] = p @ v[:, g]
            mag[b, h] = p @ v[:, g].abs()
            cond[b, h] = (k[:, g].abs() @ qh.abs()).max() * scale
            lse[h, b] = torch.logsumexp(s, 0)
    return o, lse, mag, cond


def make_pool(lens, page, Hk, d, dtype, seed, spare=3):
    """Random pages and a block table over shuffled pages (-1 behind the end)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    mk = lambda: torch.from_numpy(rng.standard_normal((n_pages, Hk, page, d)).astype(np.float32)).to(dtype)
    return mk(), mk(), torch.from_numpy(table)


def attn_bound(o, mag, cond, n, dtype):
    """Elementwise bound of a paged attention output against fp64, derived
    from the roundings: the output's own (half a step); for bf16 the
    probabilities' (each off by half a step, so at most 2^-8 of sum p |v|);
    in fp32 arithmetic a score's error is at most (d / 32 + 8) steps of its
    sum |q k| scale in either kernel, taken as 16 of them and twice (numerator
    and denominator), plus 8 steps for the exponential and the scale, plus a
    step per key a thread adds in turn (n / 8 at most) and per join."""
    c = 2 * 16 * cond + 8 * 2 + n / 8 + 64
    p = HALF_STEP[torch.bfloat16] if dtype == torch.bfloat16 else 0.0
    return HALF_STEP[dtype] * o.abs() * 1.001 + (p + c * U32) * mag
