"""64-bit plain forms of the operators of drafted tokens, and the rounding
bounds the tests hold the kernels to."""
import math

import numpy as np
import torch

from _attn_path import HALF_STEP, U32, make_pool  # noqa: F401


def random_parents(n, rng, kind="tree"):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "roots":
        return [-1] * n
    return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]


def bits_of(parents_by_seq, max_new):
    """Masks of the tokens of every sequence, and their depths."""
    words = max(1, -(-max_new // 64))
    rows, depths = [], []
    for parents in parents_by_seq:
        masks, depth = [], []
        for i, p in enumerate(parents):
            masks.append((masks[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        rows += [[m >> 64 * w & (1 << 64) - 1 for w in range(words)] for m in masks]
        depths.append(depth)
    bits = np.array(rows, dtype=np.uint64).reshape(-1, words).view(np.int64)
    return torch.from_numpy(bits.copy()), depths


def sees(bits, first, n):
    """[n, n] truth values of a segment's masks (None: a chain)."""
    i = torch.arange(n)
    if bits is None:
        return i[None, :] <= i[:, None]
    w = bits[first:first + n].numpy().view(np.uint64)
    out = np.zeros((n, n), dtype=bool)
    for j in range(n):
        out[:, j] = (w[:, j // 64] >> np.uint64(j % 64)) & np.uint64(1) == 1
    return torch.from_numpy(out)


def rows_of(pool, table_row, n):
    """Keys (or values) of a sequence, (n, H_kv, d) in fp64."""
    ps = pool.shape[2]
    x = torch.arange(n)
    return pool[table_row.long()[x // ps], :, x % ps].double()


def tree_attn(k_pages, v_pages, q, ns, table, lens, bits=None, scale=None):
    """(o, lse [H, T], sum_x p_x |v_x|, max_x sum_c |q_c k_xc| scale) in fp64; a value that a token does not see is
    no part of its sum."""
    T, H, d = q.shape
    Hk = k_pages.shape[1]
    G = H // Hk
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros(T, H, d, dtype=torch.float64)
    mag, cond = torch.zeros_like(o), torch.zeros(T, H, 1, dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    first = 0
    for b, n in enumerate(ns):
        L = int(lens[b])
        if n:
            k, v = rows_of(k_pages, table[b], L), rows_of(v_pages, table[b], L)
            see = torch.ones(n, L, dtype=torch.bool)
            see[:, L - n:] = sees(bits, first, n)
            for h in range(H):
                g = h // G
                qh = q[first:first + n, h].double()
                s = (qh @ k[:, g].T * scale).masked_fill(~see, -math.inf)
                some = see.any(1)
                p = torch.where(some[:, None], torch.softmax(s, 1), torch.zeros_like(s))
                vg = v[:, g]
                fine = torch.isfinite(vg)
                out = p @ torch.where(fine, vg, torch.zeros_like(vg))
                for x in (~fine).any(1).nonzero().flatten().tolist():
                    out[see[:, x]] += torch.where(fine[x], torch.zeros_like(vg[x]), vg[x])
                o[first:first + n, h] = out
                mag[first:first + n, h] = p @ torch.where(fine, vg, torch.zeros_like(vg)).abs()
                c = (qh.abs() @ k[:, g].abs().T * scale).masked_fill(~see, 0)
                cond[first:first + n, h, 0] = c.max(1).values
                lse[h, first:first + n] = torch.logsumexp(s, 1)
        first += n
    return o, lse, mag, cond


def tree_bound(o, mag, cond, n, dtype):
    """Elementwise bound of the attention's output against fp64, from its
    roundings: the output's own; in bf16 a probability's as the sum of two
    bf16, 2^-15; of a score at most 16 steps of its sum |q k| scale in bf16
    (eight products of 16 columns, two steps each), in numerator and
    denominator; 16 steps for exponentials and scale; of the sums of p and p v
    over n keys two steps for each 16 keys and each part of a probability
    (bf16), or one for each key in turn (fp32); 64 for joins.

    fp32 by products of tf32 parts: q = qh + ql with |ql| <= 2^-11 |q|, k = kh +
    kl with |kl| < 2^-10 |k|; ql kl is left out (2^-21 |q k|, 8 steps of 2^-24),
    kl and ql are rounded to 11 bits (2^-22 and 2^-23: 4 and 2 steps); the
    matrix instruction cuts its sums (a step of 2^-23 each, two of them to 16
    columns: 4 steps of sum |q k| in all), and d / 16 + 1 fp32 adds are a step
    each, 9 at most: 27, taken as 28, against 16 where d / 4 packed sums are added up.
    p v likewise: 14 steps for what is left out and rounded, and at most ten for
    each tile of 64 keys' sums, which the n steps and the 64 hold."""
    score = 16 if dtype == torch.bfloat16 else 28
    c = 2 * score * cond + 16 + (n / 4 if dtype == torch.bfloat16 else n) + 64
    p = 2.0 ** -15 if dtype == torch.bfloat16 else 0.0
    return HALF_STEP[dtype] * o.abs() * 1.001 + (p + c * U32) * mag + 1e-38
