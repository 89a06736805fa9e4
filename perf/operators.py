"""The attention-path operators on real work: queries and keys normalised and
rotated (forward and backward), keys and values written to the pages of a
cache, pages copied, and one new token's attention over a paged cache.

``run`` computes each operator in plain torch operations, or, where ``own``
is set, by the library's calls.  ``exact`` gives the same outputs from the
definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # One decoding step of 16 sequences deep in their contexts: latency.
        {"name": "rope_step", "op": "rope", "dtype": "bf16", "T": 16, "seg_lo": 1, "seg_hi": 1, "len_seed": 1,
         "H": 32, "Hk": 8, "d": 128, "rot": 128, "norm": True, "interleaved": False, "base": 1000000.0,
         "scaling": "bands", "factor": 4.0, "orig": 32768, "rot_scale": 1.1386, "far": 131072},
        # The packed stream of varlen attention: 65,536 tokens in segments of 16 to 512, 12 heads of 64.
        {"name": "rope_stream", "op": "rope", "dtype": "bf16", "T": 65536, "seg_lo": 16, "seg_hi": 512, "len_seed": 2,
         "H": 12, "Hk": 12, "d": 64, "rot": 64, "norm": True, "interleaved": False, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "orig": 0, "rot_scale": 1.0, "far": 0},
        # The same stream's gradients, as a training step takes them.
        {"name": "rope_bwd_stream", "op": "rope_bwd", "dtype": "bf16", "T": 65536, "seg_lo": 16, "seg_hi": 512,
         "len_seed": 2, "H": 12, "Hk": 12, "d": 64, "rot": 64, "norm": True, "interleaved": False, "base": 10000.0,
         "scaling": "none", "factor": 1.0, "orig": 0, "rot_scale": 1.0, "far": 0},
        # A small fp32 training batch, shared key heads, half of each head rotated in the interleaved layout.
        {"name": "rope_bwd_partial_f32", "op": "rope_bwd", "dtype": "f32", "T": 2777, "seg_lo": 1, "seg_hi": 700,
         "len_seed": 3, "H": 32, "Hk": 8, "d": 128, "rot": 64, "norm": True, "interleaved": True, "base": 500000.0,
         "scaling": "ntk", "factor": 2.0, "orig": 0, "rot_scale": 1.0, "far": 4096},
        # One decoding step of 24 sequences appends a token to each.
        {"name": "write_step", "op": "write", "dtype": "bf16", "T": 24, "seg_lo": 1, "seg_hi": 1, "len_seed": 4,
         "Hk": 8, "d": 128, "page": 16, "far": 2000},
        # The packed stream, prefilled: every segment's keys and values go to its pages.
        {"name": "write_prefill", "op": "write", "dtype": "bf16", "T": 65536, "seg_lo": 16, "seg_hi": 512,
         "len_seed": 2, "Hk": 12, "d": 64, "page": 64, "far": 0},
        # A fork: the partly filled last pages of 16 sequences are copied.
        {"name": "copy_fork", "op": "copy", "dtype": "bf16", "n": 16, "pool": 512, "Hk": 8, "d": 128, "page": 16},
        # Compaction of a large cache: 2,048 pages move.
        {"name": "copy_compact", "op": "copy", "dtype": "bf16", "n": 2048, "pool": 5000, "Hk": 12, "d": 64, "page": 64},
        # One user's next token over a short context, every query head with its own keys.
        {"name": "attn_one", "op": "attn", "dtype": "bf16", "B": 1, "len_lo": 777, "len_hi": 777, "len_seed": 5,
         "H": 12, "Hk": 12, "d": 64, "page": 16},
        # A serving batch: 64 contexts from a few tokens to 8,192, four query heads to a key head.
        {"name": "attn_batch", "op": "attn", "dtype": "bf16", "B": 64, "len_lo": 16, "len_hi": 8192, "len_seed": 6,
         "H": 32, "Hk": 8, "d": 128, "page": 16},
        # Four very long contexts.
        {"name": "attn_long", "op": "attn", "dtype": "bf16", "B": 4, "len_lo": 100000, "len_hi": 131071,
         "len_seed": 7, "H": 32, "Hk": 8, "d": 128, "page": 64},
        # The fp32 mode: 13 contexts, two query heads to a key head.
        {"name": "attn_f32", "op": "attn", "dtype": "f32", "B": 13, "len_lo": 1, "len_hi": 5000, "len_seed": 8,
         "H": 16, "Hk": 8, "d": 64, "page": 32},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "rope_bwd", "rope_bwd", "write", "copy", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    es = 2 if dtype == "bf16" else 4
    Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
    case = {"op": op, "dtype": dtype, "len_seed": rng.randrange(1 << 30), "Hk": Hk}
    if op in ("rope", "rope_bwd"):
        d = rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
        H = Hk * rng.choice([1, 1, 2, 4, 8])
        # the stream listed above moves 65,536 x 24 x 64 bf16 elements of q and k
        cap = max(1, min(65536, 65536 * 24 * 64 * 2 // ((H + Hk) * d * es)))
        T = _log_int(rng, 1, cap)
        case.update(T=T, seg_lo=1, seg_hi=_log_int(rng, 1, 4096), H=H, d=d,
                    rot=16 * rng.randint(1, d // 16) if rng.random() < 0.4 else d, norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.4, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    orig=rng.choice([2048, 8192, 32768]), rot_scale=rng.choice([1.0, 1.1386]),
                    far=rng.choice([0, 0, 1000, 131072, 1000000]))
    elif op == "write":
        d = rng.choice([32, 64, 128])
        T = _log_int(rng, 1, max(1, min(65536, 65536 * 12 * 64 * 2 // (Hk * d * es))))
        case.update(T=T, seg_lo=1, seg_hi=_log_int(rng, 1, 2048), d=d, page=rng.choice([8, 16, 16, 24, 32, 64, 128]),
                    far=rng.choice([0, 0, 100, 3000]))
        if T > 2000:
            case["far"] = min(case["far"], 100)
    elif op == "copy":
        d = rng.choice([32, 64, 128])
        page = rng.choice([8, 16, 16, 24, 32, 64, 128])
        n = _log_int(rng, 1, max(1, min(4000, 2048 * 12 * 64 * 64 * 2 // (Hk * d * page * es))))
        case.update(n=n, pool=2 * n + rng.randint(0, n), d=d, page=page)
    else:
        d = rng.choice([32, 64, 64, 128, 128, 128])
        B = _log_int(rng, 1, 256)
        # the long case above reads 4 x 115,000 x 8 x 128 bf16 keys and values
        cap = min(131072, 4 * 115000 * 8 * 128 * 2 // (B * Hk * d * es))
        hi = _log_int(rng, 1, max(1, cap))
        case.update(B=B, len_lo=rng.choice([0, 1, hi]), len_hi=hi, H=Hk * rng.choice([1, 1, 2, 4, 7, 8, 12, 16]), d=d,
                    page=rng.choice([8, 16, 16, 24, 32, 64, 64, 128, 256]))
    return case


# ----------------------------------------------------------------------------
# Lengths and tables: the case alone fixes the lengths, the seed their order
# ----------------------------------------------------------------------------

def _segments(case):
    """Start position and length of the packed segments of T tokens."""
    rng = random.Random(case["len_seed"])
    out, left = [], case["T"]
    while left > 0:
        n = min(left, rng.randint(case["seg_lo"], case["seg_hi"]))
        out.append((rng.randint(0, case["far"]), n))
        left -= n
    return out


def _contexts(case):
    """Context lengths of B sequences, uniform in their logarithm."""
    rng = random.Random(case["len_seed"])
    lo, hi = case["len_lo"], case["len_hi"]
    return [0 if lo == 0 and rng.random() < 0.1 else _log_int(rng, max(lo, 1), hi) for _ in range(case["B"])]


def _pages_of(lens, page):
    return [-(-n // page) for n in lens]


def _table(lens, page, rng):
    """A block table over a shuffled pool with a quarter of its pages spare;
    entries behind a sequence's last page are -1."""
    need = _pages_of(lens, page)
    pool = sum(need) + sum(need) // 4 + 1
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool


def _inv_freq(case):
    """Radians per position of each rotated pair, in 64 bits."""
    rot, base, F = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rot > 2:
        base = base * F ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        f = f / F
    elif case["scaling"] == "bands":
        turns = case["orig"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * ((1 - keep) / F + keep)
    return f


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    randn = lambda *shape, dtype=dt: torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)
    st = {"case": case}
    if case["op"] in ("rope", "rope_bwd", "write"):
        pairs = _segments(case)
        pairs = [pairs[i] for i in rng.permutation(len(pairs))]
        st["starts"], segs = [s for s, _ in pairs], [n for _, n in pairs]
        st["segs"] = segs
        st["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(segs)]).astype(np.int32), device=DEV)
        st["pos0"] = torch.tensor(st["starts"], dtype=torch.int32, device=DEV)
    if case["op"] in ("rope", "rope_bwd"):
        T, H, Hk, d = case["T"], case["H"], case["Hk"], case["d"]
        st["q"], st["k"] = randn(T, H, d), randn(T, Hk, d)
        st["qg"] = st["kg"] = None
        if case["norm"]:
            st["qg"] = 1 + 0.2 * randn(d, dtype=torch.float32)
            st["kg"] = 1 + 0.2 * randn(d, dtype=torch.float32)
        st["inv_freq"] = _inv_freq(case).to(DEV)
        if case["op"] == "rope_bwd":
            st["dq"], st["dk"] = randn(T, H, d), randn(T, Hk, d)
    elif case["op"] == "write":
        T, Hk, d = case["T"], case["Hk"], case["d"]
        st["k"], st["v"] = randn(T, Hk, d), randn(T, Hk, d)
        table, pool = _table([s + n for s, n in zip(st["starts"], st["segs"])], case["page"], rng)
        st["table"] = torch.from_numpy(table).to(DEV)
        st["k_pages"], st["v_pages"] = (randn(pool, Hk, case["page"], d) for _ in range(2))
    elif case["op"] == "copy":
        ids = rng.permutation(case["pool"])
        st["src"] = torch.from_numpy(ids[:case["n"]].astype(np.int32))
        st["dst"] = torch.from_numpy(ids[case["n"]:2 * case["n"]].astype(np.int32))
        st["k_pages"], st["v_pages"] = (randn(case["pool"], case["Hk"], case["page"], case["d"]) for _ in range(2))
    else:
        lens = [int(n) for n in rng.permutation(_contexts(case))]
        table, pool = _table(lens, case["page"], rng)
        st["lens"] = lens
        st["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        st["table"] = torch.from_numpy(table).to(DEV)
        st["q"] = 2 * randn(case["B"], case["H"], case["d"])
        st["k_pages"], st["v_pages"] = (randn(pool, case["Hk"], case["page"], case["d"]) for _ in range(2))
    if own:
        from variable_length_batching_gb300 import nt
        if case["op"] in ("rope", "rope_bwd"):
            st["turns"] = nt.nt_rope_turns(case["rot"], base=case["base"], scaling=case["scaling"],
                                           factor=case["factor"], original_len=case["orig"], low=1.0, high=32.0,
                                           device=DEV)
        else:
            st["pages"] = nt.KVPages(st["k_pages"], st["v_pages"])
        if case["op"] == "attn":
            st["workspace"] = torch.empty(nt.nt_paged_attn_workspace_bytes(case["H"], case["Hk"], case["d"]),
                                          dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------

def _positions(st):
    t = torch.arange(st["case"]["T"], device=DEV, dtype=torch.int32)
    seg = torch.searchsorted(st["cu"], t, right=True) - 1
    return seg, (t - st["cu"][seg] + st["pos0"][seg]).long()


def _cos_sin(st):
    pos = _positions(st)[1]
    angle = pos.double()[:, None] * st["inv_freq"][None, :]
    s = st["case"]["rot_scale"]
    return (angle.cos() * s).float()[:, None, :], (angle.sin() * s).float()[:, None, :]


def _split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    pair = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((pair, rest), -1)


def _plain_rope(st, x, gamma, cos, sin):
    c = st["case"]
    y = x.float()
    if gamma is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * gamma
    a, b = _split(y, c["rot"], c["interleaved"])
    return _join(a * cos - b * sin, a * sin + b * cos, y[..., c["rot"]:], c["interleaved"]).to(x.dtype)


def _plain_rope_bwd(st, dy, x, gamma, cos, sin):
    c = st["case"]
    g = dy.float()
    a, b = _split(g, c["rot"], c["interleaved"])
    g = _join(a * cos + b * sin, b * cos - a * sin, g[..., c["rot"]:], c["interleaved"])
    if gamma is None:
        return g.to(x.dtype), None
    xf = x.float()
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
    n = xf * r
    h = g * gamma
    return (r * (h - n * (h * n).mean(-1, keepdim=True))).to(x.dtype), (g * n).sum((0, 1))


def _plain_attn(st):
    c = st["case"]
    Hk, d = c["Hk"], c["d"]
    out = torch.zeros_like(st["q"])
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // c["page"])].long()
        k = st["k_pages"][ids].transpose(0, 1).reshape(Hk, -1, d)[:, :n].float()
        v = st["v_pages"][ids].transpose(0, 1).reshape(Hk, -1, d)[:, :n].float()
        q = st["q"][b].float().reshape(Hk, -1, d)
        s = q @ k.transpose(1, 2) * d ** -0.5
        p = torch.exp(s - s.amax(-1, keepdim=True))
        out[b] = ((p @ v) / p.sum(-1, keepdim=True)).reshape(-1, d).to(out.dtype)
    return out


def _run_plain(st):
    c = st["case"]
    if c["op"] in ("rope", "rope_bwd"):
        cos, sin = _cos_sin(st)
        if c["op"] == "rope":
            return _plain_rope(st, st["q"], st["qg"], cos, sin), _plain_rope(st, st["k"], st["kg"], cos, sin)
        dq, dqg = _plain_rope_bwd(st, st["dq"], st["q"], st["qg"], cos, sin)
        dk, dkg = _plain_rope_bwd(st, st["dk"], st["k"], st["kg"], cos, sin)
        return (dq, dk, dqg, dkg) if c["norm"] else (dq, dk)
    if c["op"] == "write":
        seg, pos = _positions(st)
        page = st["table"][seg, pos // c["page"]].long()
        st["k_pages"][page, :, pos % c["page"]] = st["k"]
        st["v_pages"][page, :, pos % c["page"]] = st["v"]
        return st["k_pages"], st["v_pages"]
    if c["op"] == "copy":
        src, dst = st["src"].long().to(DEV), st["dst"].long().to(DEV)
        st["k_pages"][dst] = st["k_pages"][src]
        st["v_pages"][dst] = st["v_pages"][src]
        return st["k_pages"], st["v_pages"]
    return _plain_attn(st)


def _run_own(st):
    from variable_length_batching_gb300 import nt
    c = st["case"]
    if c["op"] == "rope":
        return nt.nt_qk_norm_rope(st["q"], st["k"], st["turns"], cu_seqlens=st["cu"], pos0=st["pos0"],
                                  q_gamma=st["qg"], k_gamma=st["kg"], eps=1e-6, interleaved=c["interleaved"],
                                  rot_scale=c["rot_scale"])
    if c["op"] == "rope_bwd":
        dq, dk, dqg, dkg = nt.nt_qk_norm_rope_bwd(st["dq"], st["dk"], st["turns"], q=st["q"], k=st["k"],
                                                  cu_seqlens=st["cu"], pos0=st["pos0"], q_gamma=st["qg"],
                                                  k_gamma=st["kg"], eps=1e-6, interleaved=c["interleaved"],
                                                  rot_scale=c["rot_scale"])
        return (dq, dk, dqg, dkg) if c["norm"] else (dq, dk)
    if c["op"] == "write":
        nt.nt_paged_write(st["pages"], st["k"], st["v"], st["cu"], st["table"], pos0=st["pos0"])
        return st["k_pages"], st["v_pages"]
    if c["op"] == "copy":
        nt.nt_paged_copy(st["pages"], st["src"], st["dst"])
        return st["k_pages"], st["v_pages"]
    return nt.nt_paged_attn(st["pages"], st["q"], st["table"], st["lengths"], workspace=st["workspace"])[0]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# Work and exact values
# ----------------------------------------------------------------------------

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    Hk, d = case["Hk"], case["d"]
    if case["op"] in ("rope", "rope_bwd"):
        n = case["T"] * (case["H"] + Hk) * d
        if case["op"] == "rope":
            return {"bytes": 2 * n * es, "flops": (7 if case["norm"] else 3) * n}
        return {"bytes": (3 if case["norm"] else 2) * n * es, "flops": (13 if case["norm"] else 3) * n}
    if case["op"] == "write":
        return {"bytes": 4 * case["T"] * Hk * d * es, "flops": 0}
    if case["op"] == "copy":
        return {"bytes": 4 * case["n"] * Hk * case["page"] * d * es, "flops": 0}
    total = sum(_contexts(case))
    return {"bytes": 2 * total * Hk * d * es + 2 * case["B"] * case["H"] * d * es,
            "flops": 4 * total * case["H"] * d}


def _exact_turn(st):
    """cos and sin of every token and pair, token by token from the segments."""
    c = st["case"]
    pos = np.concatenate([np.arange(s, s + n, dtype=np.float64) for s, n in zip(st["starts"], st["segs"])])
    j = np.arange(c["rot"] // 2, dtype=np.float64)
    base = c["base"] * (c["factor"] ** (c["rot"] / (c["rot"] - 2.0)) if c["scaling"] == "ntk" else 1.0)
    f = np.exp(-2.0 * j / c["rot"] * math.log(base))
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "bands":
        w = np.minimum(1.0, np.maximum(0.0, (c["orig"] * f / (2 * math.pi) - 1.0) / 31.0))
        f = w * f + (1.0 - w) * f / c["factor"]
    z = torch.from_numpy(np.multiply.outer(pos, f)).to(DEV)
    return torch.polar(torch.full_like(z, c["rot_scale"]), z)[:, None, :]      # s e^(i theta)


def _as_complex(x, c):
    """The rotated columns as complex pairs, and the index of both parts."""
    rot = c["rot"]
    ia = torch.arange(0, rot, 2, device=DEV) if c["interleaved"] else torch.arange(rot // 2, device=DEV)
    ib = ia + (1 if c["interleaved"] else rot // 2)
    return torch.complex(x[..., ia], x[..., ib]), ia, ib


def _exact_rope(x, gamma, turn, c):
    y = x.double()
    if gamma is not None:
        y = gamma.double() * y / (y.square().sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt()
    z, ia, ib = _as_complex(y, c)
    z = z * turn
    out = y.clone()
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def _exact_rope_bwd(dy, x, gamma, turn, c):
    g = dy.double()
    z, ia, ib = _as_complex(g, c)
    z = z * turn.conj()
    g = g.clone()
    g[..., ia], g[..., ib] = z.real, z.imag
    if gamma is None:
        return g, None
    x = x.double()
    var = x.square().sum(-1, keepdim=True) / c["d"] + 1e-6
    h = g * gamma.double()
    # d/dx of h . x var^(-1/2)
    dx = h / var.sqrt() - x * ((h * x).sum(-1, keepdim=True) / c["d"]) / var.pow(1.5)
    return dx, (g * x / var.sqrt()).sum((0, 1))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        turn = _exact_turn(st)
        if case["op"] == "rope":
            return (_exact_rope(st["q"], st["qg"], turn, case), _exact_rope(st["k"], st["kg"], turn, case))
        dq, dqg = _exact_rope_bwd(st["dq"], st["q"], st["qg"], turn, case)
        dk, dkg = _exact_rope_bwd(st["dk"], st["k"], st["kg"], turn, case)
        return (dq, dk, dqg, dkg) if case["norm"] else (dq, dk)
    if case["op"] == "write":
        slots = np.concatenate([np.arange(s, s + n) for s, n in zip(st["starts"], st["segs"])])
        rows = np.repeat(np.arange(len(st["segs"])), st["segs"])
        page = st["table"].cpu().numpy()[rows, slots // case["page"]]
        flat = torch.from_numpy(page.astype(np.int64) * case["page"] + slots % case["page"]).to(DEV)
        outs = []
        for pool, new in ((st["k_pages"], st["k"]), (st["v_pages"], st["v"])):
            n, Hk, ps, d = pool.shape
            token_major = pool.permute(0, 2, 1, 3).reshape(n * ps, Hk, d).index_copy(0, flat, new)
            outs.append(token_major.reshape(n, ps, Hk, d).permute(0, 2, 1, 3).contiguous())
        return tuple(outs)
    if case["op"] == "copy":
        outs = []
        for pool in (st["k_pages"], st["v_pages"]):
            new = pool.clone()
            for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
                new[t] = pool[s]
            outs.append(new)
        return tuple(outs)
    G = case["H"] // case["Hk"]
    out = torch.zeros(case["B"], case["H"], case["d"], dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        ids = st["table"][b, :(n + case["page"] - 1) // case["page"]].long()
        for h in range(case["Hk"]):
            k = st["k_pages"][ids, h].reshape(-1, case["d"])[:n].double()
            v = st["v_pages"][ids, h].reshape(-1, case["d"])[:n].double()
            w = torch.softmax(k @ st["q"][b, h * G:(h + 1) * G].double().T / math.sqrt(case["d"]), dim=0)
            out[b, h * G:(h + 1) * G] = w.T @ v
    return out
