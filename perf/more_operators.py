"""The operators of a decoding step with drafted tokens: block tables and slot
maps built on the GPU from request lengths, the masks and positions of a tree
of drafted tokens, the attention of such trees over a paged cache, and the
accepted tokens' keys and values moved up.

``run`` computes each operator in plain torch operations, or, where ``own``
is set, by the library's calls.  ``exact`` gives the same outputs from the
definition, the attention's in 64 bits.
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
        # One user, eight drafted tokens over a short context, every query head with its own keys: latency.
        {"name": "attn_one", "op": "attn", "dtype": "bf16", "B": 1, "len_lo": 777, "len_hi": 777, "n_lo": 8, "n_hi": 8,
         "tree": True, "len_seed": 1, "H": 12, "Hk": 12, "d": 64, "page": 16},
        # A serving batch that drafts short chains: 64 contexts from a few tokens to 8,192, up to four new tokens each.
        {"name": "attn_chain", "op": "attn", "dtype": "bf16", "B": 64, "len_lo": 16, "len_hi": 8192, "n_lo": 1,
         "n_hi": 4, "tree": False, "len_seed": 2, "H": 32, "Hk": 8, "d": 128, "page": 16},
        # Trees of up to 64 drafted tokens on 16 such contexts.
        {"name": "attn_batch", "op": "attn", "dtype": "bf16", "B": 16, "len_lo": 16, "len_hi": 8192, "n_lo": 20,
         "n_hi": 64, "tree": True, "len_seed": 3, "H": 32, "Hk": 8, "d": 128, "page": 16},
        # Four very long contexts with a tree each.
        {"name": "attn_long", "op": "attn", "dtype": "bf16", "B": 4, "len_lo": 100000, "len_hi": 131071, "n_lo": 25,
         "n_hi": 32, "tree": True, "len_seed": 4, "H": 32, "Hk": 8, "d": 128, "page": 64},
        # Prompts taken in pieces of 256 tokens behind what is cached already: the products' rate counts.
        {"name": "attn_piece", "op": "attn", "dtype": "bf16", "B": 8, "len_lo": 2000, "len_hi": 16384, "n_lo": 256,
         "n_hi": 256, "tree": False, "len_seed": 5, "H": 32, "Hk": 8, "d": 128, "page": 64},
        # The fp32 mode: 13 contexts, two query heads to a key head, small trees.
        {"name": "attn_f32", "op": "attn", "dtype": "f32", "B": 13, "len_lo": 1, "len_hi": 5000, "n_lo": 1, "n_hi": 12,
         "tree": True, "len_seed": 6, "H": 16, "Hk": 8, "d": 64, "page": 32},
        # One step's tables: 64 requests get room for 8 drafted tokens each, and give it back.
        {"name": "table_step", "op": "table", "B": 64, "len_lo": 16, "len_hi": 8192, "n_lo": 8, "n_hi": 8,
         "len_seed": 7, "page": 16},
        # A wave of 512 prompts of up to 250 tokens comes in, and leaves.
        {"name": "table_prompts", "op": "table", "B": 512, "len_lo": 0, "len_hi": 0, "n_lo": 6, "n_hi": 250,
         "len_seed": 8, "page": 16},
        # One step's trees: 16 sequences of up to 64 tokens.
        {"name": "tree_step", "op": "tree", "B": 16, "n_lo": 20, "n_hi": 64, "len_seed": 9},
        # The largest trees for a large batch.
        {"name": "tree_many", "op": "tree", "B": 256, "n_lo": 128, "n_hi": 256, "len_seed": 10},
        # One step's accepted tokens, one layer: 16 sequences keep up to six of 64.
        {"name": "keep_step", "op": "keep", "dtype": "bf16", "B": 16, "len_lo": 16, "len_hi": 2000, "kept_lo": 1,
         "kept_hi": 6, "n_hi": 64, "len_seed": 11, "Hk": 8, "d": 128, "page": 16},
        # A large batch keeps long paths.
        {"name": "keep_many", "op": "keep", "dtype": "bf16", "B": 256, "len_lo": 16, "len_hi": 2000, "kept_lo": 16,
         "kept_hi": 64, "n_hi": 200, "len_seed": 12, "Hk": 8, "d": 128, "page": 16},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attn"] * 6 + ["table", "table", "tree", "keep"])
    case = {"op": op, "len_seed": rng.randrange(1 << 30)}
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128, 12])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hk, d = rng.choice([1, 2, 3, 4, 8, 12, 16]), rng.choice([32, 64, 64, 128, 128, 128])
        H = Hk * rng.choice([1, 1, 2, 4, 4, 7, 8, 16])
        B, n_hi = _log_int(rng, 1, 128), _log_int(rng, 1, 256)
        # the long case above reads 4 x 115,000 x 8 x 128 bf16 keys and values and takes 2.2e11 operations;
        # fp32 has a small part of the rate
        rows = 4 * B * H * n_hi * d
        cap = min(131072, 4 * 115000 * 8 * 128 // (B * Hk * d), int(2.2e11 if dtype == "bf16" else 2e10) // rows)
        hi = _log_int(rng, 1, max(1, cap))
        case.update(dtype=dtype, B=B, len_lo=rng.choice([0, 1, hi]), len_hi=hi, n_lo=rng.choice([0, 1, n_hi]),
                    n_hi=n_hi, tree=rng.random() < 0.6, H=H, Hk=Hk, d=d, page=page)
    elif op == "table":
        B = _log_int(rng, 1, 2048)
        hi = _log_int(rng, 1, max(1, min(8192, 300000 // B)))
        n_hi = _log_int(rng, 1, max(1, min(4096, 100000 // B)))
        case.update(B=B, len_lo=rng.choice([0, 1, hi]), len_hi=hi, n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi, page=page)
    elif op == "tree":
        n_hi = _log_int(rng, 1, 256)
        case.update(B=_log_int(rng, 1, 256), n_lo=rng.choice([0, 1, n_hi]), n_hi=n_hi)
    else:
        Hk, d, dtype = rng.choice([1, 2, 4, 8, 12]), rng.choice([32, 64, 128]), rng.choice(["bf16", "bf16", "f32"])
        kept = _log_int(rng, 1, 64)
        B = _log_int(rng, 1, max(1, min(256, 256 * 40 * 8 * 128 * 2 // (kept * Hk * d * (2 if dtype == "bf16" else 4)))))
        case.update(dtype=dtype, B=B, len_lo=rng.choice([0, 1]), len_hi=_log_int(rng, 1, 2000),
                    kept_lo=rng.choice([0, 1, kept]), kept_hi=kept, n_hi=rng.randint(2 * kept, 256), Hk=Hk, d=d,
                    page=page)
    return case


# ----------------------------------------------------------------------------
# Lengths, trees and tables: the case alone fixes the lengths, the seed their order
# ----------------------------------------------------------------------------

def _lengths(case):
    """Context length and number of new (or kept) tokens of every sequence."""
    rng = random.Random(case["len_seed"])
    lo, hi = case.get("len_lo", 0), case.get("len_hi", 0)
    n_lo, n_hi = (case["kept_lo"], case["kept_hi"]) if case["op"] == "keep" else (case["n_lo"], case["n_hi"])
    out = []
    for i in range(case["B"]):
        ctx = 0 if hi == 0 or (lo == 0 and rng.random() < 0.1) else _log_int(rng, max(lo, 1), hi)
        n = rng.randint(n_lo, n_hi)
        out.append((ctx, n_hi if i == 0 else n))
    return out


def _table(lens, page, rng, width=1):
    """A block table over a shuffled pool with spare pages; entries behind a
    sequence's last page are -1."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + sum(need) // 4 + 1
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((len(lens), max(need + [width])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pool, ids[at:]


def _parents(ns, rng):
    """A drafted tree for each sequence: a token hangs on the context or on an
    earlier token, often a recent one."""
    out = []
    for n in ns:
        i = np.arange(n)
        recent = i - rng.integers(1, 5, n)
        anywhere = (rng.random(n) * (i + 1)).astype(np.int64) - 1
        out.append(np.maximum(np.where(rng.random(n) < 0.7, recent, anywhere), -1))
    return np.concatenate(out).astype(np.int32) if out else np.zeros(0, np.int32)


def _words(n):
    return max(1, -(-n // 64))


def _bits_of(parents, cu, words):
    """Ancestors and self of every token, 64 drafted tokens to a word."""
    bits = np.zeros((len(parents), words), dtype=np.uint64)
    for lo, hi in zip(cu[:-1], cu[1:]):
        for i in range(hi - lo):
            p = parents[lo + i]
            if p >= 0:
                bits[lo + i] = bits[lo + p]
            bits[lo + i, i >> 6] |= np.uint64(1 << (i & 63))
    return bits.view(np.int64)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DTYPES[case.get("dtype", "f32")]
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV, dtype=dt)
    ints = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    pairs = _lengths(case)
    pairs = [pairs[i] for i in rng.permutation(len(pairs))]
    ctx, ns = [c for c, _ in pairs], [n for _, n in pairs]
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int64)
    T = int(cu[-1])
    st = {"case": case, "ctx": ctx, "ns": ns, "T": T, "cu": ints(cu), "pos0": ints(ctx)}
    if case["op"] == "attn":
        lens = [c + n for c, n in pairs]
        table, pool, _ = _table(lens, case["page"], rng)
        st["lens"], st["lengths"], st["table"] = lens, ints(lens), ints(table)
        st["k_pages"], st["v_pages"] = (randn(pool, case["Hk"], case["page"], case["d"]) for _ in range(2))
        st["q"] = 2 * randn(T, case["H"], case["d"])
        st["bits"] = None
        if case["tree"]:
            st["bits"] = torch.from_numpy(_bits_of(_parents(ns, rng), cu.tolist(), _words(case["n_hi"]))).to(DEV)
    elif case["op"] == "table":
        after = [c + n for c, n in pairs]
        wide = max([-(-n // case["page"]) for n in after] + [1])
        _, need, _ = _table(after, case["page"], rng)
        table, _, _ = _table(ctx, case["page"], rng, wide)
        used = int((table >= 0).sum())
        pages = rng.permutation(need).astype(np.int32)          # the sequences' pages, then the free ones
        table[table >= 0] = pages[:used]
        free = np.concatenate([pages[used:], np.full(used, -1, np.int32)])
        st["table"], st["lengths"], st["free"], st["n_free"] = ints(table), ints(ctx), ints(free), ints([need - used])
        st["before"], st["after"] = ints(ctx), ints(after)
    elif case["op"] == "tree":
        st["parents"] = ints(_parents(ns, rng))
        st["pos0"] = ints(rng.integers(0, 100000, case["B"]))
    else:
        table, pool, _ = _table([c + case["n_hi"] for c in ctx], case["page"], rng)
        st["table"] = ints(table)
        st["k_pages"], st["v_pages"] = (randn(pool, case["Hk"], case["page"], case["d"]) for _ in range(2))
        # the accepted path of a tree: its first token is the first drafted one now and then, its others lie
        # behind the places that the kept tokens take
        kept = []
        for n in ns:
            path = n + np.sort(rng.permutation(case["n_hi"] - n)[:n])
            if n and rng.random() < 0.5:
                path[0] = 0
            kept.append(path)
        st["kept_lists"] = kept
        st["kept"] = ints(np.concatenate(kept))
    if own:
        from variable_length_batching_gb300 import nt
        if case["op"] in ("attn", "keep"):
            st["pages"] = nt.KVPages(st["k_pages"], st["v_pages"])
        if case["op"] == "attn":
            st["workspace"] = torch.empty(
                nt.nt_paged_tree_attn_workspace_bytes(case["H"], case["Hk"], case["d"], case["n_hi"]),
                dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------

def _plain_attn(st):
    c = st["case"]
    Hk, d, page = c["Hk"], c["d"], c["page"]
    out = torch.empty_like(st["q"])
    at = 0
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["ns"])):
        if n == 0:
            continue
        ids = st["table"][b, :-(-(ctx + n) // page)].long()
        k = st["k_pages"][ids].transpose(0, 1).reshape(Hk, -1, d)[:, :ctx + n].float()
        v = st["v_pages"][ids].transpose(0, 1).reshape(Hk, -1, d)[:, :ctx + n].float()
        q = st["q"][at:at + n].float().reshape(n, Hk, -1, d).permute(1, 2, 0, 3)          # Hk, G, n, d
        j = torch.arange(n, device=DEV)
        if c["tree"]:
            see = (st["bits"][at:at + n][:, j >> 6] >> (j & 63)) & 1 == 1
        else:
            see = j[None, :] <= j[:, None]
        s = (q @ k[:, None].transpose(2, 3)) * d ** -0.5
        s[..., ctx:] = torch.where(see, s[..., ctx:], -math.inf)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v[:, None]) / p.sum(-1, keepdim=True)
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, -1, d).to(out.dtype)
        at += n
    return out


def _plain_resize(st, new):
    """The lengths become ``new``: pages of the rows that shrink go back to the
    stack, the first of them on top, then the rows that grow take theirs from its top."""
    page = st["case"]["page"]
    table, lengths, free, n_free = st["table"], st["lengths"], st["free"], st["n_free"]
    old = lengths.clone()
    have, want = (old + page - 1) // page, (new + page - 1) // page
    col = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)
    gone = ((col >= want[:, None]) & (col < have[:, None])).flatten()
    come = ((col >= have[:, None]) & (col < want[:, None])).flatten()
    top = n_free.long() + gone.sum() - 1
    more = torch.cat((free, free.new_zeros(1)))                # a place for what is not released
    more[torch.where(gone, top - (gone.cumsum(0) - 1), free.numel())] = table.flatten()
    free.copy_(more[:-1])
    taken = free[(top - (come.cumsum(0) - 1)).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(come, taken, torch.where(gone, -1, table.flatten())).view_as(table))
    n_free.copy_(top + 1 - come.sum())
    lengths.copy_(new)
    cu = torch.cat((old.new_zeros(1), (new - old).clamp(min=0).cumsum(0))).to(torch.int32)
    t = torch.arange(st["T"], device=DEV, dtype=torch.int32)
    seg = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=len(old) - 1)
    pos = (old[seg] + t - cu[seg]).long()
    at = table[seg, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    return cu, old, torch.where(t < cu[-1], at, -1)


def _plain_tree(st):
    T, words = st["T"], _words(st["case"]["n_hi"])
    t = torch.arange(T, device=DEV, dtype=torch.int32)
    seg = torch.searchsorted(st["cu"], t, right=True) - 1
    first = st["cu"][seg]
    i = (t - first).long()
    parents = st["parents"].long()
    bits = torch.zeros(T, words, dtype=torch.int64, device=DEV)
    bits[torch.arange(T, device=DEV), i >> 6] = torch.ones_like(i) << (i & 63)
    up = torch.where(parents >= 0, first + parents, T)         # the token above, T for none
    up = torch.cat((up, up.new_full((1,), T)))
    bits = torch.cat((bits, bits.new_zeros(1, words)))
    steps = torch.cat(((parents >= 0).long(), up.new_zeros(1)))
    for _ in range(max(1, (st["case"]["n_hi"] - 1).bit_length())):
        bits = bits | bits[up]
        steps = steps + steps[up]
        up = up[up]
    return bits[:T], (st["pos0"][seg] + steps[:T]).to(torch.int32)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "attn":
        return _plain_attn(st)
    if c["op"] == "table":
        cu, pos0, slots = _plain_resize(st, st["after"])
        _plain_resize(st, st["before"])
        return cu, pos0, slots, st["table"], st["lengths"], st["free"], st["n_free"]
    if c["op"] == "tree":
        return _plain_tree(st)
    t = torch.arange(st["kept"].numel(), device=DEV, dtype=torch.int32)
    seg = torch.searchsorted(st["cu"], t, right=True) - 1
    dst = (st["pos0"][seg] + t - st["cu"][seg]).long()
    src = (st["pos0"][seg] + st["kept"]).long()
    sp, dp = st["table"][seg, src // c["page"]].long(), st["table"][seg, dst // c["page"]].long()
    for pool in (st["k_pages"], st["v_pages"]):
        pool[dp, :, dst % c["page"]] = pool[sp, :, src % c["page"]]
    return st["k_pages"], st["v_pages"]


def _run_own(st):
    from variable_length_batching_gb300 import nt
    c = st["case"]
    if c["op"] == "attn":
        return nt.nt_paged_tree_attn(st["pages"], st["q"], st["cu"], st["table"], st["lengths"], c["n_hi"],
                                     bits=st["bits"], workspace=st["workspace"])[0]
    if c["op"] == "table":
        state = (st["table"], st["lengths"], st["free"], st["n_free"], c["page"])
        cu, pos0, slots, _ = nt.nt_paged_resize(*state, st["after"], st["T"])
        nt.nt_paged_resize(*state, st["before"], st["T"])
        return cu, pos0, slots, st["table"], st["lengths"], st["free"], st["n_free"]
    if c["op"] == "tree":
        return nt.nt_draft_tree(st["parents"], st["cu"], c["n_hi"], pos0=st["pos0"])
    nt.nt_paged_keep(st["pages"], st["kept"], st["cu"], st["table"], st["pos0"])
    return st["k_pages"], st["v_pages"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# Work and exact values
# ----------------------------------------------------------------------------

def work(case):
    pairs = _lengths(case)
    T = sum(n for _, n in pairs)
    if case["op"] == "attn":
        es = 2 if case["dtype"] == "bf16" else 4
        Hk, H, d = case["Hk"], case["H"], case["d"]
        keys = sum(c + n for c, n in pairs if n)
        mask = 8 * _words(case["n_hi"]) * T if case["tree"] else 0
        see = sum(n * c + (n * (n + 1) // 2) for c, n in pairs)
        return {"bytes": 2 * keys * Hk * d * es + 2 * T * H * d * es + mask, "flops": 4 * see * H * d}
    if case["op"] == "table":
        pages = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in pairs)
        # each way: lengths read and written, new ones read, offsets written, slots written, pages moved
        return {"bytes": 2 * (20 * case["B"] + 8 * T + 8 * pages), "flops": 0}
    if case["op"] == "tree":
        return {"bytes": (8 + 8 * _words(case["n_hi"])) * T, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": 4 * T * case["Hk"] * case["d"] * es + 4 * T, "flops": 0}


def _exact_attn(st):
    c = st["case"]
    G, d, page = c["H"] // c["Hk"], c["d"], c["page"]
    out = torch.zeros(st["T"], c["H"], d, dtype=torch.float64, device=DEV)
    bits = st["bits"].cpu().numpy().view(np.uint64) if c["tree"] else None
    t0 = 0
    for b, n in enumerate(st["ns"]):
        ctx = st["lens"][b] - n
        hide = np.zeros((n, ctx + n), dtype=bool)
        for i in range(n):
            if c["tree"]:
                row = sum(int(w) << (64 * x) for x, w in enumerate(bits[t0 + i]))
                hide[i, ctx:] = [not row >> j & 1 for j in range(n)]
            else:
                hide[i, ctx + i + 1:] = True
        hide = torch.from_numpy(hide).to(DEV)
        ids = st["table"][b, :(ctx + n + page - 1) // page].long()
        for h in range(c["Hk"]):
            k = st["k_pages"][ids, h].reshape(-1, d)[:ctx + n].double()
            v = st["v_pages"][ids, h].reshape(-1, d)[:ctx + n].double()
            for g in range(h * G, (h + 1) * G):
                s = (st["q"][t0:t0 + n, g].double() @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                out[t0:t0 + n, g] = torch.softmax(s, dim=1) @ v
        t0 += n
    return out


def _exact_table(st):
    """Page by page, with a stack that is a list."""
    page = st["case"]["page"]
    table, free = st["table"].cpu().numpy().copy(), st["free"].cpu().numpy().copy()
    top = int(st["n_free"])
    cu, slots = [0], []
    for ctx, n in zip(st["ctx"], st["ns"]):
        cu.append(cu[-1] + n)
    for b, (ctx, n) in enumerate(zip(st["ctx"], st["ns"])):
        for p in range((ctx + page - 1) // page, (ctx + n + page - 1) // page):
            top -= 1
            table[b, p] = free[top]
        slots += [int(table[b, x // page]) * page + x % page for x in range(ctx, ctx + n)]
    # the way back leaves the table and the stack as they were
    as_ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    return (as_ints(cu), as_ints(st["ctx"]), torch.tensor(slots, dtype=torch.int64, device=DEV), st["table"],
            st["lengths"], st["free"], st["n_free"])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(st)
    if case["op"] == "table":
        return _exact_table(st)
    if case["op"] == "tree":
        parents, cu = st["parents"].tolist(), st["cu"].tolist()
        bits = _bits_of(np.array(parents, dtype=np.int64), cu, _words(case["n_hi"]))
        positions = []
        for b, start in enumerate(st["pos0"].tolist()):
            depth = []
            for p in parents[cu[b]:cu[b + 1]]:
                depth.append(depth[p] + 1 if p >= 0 else 0)
            positions += [start + x for x in depth]
        return torch.from_numpy(bits).to(DEV), torch.tensor(positions, dtype=torch.int32, device=DEV)
    outs = []
    table = st["table"].cpu().numpy()
    for pool in (st["k_pages"], st["v_pages"]):
        new = pool.clone()
        for b, path in enumerate(st["kept_lists"]):
            at = lambda x: (table[b, x // case["page"]], slice(None), x % case["page"])
            for i, j in enumerate(path):
                new[at(st["ctx"][b] + i)] = pool[at(st["ctx"][b] + int(j))]
        outs.append(new)
    return tuple(outs)
