"""Operators of a speculative decoding step whose drafted tokens form a tree, as they are measured.

A step verifies, for every request, T drafted tokens (nodes) at once.  Node i follows node parents[i] < i (-1: the
committed context), so several nodes share a position and each sees the context, its ancestors and itself.

* ``tree``: the nodes' masks and positions from their parents;
* ``append``: q and k rotated by their positions, k and v written into their pages (bf16, f32, or e4m3 with a scale a head);
* ``attention``: attention of the nodes over the paged context and the tree;
* ``commit``: the accepted path's K/V rows moved to the places behind the context;
* ``trim``: the rejected nodes' pages given back to the stack of free pages.

With ``own`` false ``run`` computes plain forms (elementary torch operations); with ``own`` true it makes
the framework's calls.
"""

import math
import random

import numpy as np
import torch

own = False

_DEV = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # The repository's drafted tokens as trees: 128 requests of 8 nodes, windows of none.
        _tree("tree_128x8", 128, 8, 8, 1, 0, 11),
        # Wide drafts: 64 requests of 100 to 256 nodes, masks of four words, every second request windowed.
        _tree("tree_64x256", 64, 100, 256, 4, -24, 12),
        # The rows of one such step (8 heads on one of 256), sliced out of one projection's output.
        _append("append_tree_1024", 1024, 8, 1, 256, 128, "bf16", "bf16", 256, False, True, 131072, 21),
        # A prompt's rows into 8-bit pages: 8192 tokens, 32 heads on 16 of 256.
        _append("append_prompt_8192", 8192, 32, 16, 256, 128, "bf16", "fp8", 256, False, False, 8192, 22),
        # The smallest call: one request, six nodes, a short context.
        _attn("attn_single_6", 4, 1, 64, 16, 1, 6, 6, 700, 700, 0, 31),
        # The repository's drafted tokens: 128 requests of 8 nodes over 120 to 2040 keys, 8 heads on one of 256.
        _attn("attn_128x8", 8, 1, 256, 128, 128, 8, 8, 120, 2040, 0, 32),
        # Long contexts with grouped heads: 32 requests of 16 to 48 nodes over 4k to 32k keys, 32 heads on 8 of 128.
        _attn("attn_long_32x48", 32, 8, 128, 64, 32, 16, 48, 4096, 32768, 0, 33),
        # Large trees, where the products count: 8 requests of 256 nodes over 2k to 8k keys, 64 heads on 8 of 128.
        _attn("attn_wide_8x256", 64, 8, 128, 128, 8, 256, 256, 2048, 8192, 0, 34),
        # The accepted paths of 128 requests of 8 nodes, one head of 256.
        _commit("commit_128x8", 128, 8, 8, 4, 1, 256, 128, "bf16", 41),
        # The same of 64 requests of 48 to 64 nodes, 16 heads of 256.
        _commit("commit_64x64", 64, 48, 64, 16, 16, 256, 128, "bf16", 42),
        # 512 requests drop what was rejected of 8 nodes each.
        _trim("trim_512", 512, 8, 4096, 16, 51),
        # 2048 requests drop what was rejected of up to 256 nodes.
        _trim("trim_2048", 2048, 256, 4096, 16, 52),
    ]


def _tree(name, seqs, lo, hi, words, window, lens):
    # `window` 0: none, w > 0: every request, w < 0: every second one.
    return {"name": name, "op": "tree", "seqs": seqs, "lo": lo, "hi": hi, "words": words, "window": window, "lens": lens}


def _append(name, tokens, hq, hkv, dim, page, dtype, kv, rotary, pairs, fused, reach, lens):
    # `pairs`: neighbouring dimensions turn together (else the two halves); `fused`: q, k and v are slices of one array.
    return {"name": name, "op": "append", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "page": page,
            "dtype": dtype, "kv": kv, "rotary": rotary, "pairs": pairs, "fused": fused, "reach": reach, "lens": lens}


def _attn(name, hq, hkv, dim, page, seqs, lo, hi, ctx_lo, ctx_hi, window, lens):
    return {"name": name, "op": "attention", "hq": hq, "hkv": hkv, "dim": dim, "page": page, "seqs": seqs, "lo": lo,
            "hi": hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "window": window, "lens": lens}


def _commit(name, seqs, lo, hi, most, hkv, dim, page, dtype, lens):
    # Requests of lo..hi nodes that keep 1..most of them.
    return {"name": name, "op": "commit", "seqs": seqs, "lo": lo, "hi": hi, "most": most, "hkv": hkv, "dim": dim,
            "page": page, "dtype": dtype, "lens": lens}


def _trim(name, seqs, drop, longest, page, lens):
    return {"name": name, "op": "trim", "seqs": seqs, "drop": drop, "longest": longest, "page": page, "lens": lens}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges that costs no more than the largest of them."""
    costs = [work(c) for c in listed()]
    while True:
        case = _draw(rng)
        cost = work(case)
        if all(cost[x] <= max(c[x] for c in costs) for x in ("bytes", "flops")):
            return case


def _draw(rng):
    what = rng.random()
    lens = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128, 256])
    window = rng.choice([0, 0, 1, -1])
    if what < 0.15:
        hi = _log_int(rng, 1, 256)
        case = _tree("", _log_int(rng, 1, 512), max(1, hi // 3), hi, -(-hi // 64) + rng.randrange(2),
                     window * _log_int(rng, 1, 64), lens)
    elif what < 0.4:
        dim = rng.choice([64, 128, 256])
        dtype, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "fp8"), ("f32", "f32"), ("f32", "fp8")])
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        most = min(8192, 8192 * 64 * 256 // ((hq + 2 * hkv) * dim * (2 if dtype == "f32" else 1)))
        case = _append("", _log_int(rng, 1, most), hq, hkv, dim, page, dtype, kv, dim // rng.choice([1, 1, 1, 2, 4]),
                       rng.random() < 0.3, rng.random() < 0.5, _log_int(rng, 1024, 1 << 20), lens)
    elif what < 0.75:
        dim = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
        seqs = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, 256)
        ctx = _log_int(rng, 16, 32768)
        # (The plain form holds every request padded to the longest, and their scores.)
        while seqs * (ctx + 512) * hkv * dim > 1 << 30 or seqs * hi * hq * (ctx + 512) > 1 << 32:
            if rng.random() < 0.5:
                seqs = max(1, seqs // 2)
            elif rng.random() < 0.5:
                ctx //= 2
            else:
                hi = max(1, hi // 2)
        case = _attn("", hq, hkv, dim, page, seqs, max(1, hi // 3), hi, rng.choice([0, ctx // 8, ctx]), ctx,
                     window * _log_int(rng, 16, 2048), lens)
    elif what < 0.88:
        hkv, dim, dtype = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 256]), rng.choice(["bf16", "f32", "fp8"])
        hi = _log_int(rng, 2, 256)
        seqs = _log_int(rng, 1, max(1, min(512, (1 << 28) // ((hi + 256) * hkv * dim))))
        case = _commit("", seqs, max(1, hi // 2), hi, _log_int(rng, 1, 24), hkv, dim, page, dtype, lens)
    else:
        case = _trim("", _log_int(rng, 1, 2048), _log_int(rng, 1, 256), _log_int(rng, 1, 4096), page, lens)
    del case["name"]
    return case


# ---------------------------------------------------------------- lengths

def _nodes(case):
    """Nodes of each request, and the context's length."""
    rng = random.Random(case["lens"])
    n = [rng.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    return n, [rng.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 4096)) for _ in n]


def _windows(case):
    w = case["window"]
    return None if w == 0 else [w if w > 0 else (-w if i % 2 == 0 else 0) for i in range(case["seqs"])]


def _kept(case):
    """Nodes that each request keeps: so many that the moved ones' places and sources differ."""
    n, _ = _nodes(case)
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(1, max(1, min(case["most"], (t + 1) // 2))) for t in n]


def _trim_lens(case):
    rng = random.Random(case["lens"])
    kv = [rng.randint(1, case["longest"]) for _ in range(case["seqs"])]
    return kv, [min(k, rng.randint(0, case["drop"])) for k in kv]


def _pages(n, page):
    return -(-n // page)


def _size(dtype):
    return {"bf16": 2, "f32": 4, "fp8": 1}[dtype]


def work(case):
    if case["op"] == "tree":
        n = sum(_nodes(case)[0])
        return {"bytes": n * (8.0 + 8.0 * case["words"]) + 8.0 * case["seqs"], "flops": float(n)}
    if case["op"] == "append":
        t, size, kv = case["tokens"], _size(case["dtype"]), _size(case["kv"])
        row = case["dim"] * (2.0 * size * case["hq"] + 2.0 * (size + kv) * case["hkv"])
        return {"bytes": t * (row + 12.0), "flops": 3.0 * t * (case["hq"] + case["hkv"]) * case["rotary"]}
    if case["op"] == "attention":
        n, ctx = _nodes(case)
        win = _windows(case) or [0] * len(n)
        # Of the tree each node counts itself (its ancestors are the input's); a window hides what no node sees.
        seen = [min(c, w - 1) if w > 0 else c for c, w in zip(ctx, win)]
        keys = sum(s + t for s, t in zip(seen, n))
        pairs = float(sum(t * (min(c, max(0, w - t)) if w > 0 else c) + t for t, c, w in zip(n, ctx, win)))
        data = 4.0 * keys * case["hkv"] * case["dim"] + 4.0 * sum(n) * case["hq"] * case["dim"]
        return {"bytes": data + 4.0 * sum(_pages(s + t, case["page"]) for s, t in zip(seen, n)) + 8.0 * sum(n),
                "flops": 4.0 * case["hq"] * case["dim"] * pairs}
    if case["op"] == "commit":
        moved = sum(k - 1 for k in _kept(case))
        row = float(case["hkv"] * case["dim"] * _size(case["dtype"]))
        return {"bytes": 4.0 * moved * row + 20.0 * sum(_kept(case)) + 4.0 * case["seqs"], "flops": 0.0}
    kv, drop = _trim_lens(case)
    moved = sum(_pages(k, case["page"]) - _pages(k - d, case["page"]) for k, d in zip(kv, drop))
    return {"bytes": 8.0 * moved + 12.0 * case["seqs"] + 8, "flops": float(moved + case["seqs"])}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    return {"tree": _prepare_tree, "append": _prepare_append, "attention": _prepare_attention,
            "commit": _prepare_commit, "trim": _prepare_trim}[case["op"]](case, gen, random.Random(seed))


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=_DEV)


def _sums(values):
    out = [0]
    for n in values:
        out.append(out[-1] + n)
    return out


def _workspace(st):
    if own:
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device=_DEV)
    return st


def _parents(n, rng):
    """Parents of a request's n nodes: a chain, a star, a tree of equal branches, or grown at random."""
    kind, branch = rng.randrange(5), rng.randint(2, 4)
    if kind == 0:
        return [i - 1 for i in range(n)]
    if kind == 1:
        return [min(0, i - 1) for i in range(n)]
    if kind == 2:
        return [-1] + [(i - 1) // branch for i in range(1, n)]
    if kind == 3:
        return [-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, n)]
    return [rng.randrange(-1, i) for i in range(n)]


def _prepare_tree(case, gen, rng):
    n, ctx = _nodes(case)
    win = _windows(case)
    parents = [p for t in n for p in _parents(t, rng)]
    st = {"op": "tree", "parents": _ints(parents), "cu": _ints(_sums(n)), "kv": _ints([c + t for c, t in zip(ctx, n)]),
          "win": None if win is None else _ints(win), "words": case["words"], "most": max(n),
          "mask": torch.zeros((len(parents), case["words"]), dtype=torch.int64, device=_DEV),
          "pos": torch.zeros(len(parents), dtype=torch.int32, device=_DEV)}
    return _workspace(st)


def _rows(shape, gen, dtype=torch.float32, key=False):
    """Rows as a projection leaves them: normal, and for keys a few channels several times larger."""
    x = torch.randn(shape, generator=gen, device=_DEV)
    if key:
        x[..., ::29] *= 4.0
    return x.to(dtype)


def _pool(shape, gen, dtype):
    """Pages that hold other rows already."""
    return torch.randn(shape, generator=gen, device=_DEV).to(_types()[dtype])


def _types():
    return {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}


def _prepare_append(case, gen, rng):
    t, hq, hkv, dim, page = case["tokens"], case["hq"], case["hkv"], case["dim"], case["page"]
    dt = _types()[case["dtype"]]
    x = _rows((t, hq + 2 * hkv, dim), gen, dt, key=True)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not case["fused"]:
        parts = tuple(p.contiguous() for p in parts)
    pool = _pages(t, page) + 3
    pages = torch.randperm(pool, generator=gen, device=_DEV)
    i = torch.arange(t, device=_DEV)
    # Consecutive slots of pages in any order; one token in thirty is padding.
    slots = pages[i // page] * page + i % page
    slots[torch.rand(t, generator=gen, device=_DEV) < 1 / 30] = -1
    half = case["rotary"] // 2
    st = {"op": "append", "q": parts[0], "k": parts[1], "v": parts[2], "slots": slots, "page": page,
          "pos": torch.randint(0, case["reach"], (t,), generator=gen, device=_DEV, dtype=torch.int32),
          "freq": (10000.0 ** (-torch.arange(half, device=_DEV, dtype=torch.float64) / half)).float(),
          "pairs": case["pairs"], "q_out": torch.empty((t, hq, dim), dtype=dt, device=_DEV),
          "k_pages": _pool((pool, page, hkv, dim), gen, case["kv"]),
          "v_pages": _pool((pool, page, hkv, dim), gen, case["kv"]), "k_scale": None, "v_scale": None}
    if case["kv"] == "fp8":
        for n in ("k_scale", "v_scale"):
            st[n] = 0.01 + 0.05 * torch.rand(hkv, generator=gen, device=_DEV)
    return _workspace(st)


def _prepare_attention(case, gen, rng):
    n, ctx = _nodes(case)
    win = _windows(case)
    kv = [c + t for c, t in zip(ctx, n)]
    page, hkv, dim = case["page"], case["hkv"], case["dim"]
    held = [_pages(m, page) for m in kv]
    pool = sum(held) + 2
    perm = torch.randperm(pool, generator=gen, device=_DEV, dtype=torch.int32)
    table = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device=_DEV)
    row = torch.repeat_interleave(torch.arange(len(kv)), torch.tensor(held)).to(_DEV)
    col = torch.cat([torch.arange(h) for h in held]).to(_DEV)
    table[row, col] = perm[:sum(held)]
    words = _pages(max(n), 64)
    parents = [p for t in n for p in _parents(t, rng)]
    mask, depth = _walk(parents, n, win, words)
    cu = _sums(n)
    st = {"op": "attention", "page": page, "hkv": hkv, "scale": dim ** -0.5, "table": table, "cu": _ints(cu),
          "kv": _ints(kv), "win": None if win is None else _ints(win), "most": max(n),
          "mask": torch.from_numpy(mask).to(_DEV),
          "pos": _ints([c + d for c, t, d0 in zip(ctx, n, cu) for d in depth[d0:d0 + t]]),
          "q": _rows((cu[-1], case["hq"], dim), gen, torch.bfloat16)}
    for x in ("k", "v"):
        pages = torch.empty((pool, page, hkv, dim), dtype=torch.bfloat16, device=_DEV)
        step = max(1, (1 << 27) // (hkv * page * dim))
        for p0 in range(0, pool, step):
            pages[p0:p0 + step] = _rows(pages[p0:p0 + step].shape, gen, key=x == "k")
        st[x + "_pages"] = pages
    if own:
        from ragged_paged_attention_rpa_gb300 import binding
        plan = binding.rpa_plan(np.array(cu, dtype=np.int32), np.array(kv, dtype=np.int32),
                                None if win is None else np.array(win, dtype=np.int32), case["hq"], hkv, dim, page,
                                table.shape[1], pool, tree_words=words)
        st.update(plan=plan, ws=binding.alloc_workspace(plan), out=torch.empty_like(st["q"]))
    return st


def _walk(parents, n, win, words):
    """Masks [nodes, words] (int64) and depths of the nodes, on the host."""
    mask = np.zeros((len(parents), words), dtype=np.uint64)
    depth, t0 = [], 0
    for s, t in enumerate(n):
        w = win[s] if win and win[s] > 0 else t
        for i in range(t):
            p = parents[t0 + i]
            depth.append(0 if p < 0 else depth[t0 + p] + 1)
            j, d = i, 0
            while j >= 0 and d < w:
                mask[t0 + i, j // 64] |= np.uint64(1 << (j % 64))
                j, d = parents[t0 + j], d + 1
        t0 += t
    return mask.view(np.int64), depth


def _prepare_commit(case, gen, rng):
    n, _ = _nodes(case)
    keep, page = _kept(case), case["page"]
    width = max(keep)
    path = torch.full((len(n), width), -1, dtype=torch.int32)
    for s, (t, k) in enumerate(zip(n, keep)):
        path[s, :k] = torch.tensor([0] + sorted(rng.sample(range(k, t), k - 1)), dtype=torch.int32)
    total = sum(n)
    pool = _pages(total, page) + 3
    pages = torch.randperm(pool, generator=gen, device=_DEV)
    i = torch.arange(total, device=_DEV)
    shape = (pool, page, case["hkv"], case["dim"])
    st = {"op": "commit", "cu": _ints(_sums(n)), "path": path.to(_DEV), "page": page,
          "slots": pages[i // page] * page + i % page, "k_pages": _pool(shape, gen, case["dtype"]),
          "v_pages": _pool(shape, gen, case["dtype"])}
    return _workspace(st)


def _prepare_trim(case, gen, rng):
    kv, drop = _trim_lens(case)
    page, seqs = case["page"], case["seqs"]
    held = [_pages(k, page) for k in kv]
    spare = 5
    pool = sum(held) + spare
    perm = torch.randperm(pool, generator=gen, device=_DEV, dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(seqs), torch.tensor(held)).to(_DEV)
    col = torch.cat([torch.arange(h) for h in held]).to(_DEV)
    table = torch.full((seqs, max(held)), -1, dtype=torch.int32, device=_DEV)
    table[row, col] = perm[:sum(held)]
    free = torch.full((pool,), -1, dtype=torch.int32, device=_DEV)
    free[:spare] = perm[sum(held):]
    st = {"op": "trim", "page": page, "table": table, "free": free, "count": _ints([spare]), "count_out": _ints([0]),
          "kv_prev": _ints(kv), "drop": _ints(drop), "kv": torch.zeros(seqs, dtype=torch.int32, device=_DEV)}
    return _workspace(st)


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        return _run_own(st)
    return {"tree": _plain_tree, "append": _plain_append, "attention": _plain_attention, "commit": _plain_commit,
            "trim": _plain_trim}[st["op"]](st)


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _run_own(st):
    from ragged_paged_attention_rpa_gb300 import binding
    op = st["op"]
    if op == "tree":
        binding.rpa_build_tree(st["parents"], st["cu"], st["kv"], st["win"], st["mask"], st["pos"], st["ws"])
        return st["mask"], st["pos"]
    if op == "append":
        binding.rpa_append_rope(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["freq"], st["q_out"],
                                _bytes(st["k_pages"]), _bytes(st["v_pages"]), k_scale=st["k_scale"],
                                v_scale=st["v_scale"], interleaved=st["pairs"], workspace=st["ws"])
        return st["q_out"], st["k_pages"], st["v_pages"]
    if op == "commit":
        binding.rpa_commit_tree(_bytes(st["k_pages"]), _bytes(st["v_pages"]), st["slots"], st["cu"], st["path"], st["ws"])
        return st["k_pages"], st["v_pages"]
    if op == "trim":
        binding.rpa_trim_tables(st["drop"], st["kv_prev"], st["table"], st["free"], st["count"], st["kv"],
                                st["count_out"], st["page"], st["ws"])
        return st["free"], st["kv"], st["count_out"]
    binding.rpa_forward_tree(st["q"], st["k_pages"], st["v_pages"], st["table"], st["cu"], st["kv"], st["mask"],
                             None if st["win"] is None else st["pos"], st["win"], st["scale"], st["out"], st["plan"],
                             st["ws"])
    return st["out"]


def _owner(cu, total):
    """The request of each of `total` nodes."""
    return torch.searchsorted(cu[1:].long(), torch.arange(total, device=_DEV), right=True)


def _plain_tree(st):
    cu, par, most, words = st["cu"].long(), st["parents"].long(), st["most"], st["words"]
    total, seqs = par.shape[0], cu.shape[0] - 1
    s = _owner(cu, total)
    i = torch.arange(total, device=_DEV) - cu[s]
    # One step to the parent as a matrix a request, the closure by squaring (1, 2, 4, ... steps).
    reach = torch.zeros((seqs, most, most), device=_DEV)
    reach[s, i, i] = 1.0
    up = par >= 0
    reach[s[up], i[up], par[up]] = 1.0
    reach = _closure(reach, (most - 1).bit_length())
    depth = (reach.sum(-1) - 1).long()
    if st["win"] is not None:
        w = st["win"].long()[:, None, None]
        far = depth[:, :, None] - depth[:, None, :] >= w
        reach = torch.where((w > 0) & far, torch.zeros_like(reach), reach)
    bits = torch.nn.functional.pad(reach.long(), (0, words * 64 - most))
    bits = bits.unflatten(-1, (words, 64)) << torch.arange(64, device=_DEV)
    st["mask"].copy_(bits.sum(-1)[s, i])
    st["pos"].copy_(st["kv"].long()[s] - (cu[s + 1] - cu[s]) + depth[s, i])
    return st["mask"], st["pos"]


def _closure(reach, squarings):
    return reach if squarings == 0 else _closure(torch.matmul(reach, reach).clamp_(max=1.0), squarings - 1)


def _turned(x, c, s, pairs):
    """Rows x [t, heads, dim] (float32) with their first dimensions turned; c, s [t, 1, rotary / 2]."""
    half = c.shape[-1]
    if pairs:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _plain_append(st):
    angle = (st["pos"].double()[:, None] * st["freq"].double()[None])[:, None]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    st["q_out"].copy_(_turned(st["q"].float(), c, s, st["pairs"]))
    use = st["slots"] >= 0
    at = st["slots"][use]
    page, slot = at // st["page"], at % st["page"]
    for n, x in (("k", _turned(st["k"].float(), c, s, st["pairs"])), ("v", st["v"].float())):
        if st[n + "_scale"] is not None:
            x = (x / st[n + "_scale"][None, :, None]).clamp(-448.0, 448.0)
        _bytes(st[n + "_pages"])[page, slot] = _bytes(x[use].to(st[n + "_pages"].dtype))
    return st["q_out"], st["k_pages"], st["v_pages"]


def _plain_attention(st):
    q, page, hkv, most = st["q"], st["page"], st["hkv"], st["most"]
    total, hq, dim = q.shape
    group, seqs = hq // hkv, st["kv"].shape[0]
    cu, kv = st["cu"].long(), st["kv"].long()
    s = _owner(cu, total)
    i = torch.arange(total, device=_DEV) - cu[s]
    rows = torch.zeros((seqs, most, hq, dim), device=_DEV)
    rows[s, i] = q.float()
    rows = rows.view(seqs, most, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, most * group, dim)
    at = st["table"].long().clamp(min=0)
    k, v = (st[x + "_pages"][at].flatten(1, 2).transpose(1, 2).float() for x in ("k", "v"))
    keys = k.shape[2]
    j = torch.arange(keys, device=_DEV)
    ctx = (kv - (cu[1:] - cu[:-1]))[s][:, None]
    node = j[None] - ctx
    word = (node // 64).clamp(0, st["mask"].shape[1] - 1)
    seen = ((torch.gather(st["mask"], 1, word) >> (node % 64)) & 1) != 0
    before = torch.ones_like(seen)
    if st["win"] is not None:
        w = st["win"].long()[s][:, None]
        before = (w <= 0) | (st["pos"].long()[:, None] - j[None] < w)
    seen = torch.where(node < 0, before, seen & (j[None] < kv[s][:, None]))
    hide = torch.ones((seqs, most, keys), dtype=torch.bool, device=_DEV)
    hide[s, i] = ~seen
    a = torch.matmul(rows, k.transpose(2, 3)).mul_(st["scale"])
    a = a.view(seqs, hkv, most, group, keys).masked_fill_(hide[:, None, :, None], float("-inf"))
    top = a.amax(-1, keepdim=True)
    a = a.sub_(torch.where(top == float("-inf"), torch.zeros_like(top), top)).exp_()
    total_p = a.sum(-1, keepdim=True)
    o = torch.matmul(a.view(seqs, hkv, most * group, keys), v).view(seqs, hkv, most, group, dim)
    o = torch.where(total_p > 0, o / total_p, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4)[s, i].reshape(total, hq, dim).to(q.dtype)


def _plain_commit(st):
    path, cu = st["path"].long(), st["cu"].long()
    use = path >= 0
    base = cu[:-1, None].expand_as(path)
    to = st["slots"][(base + torch.arange(path.shape[1], device=_DEV)[None])[use]]
    src = st["slots"][(base + path)[use]]
    for n in ("k_pages", "v_pages"):
        flat = _bytes(st[n]).flatten(0, 1)
        flat[to] = flat[src]
    return st["k_pages"], st["v_pages"]


def _plain_trim(st):
    p, table, free = st["page"], st["table"], st["free"]
    old = st["kv_prev"].long()
    left = old - st["drop"].long()
    first, last = (left + p - 1) // p, (old + p - 1) // p
    n = last - first
    base = n.cumsum(0) - n
    count = st["count"].long()
    col = torch.arange(table.shape[1], device=_DEV)[None]
    gone = (col >= first[:, None]) & (col < last[:, None])
    at = torch.where(gone, count + base[:, None] + col - first[:, None], torch.full_like(col, free.shape[0]))
    grown = torch.cat([free, free[:1]])
    grown[at.flatten()] = table.flatten()
    free.copy_(grown[:-1])
    st["kv"].copy_(left)
    st["count_out"].copy_(count + n.sum())
    return free, st["kv"], st["count_out"]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "tree":
        return _exact_tree(case, st)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "commit":
        return _exact_commit(st)
    if case["op"] == "trim":
        return _exact_trim(st)
    return _exact_attention(case, st)


def _exact_tree(case, st):
    n, _ = _nodes(case)
    mask, depth = _walk(st["parents"].tolist(), n, _windows(case), case["words"])
    left = [m - t for m, t in zip(st["kv"].tolist(), n) for _ in range(t)]
    return torch.from_numpy(mask).to(_DEV), _ints([c + d for c, d in zip(left, depth)])


def _exact_append(case, st):
    half, dim = case["rotary"] // 2, case["dim"]
    first = torch.arange(half, device=_DEV) * (2 if case["pairs"] else 1)
    second = first + (1 if case["pairs"] else half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV).expand(case["tokens"], half).contiguous(),
                       st["pos"].double()[:, None] * st["freq"].double()[None])

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = [turned(st["q"])]
    for n, x in (("k", turned(st["k"])), ("v", st["v"].double())):
        pages = st[n + "_pages"].double()
        if st[n + "_scale"] is not None:
            x = _nearest_e4m3(x / st[n + "_scale"].double()[None, :, None])
        flat = pages.flatten(0, 1)
        use = st["slots"] >= 0
        flat[st["slots"][use]] = x[use]
        out.append(pages)
    return tuple(out)


def _nearest_e4m3(x):
    """The nearest number of 3 mantissa bits from 2^-9 to 448 (ties to even)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.pow(2.0, e) > x.abs().clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= x.abs(), e + 1, e)
    step = torch.pow(2.0, e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_commit(st):
    cu, path, slots = st["cu"].tolist(), st["path"].tolist(), st["slots"].tolist()
    to, src = [], []
    for s, row in enumerate(path):
        for k, j in enumerate(row):
            if j >= 0:
                to.append(slots[cu[s] + k])
                src.append(slots[cu[s] + j])
    out = []
    for n in ("k_pages", "v_pages"):
        pages = st[n].double()
        flat = pages.flatten(0, 1)
        flat[_ints(to, torch.int64)] = flat[_ints(src, torch.int64)].clone()
        out.append(pages)
    return tuple(out)


def _exact_trim(st):
    p, table = st["page"], st["table"].cpu().numpy()
    free, count = st["free"].cpu().numpy().copy(), int(st["count"])
    kv = st["kv_prev"].tolist()
    for s, d in enumerate(st["drop"].tolist()):
        for j in range(_pages(kv[s] - d, p), _pages(kv[s], p)):
            free[count] = table[s, j]
            count += 1
        kv[s] -= d
    return torch.as_tensor(free, device=_DEV), _ints(kv), _ints([count])


def _exact_attention(case, st):
    n, ctx = _nodes(case)
    page, hkv, group, dim = case["page"], case["hkv"], case["hq"] // case["hkv"], case["dim"]
    win = _windows(case) or [0] * len(n)
    bits = st["mask"].cpu().numpy().view(np.uint8)
    pos = st["pos"].tolist()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=_DEV)
    t0 = 0
    for s, (t, c) in enumerate(zip(n, ctx)):
        rows = st["table"][s, :_pages(c + t, page)].long()
        seen = torch.ones((t, c + t), dtype=torch.bool, device=_DEV)
        tree = np.unpackbits(bits[t0:t0 + t], axis=1, bitorder="little")[:, :t]
        seen[:, c:] = torch.from_numpy(tree.astype(bool)).to(_DEV)
        if win[s] > 0:
            back = _ints(pos[t0:t0 + t])[:, None] - torch.arange(c, device=_DEV)[None]
            seen[:, :c] &= back < win[s]
        for g in range(hkv):
            k, v = (st[x + "_pages"][rows, :, g].flatten(0, 1)[:c + t].double() for x in ("k", "v"))
            q = st["q"][t0:t0 + t, g * group:(g + 1) * group].double()
            a = torch.einsum("tgd,kd->tgk", q, k) * case["dim"] ** -0.5
            a = a.masked_fill(~seen[:, None], -math.inf)
            out[t0:t0 + t, g * group:(g + 1) * group] = torch.einsum("tgk,kd->tgd", torch.softmax(a, -1), v)
        t0 += t
    return out
