"""Operators of a paged KV cache held in 4 bits, as they are measured.

Three operators that a serving step runs one after the other:

* ``tables``: the step's page table, slot map and lengths from the requests' lengths, on the GPU
  (and the return of finished requests' pages to the free stack);
* ``cache``: the step's K and V rows written into 4-bit pages, and rows taken back as values;
* ``attention``: ragged paged attention over those pages.

The cache's format: blocks of 16 dimensions, one 4-bit code (sign, 2 exponent bits, 1 mantissa bit:
0, .5, 1, 1.5, 2, 3, 4, 6) a dimension, two to a byte with the even dimension in the low half, and one
8-bit scale a block (5 exponent bits of bias 15, 3 mantissa bits, no sign; 255 is NaN).  The scale is
max|x| / 6, rounded to nearest even and at most 10240; a code is x / scale, rounded to nearest even and at
most 6; a block that holds a NaN or an infinity reads as NaN.  Pages are [page, KV head, slot, dimension].

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
        # One decode step of the repository's mixed batch: 512 requests, one new token each.
        _tables("tables_decode_512", 512, 1, 1, 256, 4096, 128, 512, 11),
        # Admission of prompts: 192 new requests of up to 2048 tokens, nothing cached before.
        _tables("tables_prompts_192", 192, 1, 2048, 0, 0, 128, 262144, 12),
        # The end of 300 of 2048 requests: their pages go back to the free stack.
        dict(_tables("tables_release_2048", 2048, 1, 1, 1, 4096, 16, 0, 13), release=True),
        # The K/V rows of one decode step (512 requests, one 256-wide KV head).
        _cache("cache_decode_512", 512, 1, 1, 256, 128, "bf16", 21),
        # The rows of an 8192-token prompt, 16 KV heads of 256.
        _cache("cache_prompt_8192", 8192, 8192, 16, 256, 128, "bf16", 22),
        # An odd number of rows in float32, as the fp32 debug build has them.
        _cache("cache_f32_777", 777, 37, 4, 64, 16, "f32", 23),
        # The smallest call: one request, one token, a short context.
        _attn("attn_single_700", 4, 1, 64, 16, 1, 700, 700, 0, 1, 1, 0, 0, 0, 31),
        # The repository's decode batch: 128 requests of 128 to 2048 tokens, 8 heads on one of 256.
        _attn("attn_decode_128", 8, 1, 256, 128, 128, 128, 2048, 0, 1, 1, 0, 0, 0, 32),
        # Long contexts with grouped heads: 32 requests of 4k to 32k tokens, 32 heads on 8 of 128.
        _attn("attn_decode_long", 32, 8, 128, 64, 32, 4096, 32768, 0, 1, 1, 0, 0, 0, 33),
        # Verification of drafted tokens: 128 requests of 8 new tokens each.
        _attn("attn_drafted_128x8", 8, 1, 256, 128, 0, 0, 0, 128, 8, 8, 120, 2040, 0, 34),
        # The repository's mixed batch: 512 decoding requests and 4 chunks of 2048, every second one windowed.
        _attn("attn_mixed_512_4", 8, 1, 256, 128, 512, 256, 4096, 4, 2048, 2048, 0, 4096, -1024, 35),
        # The repository's causal prompt: 8192 tokens, 32 heads on 16 of 256.
        _attn("attn_prompt_8192", 32, 16, 256, 128, 0, 0, 0, 1, 8192, 8192, 0, 0, 0, 36),
    ]


def _tables(name, seqs, new_lo, new_hi, old_lo, old_hi, page, room, lens):
    return {"name": name, "op": "tables", "release": False, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi,
            "old_lo": old_lo, "old_hi": old_hi, "page": page, "room": room, "lens": lens}


def _cache(name, tokens, run_len, hkv, dim, page, dtype, lens):
    # `run_len`: consecutive tokens of one request (1: a decode step; all: one prompt).
    return {"name": name, "op": "cache", "tokens": tokens, "run_len": run_len, "hkv": hkv, "dim": dim,
            "page": page, "dtype": dtype, "lens": lens}


def _attn(name, hq, hkv, dim, page, dec, dec_lo, dec_hi, chunks, new_lo, new_hi, prior_lo, prior_hi, window, lens):
    # `dec` requests of one new token over dec_lo..dec_hi keys, then `chunks` requests of new_lo..new_hi new
    # tokens after prior_lo..prior_hi cached ones; window 0: none, w > 0: every request, w < 0: every second one.
    return {"name": name, "op": "attention", "hq": hq, "hkv": hkv, "dim": dim, "page": page, "dec": dec,
            "dec_lo": dec_lo, "dec_hi": dec_hi, "chunks": chunks, "new_lo": new_lo, "new_hi": new_hi,
            "prior_lo": prior_lo, "prior_hi": prior_hi, "window": window, "lens": lens}


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
    if what < 0.25:
        seqs = _log_int(rng, 1, 2048)
        if rng.random() < 0.3:
            case = dict(_tables("", seqs, 1, 1, 1, _log_int(rng, 1, 4096), page, 0, lens), release=True)
        elif rng.random() < 0.5:
            new = _log_int(rng, 1, 16)
            case = _tables("", seqs, 0, new, 0, _log_int(rng, 1, 4096), page, seqs * new, lens)
        else:
            seqs = min(seqs, 192)
            new = _log_int(rng, 16, 2048)
            # Some room behind the last token, as a call captured for the largest step has.
            case = _tables("", seqs, 0, new, 0, _log_int(rng, 1, 2048), page, min(262144, seqs * new + rng.randrange(64)),
                           lens)
    elif what < 0.5:
        dim = rng.choice([64, 128, 256])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        most = 8192 * 16 * 256 // (hkv * dim * (2 if dtype == "f32" else 1))
        tokens = _log_int(rng, 1, min(most, 8192))
        case = _cache("", tokens, rng.choice([1, _log_int(rng, 1, tokens), tokens]), hkv, dim, page, dtype, lens)
    else:
        dim = rng.choice([64, 128, 256])
        hkv = rng.choice([1, 1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8, 8, 16])
        window = rng.choice([0, 0, 1, -1]) * _log_int(rng, 16, 2048)
        kind = rng.random()
        if kind < 0.45:
            seqs = _log_int(rng, 1, 512)
            hi = _log_int(rng, 1, min(32768, max(64, 600000 // seqs)))
            args = (seqs, max(1, hi // 16), hi, 0, 1, 1, 0, 0)
        elif kind < 0.65:
            seqs = _log_int(rng, 1, 128)
            new = rng.randrange(2, 17)
            prior = _log_int(rng, 1, 2048)
            args = (0, 0, 0, seqs, 1, new, prior // 16, prior)
        elif kind < 0.85:
            new = _log_int(rng, 17, 4096)
            prior = _log_int(rng, 1, 2048)
            args = (0, 0, 0, rng.randrange(1, 5), max(1, new // 4), new, 0, prior)
        else:
            hi = _log_int(rng, 64, 4096)
            new = _log_int(rng, 17, 2048)
            args = (_log_int(rng, 1, 256), max(1, hi // 16), hi, rng.randrange(1, 4), max(1, new // 4), new, 0, hi)
        case = _attn("", hq, hkv, dim, page, *args, window, lens)
    del case["name"]
    return case


# ---------------------------------------------------------------- lengths

def _table_lens(case):
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    old = [rng.randint(case["old_lo"], case["old_hi"]) for _ in range(case["seqs"])]
    done = [rng.random() < 300 / 2048 for _ in range(case["seqs"])]
    while not case["release"] and sum(new) > case["room"]:  # a full step: the last requests wait
        new[max(i for i, n in enumerate(new) if n)] = 0
    return new, old, done


def _attn_lens(case):
    rng = random.Random(case["lens"])
    new = [1] * case["dec"]
    kv = [rng.randint(case["dec_lo"], case["dec_hi"]) for _ in range(case["dec"])]
    for _ in range(case["chunks"]):
        n = rng.randint(case["new_lo"], case["new_hi"])
        new.append(n)
        kv.append(n + rng.randint(case["prior_lo"], case["prior_hi"]))
    w = case["window"]
    win = None if w == 0 else [w if w > 0 else (-w if i % 2 == 0 else 0) for i in range(len(kv))]
    return new, kv, win


def _pages(n, page):
    return -(-n // page)


def _per_elem():
    return 0.5 + 1.0 / 16  # bytes of a cached element: a code and its share of the block's scale


def work(case):
    if case["op"] == "tables":
        new, old, done = _table_lens(case)
        p = case["page"]
        if case["release"]:
            moved = sum(_pages(o, p) for o, d in zip(old, done) if d)
            return {"bytes": 8.0 * moved + 12.0 * case["seqs"] + 8, "flops": float(moved + case["seqs"])}
        fresh = sum(_pages(o + n, p) - _pages(o, p) for o, n in zip(old, new))
        partly = sum(1 for o, n in zip(old, new) if n and o % p)
        return {"bytes": 8.0 * case["room"] + 8.0 * fresh + 4.0 * partly + 16.0 * case["seqs"] + 12,
                "flops": float(case["room"] + fresh + 3 * case["seqs"])}
    if case["op"] == "cache":
        n = 2.0 * case["tokens"] * case["hkv"] * case["dim"]
        size = 2 if case["dtype"] == "bf16" else 4
        # Rows in, their pages written; the rows' values out.
        return {"bytes": n * (2 * size + _per_elem()) + 8.0 * case["tokens"], "flops": 4.0 * n}
    new, kv, win = _attn_lens(case)
    flops, keys, queries = 0.0, 0, sum(new)
    for s, (n, m) in enumerate(zip(new, kv)):
        w = win[s] if win and win[s] > 0 else m
        first = m - n + 1  # keys up to the first query
        seen = sum(min(first + i, w) for i in range(n)) if w < m else n * first + n * (n - 1) // 2
        flops += 4.0 * case["hq"] * case["dim"] * seen
        keys += min(m, n - 1 + w)
    data = 2.0 * keys * case["hkv"] * case["dim"] * _per_elem() + 4.0 * queries * case["hq"] * case["dim"]
    return {"bytes": data + 4.0 * sum(_pages(m, case["page"]) for m in kv), "flops": flops}


# ---------------------------------------------------------------- the format, plainly

def _quantise(x):
    """Codes [..., D / 2] and scales [..., D / 16] (uint8) of rows [..., D]."""
    b = x.float().unflatten(-1, (-1, 16))
    top = b.abs().amax(-1)
    t = top / 6
    e = torch.frexp(t)[1] - 1
    step = torch.ldexp(torch.ones_like(t), e.clamp(min=-14) - 3)
    s = (torch.round(t / step) * step).clamp(max=10240.0)
    good = torch.isfinite(top)
    use = (good & (s > 0)).unsqueeze(-1)
    v = torch.where(use, b / s.unsqueeze(-1), torch.zeros_like(b))
    a = v.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int()) + 8 * (v < 0).int()
    code = code.flatten(-2)
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    bits = torch.where(good, s, torch.zeros_like(s)).half().view(torch.int16).int() >> 7
    return packed, torch.where(good, bits, torch.full_like(bits, 255)).to(torch.uint8)


def _values(packed, scales):
    """Values [..., D] (float32) of codes [..., D / 2] and scales [..., D / 16]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                       device=packed.device)
    p = packed.long()
    v = torch.stack([lut[p & 15], lut[p >> 4]], -1).flatten(-2)
    s = (scales.int() << 7).to(torch.int16).view(torch.float16).float()
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(seed)
    return {"tables": _prepare_tables, "cache": _prepare_cache, "attention": _prepare_attention}[case["op"]](
        case, gen)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=_DEV)


def _prepare_tables(case, gen):
    new, old, done = _table_lens(case)
    page, seqs = case["page"], case["seqs"]
    held = [_pages(o, page) for o in old]
    need = [_pages(o + n, page) for o, n in zip(old, new)]
    width = max(1, max(need))
    spare = sum(need) - sum(held) + 3
    pool = sum(held) + spare
    perm = torch.randperm(pool, generator=gen, device=_DEV, dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(seqs), torch.tensor(held)).to(_DEV)
    col = torch.cat([torch.arange(n) for n in held] + [torch.arange(0)]).to(_DEV)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=_DEV)
    table[row, col] = perm[:sum(held)]
    free = torch.full((pool,), -1, dtype=torch.int32, device=_DEV)
    free[:spare] = perm[sum(held):]
    st = {"op": "release" if case["release"] else "tables", "page": page, "table": table, "free": free,
          "count": _ints([spare]), "count_out": _ints([0]), "kv_prev": _ints(old),
          "kv": torch.zeros(seqs, dtype=torch.int32, device=_DEV)}
    if case["release"]:
        st["done"] = _ints([1 if d else 0 for d in done])
    else:
        st["new"] = _ints(new)
        st["cu"] = torch.zeros(seqs + 1, dtype=torch.int32, device=_DEV)
        st["slots"] = torch.zeros(case["room"], dtype=torch.int64, device=_DEV)
    if own:
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device=_DEV)
    return st


def _rows(shape, gen, dtype=torch.float32, key=False):
    """Rows as a projection leaves them: normal, and for keys a few channels several times larger."""
    x = torch.randn(shape, generator=gen, device=_DEV)
    if key:
        x[..., ::29] *= 4.0
    return x.to(dtype)


def _prepare_cache(case, gen):
    t, page, run_len = case["tokens"], case["page"], case["run_len"]
    reqs = _pages(t, run_len)
    per = _pages(run_len + page - 1, page)  # pages a request can touch
    pool = reqs * per + 3
    pages = torch.randperm(pool, generator=gen, device=_DEV)[:reqs * per].view(reqs, per)
    start = torch.randint(0, page, (reqs,), generator=gen, device=_DEV)
    i = torch.arange(t, device=_DEV)
    r, pos = i // run_len, start[i // run_len] + i % run_len
    slots = pages[r, pos // page] * page + pos % page
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    shape = (t, case["hkv"], case["dim"])
    st = {"op": "cache", "k": _rows(shape, gen, dt, key=True), "v": _rows(shape, gen, dt), "slots": slots}
    for n in ("k", "v"):
        st[n + "_pages"] = torch.zeros((pool, case["hkv"], page, case["dim"] // 2), dtype=torch.uint8, device=_DEV)
        st[n + "_scales"] = torch.zeros((pool, case["hkv"], page, case["dim"] // 16), dtype=torch.uint8, device=_DEV)
    if own:
        st["k_out"], st["v_out"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    return st


def _prepare_attention(case, gen):
    new, kv, win = _attn_lens(case)
    page, hkv, dim = case["page"], case["hkv"], case["dim"]
    held = [_pages(n, page) for n in kv]
    pool = sum(held) + 2
    perm = torch.randperm(pool, generator=gen, device=_DEV, dtype=torch.int32)
    table = torch.full((len(kv), max(held)), -1, dtype=torch.int32, device=_DEV)
    row = torch.repeat_interleave(torch.arange(len(kv)), torch.tensor(held)).to(_DEV)
    col = torch.cat([torch.arange(n) for n in held]).to(_DEV)
    table[row, col] = perm[:sum(held)]
    st = {"op": "attention", "page": page, "hkv": hkv, "scale": dim ** -0.5, "table": table, "new": new,
          "kv_host": kv, "win_host": win}
    for n in ("k", "v"):
        codes = torch.empty((pool, hkv, page, dim // 2), dtype=torch.uint8, device=_DEV)
        scales = torch.empty((pool, hkv, page, dim // 16), dtype=torch.uint8, device=_DEV)
        step = max(1, (1 << 25) // (hkv * page * dim))
        for p0 in range(0, pool, step):
            m = min(step, pool - p0)
            codes[p0:p0 + m], scales[p0:p0 + m] = _quantise(_rows((m, hkv, page, dim), gen, key=n == "k"))
        st[n + "_pages"], st[n + "_scales"] = codes, scales
    st["q"] = _rows((sum(new), case["hq"], dim), gen, torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    if own:
        from ragged_paged_attention_rpa_gb300 import binding
        plan = binding.rpa_plan(np.array(cu, dtype=np.int32), np.array(kv, dtype=np.int32),
                                None if win is None else np.array(win, dtype=np.int32), case["hq"], hkv, dim, page,
                                table.shape[1], pool, kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
        st.update(plan=plan, ws=binding.alloc_workspace(plan), cu=_ints(cu), kv=_ints(kv),
                  win=None if win is None else _ints(win), out=torch.empty_like(st["q"]))
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        return _run_own(st)
    return {"tables": _plain_tables, "release": _plain_release, "cache": _plain_cache,
            "attention": _plain_attention}[st["op"]](st)


def _run_own(st):
    from ragged_paged_attention_rpa_gb300 import binding
    op = st["op"]
    if op == "tables":
        binding.rpa_build_tables(st["new"], st["kv_prev"], st["table"], st["free"], st["count"], st["cu"], st["kv"],
                                 st["slots"], st["count_out"], st["page"], st["ws"])
        return st["table"], st["cu"], st["kv"], st["slots"], st["count_out"]
    if op == "release":
        binding.rpa_release_tables(st["done"], st["kv_prev"], st["table"], st["free"], st["count"], st["kv"],
                                   st["count_out"], st["page"], st["ws"])
        return st["free"], st["kv"], st["count_out"]
    if op == "cache":
        pools = (st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"])
        binding.rpa_write_kv4(st["k"], st["v"], *pools, st["slots"])
        binding.rpa_read_kv4(*pools, st["slots"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    binding.rpa_forward_kv4(st["q"], st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"], st["table"],
                            st["cu"], st["kv"], st["win"], st["scale"], st["out"], st["plan"], st["ws"])
    return st["out"]


def _plain_tables(st):
    p, table, free = st["page"], st["table"], st["free"]
    new, old = st["new"].long(), st["kv_prev"].long()
    held = (old + p - 1) // p
    want = (old + new + p - 1) // p
    need = want - held
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    base = need.cumsum(0) - need
    count = st["count"].long()
    room = st["slots"].shape[0]
    ok = (need.sum() <= count) & (cu[-1] <= room)
    col = torch.arange(table.shape[1], device=_DEV)[None]
    k = base[:, None] + col - held[:, None]
    fresh = (col >= held[:, None]) & (col < want[:, None]) & ok
    table.copy_(torch.where(fresh, free[(count - 1 - k).clamp(0, free.shape[0] - 1)], table))
    t = torch.arange(room, device=_DEV)
    s = torch.searchsorted(cu[1:], t, right=True).clamp(max=new.shape[0] - 1)
    pos = old[s] + t - cu[s]
    page = table[s, (pos // p).clamp(max=table.shape[1] - 1)].long()
    st["slots"].copy_(torch.where((t < cu[-1]) & ok, page * p + pos % p, torch.full_like(t, -1)))
    st["cu"].copy_(torch.where(ok, cu, torch.zeros_like(cu)))
    st["kv"].copy_(torch.where(ok, old + new, old))
    st["count_out"].copy_(torch.where(ok, count - need.sum(), count))
    return table, st["cu"], st["kv"], st["slots"], st["count_out"]


def _plain_release(st):
    p, table, free = st["page"], st["table"], st["free"]
    old, done = st["kv_prev"].long(), st["done"] != 0
    n = torch.where(done, (old + p - 1) // p, torch.zeros_like(old))
    base = n.cumsum(0) - n
    count = st["count"].long()
    col = torch.arange(table.shape[1], device=_DEV)[None]
    at = torch.where(col < n[:, None], count + base[:, None] + col, torch.full_like(col, free.shape[0]))
    grown = torch.cat([free, free[:1]])
    grown[at.flatten()] = table.flatten()
    free.copy_(grown[:-1])
    st["kv"].copy_(torch.where(done, torch.zeros_like(old), old))
    st["count_out"].copy_(count + n.sum())
    return free, st["kv"], st["count_out"]


def _plain_cache(st):
    page = st["k_pages"].shape[2]
    at, slot = st["slots"] // page, st["slots"] % page
    out = []
    for n in ("k", "v"):
        codes, scales = _quantise(st[n])
        st[n + "_pages"][at, :, slot] = codes
        st[n + "_scales"][at, :, slot] = scales
        out.append(_values(st[n + "_pages"][at, :, slot], st[n + "_scales"][at, :, slot]).to(st[n].dtype))
    return tuple(out)


def _plain_attention(st):
    q, page, hkv = st["q"], st["page"], st["hkv"]
    out = torch.empty_like(q)
    group, dim = q.shape[1] // hkv, q.shape[2]
    t0 = 0
    for s, (n, m) in enumerate(zip(st["new"], st["kv_host"])):
        w = st["win_host"][s] if st["win_host"] is not None else 0
        rows = st["table"][s, :_pages(m, page)].long()
        k, v = (_values(st[x + "_pages"][rows], st[x + "_scales"][rows]).transpose(0, 1).reshape(hkv, -1, dim)[:, :m]
                for x in ("k", "v"))
        step = max(1, (1 << 28) // (m * group * hkv))
        j = torch.arange(m, device=_DEV)
        for i0 in range(0, n, step):
            c = min(step, n - i0)
            x = q[t0 + i0:t0 + i0 + c].float().view(c, hkv, group, dim).permute(1, 0, 2, 3).reshape(hkv, c * group, dim)
            a = torch.matmul(x, k.transpose(1, 2)).mul_(st["scale"])
            pos = m - n + i0 + torch.arange(c, device=_DEV)
            hidden = j[None] > pos[:, None]
            if w > 0:
                hidden |= pos[:, None] - j[None] >= w
            a.masked_fill_(hidden.repeat_interleave(group, 0)[None], float("-inf"))
            a = a.sub_(a.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(a, v) / a.sum(-1, keepdim=True)
            out[t0 + i0:t0 + i0 + c] = o.view(hkv, c, group, dim).permute(1, 0, 2, 3).reshape(c, -1, dim).to(out.dtype)
        t0 += n
    return out


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "tables":
        return _exact_release(st) if case["release"] else _exact_tables(st)
    if case["op"] == "cache":
        return tuple(_exact_held(st[n].double()) for n in ("k", "v"))
    if work(case)["flops"] > 8e12:
        return None
    return _exact_attention(case, st)


def _exact_tables(st):
    p = st["page"]
    new, old = st["new"].tolist(), st["kv_prev"].tolist()
    table, free = st["table"].cpu().numpy().astype(np.int64), st["free"].tolist()
    stack = free[:int(st["count"])]
    cu, slots = [0], []
    for s, (n, o) in enumerate(zip(new, old)):
        for j in range(_pages(o, p), _pages(o + n, p)):
            table[s, j] = stack.pop()
        pos = np.arange(o, o + n)
        slots.append(table[s, pos // p] * p + pos % p)
        cu.append(cu[-1] + n)
    slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
    slots = np.concatenate([slots, np.full(st["slots"].shape[0] - len(slots), -1, np.int64)])
    to = lambda a, dt: torch.as_tensor(np.asarray(a), device=_DEV).to(dt)
    return (to(table, torch.int32), to(cu, torch.int32), to([n + o for n, o in zip(new, old)], torch.int32),
            to(slots, torch.int64), to([len(stack)], torch.int32))


def _exact_release(st):
    p, table = st["page"], st["table"].cpu().numpy()
    free, count = st["free"].cpu().numpy().copy(), int(st["count"])
    kv = st["kv_prev"].cpu().numpy().copy()
    for s, d in enumerate(st["done"].tolist()):
        if d:
            n = _pages(int(kv[s]), p)
            free[count:count + n] = table[s, :n]
            count += n
            kv[s] = 0
    return (torch.as_tensor(free, device=_DEV), torch.as_tensor(kv, device=_DEV), _ints([count]))


def _exact_held(x):
    """What the cache holds of rows x (float64): the nearest value of the format, found by search."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    grid = [m * 2.0 ** -17 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 15) for e in range(1, 31) for m in range(8)]
    grid = torch.tensor([g for g in grid if g <= 10240.0], dtype=torch.float64, device=x.device)

    def nearest(v, points):
        # The lower neighbour and the one above; an exact middle goes to the even position.
        lo = (torch.searchsorted(points, v.contiguous(), right=True) - 1).clamp(0, len(points) - 2)
        below, above = v - points[lo], points[lo + 1] - v
        up = (above < below) | ((above == below) & (lo % 2 == 1))
        return points[lo + up.long()]

    flat = x.reshape(-1, 16)
    out = torch.empty_like(flat)
    for i in range(0, flat.shape[0], 1 << 20):
        b = flat[i:i + (1 << 20)]
        s = nearest((b.abs().amax(1) / 6).clamp(max=10240.0), grid)[:, None]
        a = torch.where(s > 0, b.abs() / s.clamp(min=1e-30), torch.zeros_like(b)).clamp(max=6.0)
        out[i:i + (1 << 20)] = torch.where(torch.isfinite(b).all(1, keepdim=True), nearest(a, lut) * s * torch.sign(b),
                                           torch.full_like(b, math.nan))
    return out.view_as(x)


def _exact_read(packed, scales):
    p, b = packed.long(), scales.double()
    c = torch.stack([p % 16, torch.div(p, 16, rounding_mode="floor")], -1).flatten(-2)
    e, m = torch.div(c % 8, 2, rounding_mode="floor"), (c % 2).double()
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.pow(2.0, (e - 1).double()))
    se, sm = torch.div(b, 8, rounding_mode="floor"), b % 8
    s = torch.where(se == 0, sm * 2.0 ** -17, (1 + sm / 8) * torch.pow(2.0, se - 15))
    return mag * torch.where(c >= 8, -1.0, 1.0) * s.repeat_interleave(16, -1)


def _exact_attention(case, st):
    q, page, hkv, group = st["q"].double(), case["page"], case["hkv"], case["hq"] // case["hkv"]
    out = torch.empty_like(q)
    t0 = 0
    for s, (n, m) in enumerate(zip(st["new"], st["kv_host"])):
        w = st["win_host"][s] if st["win_host"] is not None else 0
        rows = st["table"][s, :_pages(m, page)].long()
        for g in range(hkv):
            k, v = (_exact_read(st[x + "_pages"][rows, g].flatten(0, 1)[:m], st[x + "_scales"][rows, g].flatten(0, 1)[:m])
                    for x in ("k", "v"))
            step = max(1, (1 << 27) // (m * group))
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                x = q[t0 + i0:t0 + i1, g * group:(g + 1) * group].reshape(-1, case["dim"])
                a = (x @ k.T) * st["scale"]
                back = (m - n + torch.arange(i0, i1, device=_DEV))[:, None] - torch.arange(m, device=_DEV)[None]
                seen = back >= 0 if w <= 0 else (back >= 0) & (back < w)
                a = torch.where(seen.repeat_interleave(group, 0), a, torch.full_like(a, -math.inf))
                a = torch.softmax(a, -1)
                out[t0 + i0:t0 + i1, g * group:(g + 1) * group] = (a @ v).view(i1 - i0, group, -1)
        t0 += n
    return out
