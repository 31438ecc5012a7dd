"""Drafted trees by their definitions, in 64 bits (numpy and torch on the CPU), and
batches of them for the tests.  Imports nothing from the library."""

from __future__ import annotations

import math
from types import SimpleNamespace

import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


def random_parents(n, rng):
    """A chain, a star, equal branches, or grown at random (several roots too)."""
    kind = int(rng.integers(5))
    if kind == 0:
        return [i - 1 for i in range(n)]
    if kind == 1:
        return [min(0, i - 1) for i in range(n)]
    if kind == 2:
        return [-1] + [(i - 1) // 3 for i in range(1, n)]
    return [int(rng.integers(-1, i)) if i else -1 for i in range(n)]


def tree_of(parents, window=0):
    """sees [n, n] (bool) and depths of one request's nodes."""
    n = len(parents)
    sees, depth = np.zeros((n, n), bool), np.zeros(n, int)
    for i, p in enumerate(parents):
        depth[i] = 0 if p < 0 else depth[p] + 1
        j = i
        while j >= 0:
            sees[i, j] = window <= 0 or depth[i] - depth[j] < window
            j = parents[j]
    return sees, depth


def mask_words(sees, words):
    """[n, words] uint64 of [n, m] bool."""
    n, m = sees.shape
    bits = np.zeros((n, 64 * words), np.uint8)
    bits[:, :m] = sees
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint64)


def to_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16()


def tree_batch(nodes, ctx, hq, hkv, d, page, windows=None, seed=0, words=None, sees=None, dtype="bf16", scale=None,
               spare=2):
    """A batch of drafted trees over a paged cache.  `sees`: [T, T] bools a request (else random trees)."""
    rng = np.random.default_rng(seed)
    s = len(nodes)
    kv = [c + t for c, t in zip(ctx, nodes)]
    cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    total = int(cu[-1])
    words = words or max(1, ceil_div(max(nodes), 64))
    held = [ceil_div(k, page) for k in kv]
    pool = sum(held) + spare
    perm = rng.permutation(pool)
    width = max(1, max(held))
    table = np.full((s, width), -1, np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[at:at + h]
        at += h
    win = [0] * s if windows is None else windows
    mask, pos, rows = np.zeros((total, words), np.uint64), np.zeros(total, np.int32), []
    for i, t in enumerate(nodes):
        r, depth = tree_of(random_parents(t, rng), win[i]) if t else (np.zeros((0, 0), bool), [])
        if sees is not None:
            r = sees[i]
        rows.append(r)
        mask[cu[i]:cu[i + 1]] = mask_words(r, words) if t else 0
        pos[cu[i]:cu[i + 1]] = ctx[i] + np.asarray(depth, int)
    conv = to_bf16 if dtype == "bf16" else (lambda x: torch.from_numpy(np.ascontiguousarray(x, np.float32)))
    b = SimpleNamespace(nodes=list(nodes), ctx=list(ctx), hq=hq, hkv=hkv, d=d, page=page, windows=windows, words=words,
                        cu=cu, kv=np.array(kv, np.int32), table=table, pool=pool, mask=mask, pos=pos, sees=rows,
                        win=None if windows is None else np.array(windows, np.int32), dtype=dtype,
                        scale=d ** -0.5 if scale is None else scale)
    b.q = conv(rng.standard_normal((total, hq, d)))
    k = rng.standard_normal((pool, page, hkv, d))
    k[..., ::29] *= 4
    b.k_pages, b.v_pages = conv(k), conv(rng.standard_normal((pool, page, hkv, d)))
    return b


def slot(b, s, key):
    return int(b.table[s, key // b.page]), key % b.page


def rows_of(b, s, pages):
    """[keys, hkv, d] float64 of a request's cache."""
    key = np.arange(b.kv[s])
    return pages[torch.from_numpy(b.table[s, key // b.page].astype(np.int64)), torch.from_numpy(key % b.page)].double()


def visible(b, s):
    """[T, keys] bool."""
    t, c = b.nodes[s], b.ctx[s]
    seen = np.zeros((t, c + t), bool)
    seen[:, :c] = True
    w = 0 if b.windows is None else b.windows[s]
    if w > 0:
        seen[:, :c] = b.pos[b.cu[s]:b.cu[s + 1], None] - np.arange(c)[None] < w
    seen[:, c:] = b.sees[s]
    return seen


def attention(b):
    """Output [total, hq, d] in 64 bits; the same with |v| for v (what roundings of the weights scale with); the
    largest scale * sum |q k| of each row, and its keys."""
    group = b.hq // b.hkv
    out, mag, smax = torch.zeros(b.q.shape, dtype=torch.float64), torch.zeros(b.q.shape, dtype=torch.float64), torch.zeros(b.q.shape[:2], dtype=torch.float64)
    for s, t in enumerate(b.nodes):
        if t == 0:
            continue
        k, v = rows_of(b, s, b.k_pages), rows_of(b, s, b.v_pages)
        seen = torch.from_numpy(visible(b, s))
        for g in range(b.hkv):
            at = (slice(int(b.cu[s]), int(b.cu[s + 1])), slice(g * group, (g + 1) * group))
            q = b.q[at].double()
            a = torch.einsum("tgd,kd->tgk", q, k[:, g]) * b.scale
            a = torch.where(seen[:, None], a, -math.inf)
            m = a.amax(-1, keepdim=True)
            p = torch.where(seen[:, None], torch.exp(a - torch.where(m == -math.inf, 0.0, m)), 0.0)
            n = p.sum(-1, keepdim=True)
            p = torch.where(n == 0, 0.0, p / n)
            # (A key that a row does not see takes no part, whatever its row holds.)
            out[at] = weigh(p, v[:, g], seen)
            mag[at] = weigh(p, v[:, g].abs(), seen)
            smax[at] = abs(b.scale) * (q.abs().amax(-1) * 0 + torch.einsum("tgd,d->tg", q.abs(), torch.nan_to_num(k[:, g], 0, 0, 0).abs().amax(0)))
    return out, mag, smax


def weigh(p, v, seen):
    bad = ~torch.isfinite(v)
    o = torch.einsum("tgk,kd->tgd", p, torch.where(bad, 0.0, v))
    for key in bad.any(-1).nonzero().flatten().tolist():
        sees = seen[:, key]
        o[sees] = o[sees] + torch.where(bad[key], v[key], 0.0)
    return o


def attention_bound(b, ref):
    """How far a kernel may be from `ref` (attention()): the output rounded to b's dtype; the weights rounded to bf16
    (2^-8 of each) where the products run on tensor cores; 32-bit sums of d and of n terms; 2^x to 2^-21."""
    out, mag, smax = ref
    n = max(int(k) for k in b.kv)
    half = 2.0 ** -8 if b.dtype == "bf16" else 2.0 ** -24
    weight = half if b.dtype == "bf16" else 0.0
    e = 2 * (b.d + 4) * 2.0 ** -24 * smax[..., None]
    return half * out.abs() + mag * (weight * 1.01 + (2 * torch.expm1(e)) + (n + 16) * 2.0 ** -24 + 2.0 ** -20)


def turned(x, pos, freq, pairs):
    """Rows x [t, heads, d] (float64) turned by pos * freq."""
    half = len(freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None]
    c, s = torch.from_numpy(np.cos(a))[:, None], torch.from_numpy(np.sin(a))[:, None]
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y
