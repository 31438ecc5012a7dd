"""Rotation and cache write where their arithmetic could go wrong: angles of either sign, frequencies that are no
numbers, quotients beyond 32 bits.  The bounds are worked out pair by pair."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from ragged_paged_attention_rpa_gb300 import binding, build

from . import tree_reference as ref
from .test_gpu_tree_step import e4m3, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def turn(x, pos, freq, pairs, dt=torch.float32):
    """Rows x [t, heads, d] turned as q, and as k through fresh pages of the same type."""
    t, heads, d = x.shape
    x = x.to(dt).cuda()
    out = torch.empty_like(x)
    pages = torch.zeros((t, 1, heads, d), dtype=dt, device="cuda")
    freq = torch.as_tensor(np.asarray(freq, np.float32)).cuda()
    binding.rpa_append_rope(x, x, x, i32(pos), torch.arange(t, device="cuda"), freq, out, pages, pages.clone(),
                            interleaved=pairs)
    assert torch.equal(out.view(torch.uint8), pages[:, 0].view(torch.uint8))
    return out


def pair_sums(x, n, pairs):
    """|x| + |y| of each dimension's pair; zero where nothing turns."""
    i = torch.arange(n)
    first, second = (2 * i, 2 * i + 1) if pairs else (i, i + n)
    both = torch.zeros_like(x)
    both[..., first] = both[..., second] = x[..., first].abs() + x[..., second].abs()
    return both, first, second


def sine_error(pos, freq, first, second, d):
    """[t, 1, d]: the angle's error (2^-47 of itself + 2^-28), a sine's two roundings (one unit and half a unit in the
    last place, under 2^-23) and the products' (2^-24 of each, 2^-24 of their sum: under 2^-23 of |x| + |y|)."""
    a = np.abs(np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)[None])
    e = torch.zeros((len(pos), 1, d), dtype=torch.float64)
    e[..., first] = e[..., second] = torch.from_numpy(a * 2.0 ** -47 + 2.0 ** -28 + 2.0 ** -22)[:, None]
    return e


def near(got, x, pos, freq, pairs, half):
    x = x.double()
    both, first, second = pair_sums(x, len(freq), pairs)
    want = ref.turned(x, pos, freq, pairs)
    off = sine_error(pos, freq, first, second, x.shape[-1]) * both
    bound = off + half * (want.abs() + off)
    diff = (got.double().cpu() - want).abs()
    assert (diff <= bound).all(), "%g of the bound" % float((diff / bound.clamp(min=1e-300)).max())


POSITIONS = [0, 1, -1, 1001, 4095, 8191, 20001, 65537, 131071, 999999, -8191, -131071, 16777215, (1 << 31) - 1, -(1 << 31) + 1]


def frequencies(kind, n, rng):
    table = 10000.0 ** (-np.arange(n) / n)
    if kind == "negative":
        return -table
    if kind == "mixed":
        return table * np.where(np.arange(n) % 2, -1.0, 1.0)
    if kind == "listed":
        f = np.array([-1.0, -0.1, -1e-3, -1e-5, -1e-7, -2.0 ** -24, -2.0 ** -26, -0.3, -7.5, -100.0, -3.0, -6.2831855])
        return np.resize(np.concatenate([f, -f]), n)
    return rng.choice([-1.0, 1.0], n) * 2.0 ** rng.uniform(-40, 12, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["negative", "mixed", "listed", "random"])
def test_frequencies_of_either_sign(kind, pairs, dtype):
    rng = np.random.default_rng(5)
    dt, half = (torch.bfloat16, 2.0 ** -8) if dtype == "bf16" else (torch.float32, 2.0 ** -24)
    pos = np.array(POSITIONS + rng.integers(1000, 1000000, 50).tolist())
    freq = np.float32(frequencies(kind, 64, rng))
    x = torch.from_numpy(rng.standard_normal((len(pos), 3, 128))).to(dt)
    near(turn(x, pos, freq, pairs, dt), x, pos, freq, pairs, half)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("kind", ["negative", "mixed", "random"])
def test_turned_there_and_back(kind, pairs):
    """By f, then by -f.  The first turn's error of a pair is turned itself (2 of it at most), the second's goes with
    |x| + |y| after the first (sqrt 2 of it before)."""
    rng = np.random.default_rng(6)
    pos = np.array(POSITIONS + rng.integers(1000, 1000000, 50).tolist())
    freq = np.float32(frequencies(kind, 64, rng))
    x = torch.from_numpy(rng.standard_normal((len(pos), 2, 128))).float()
    back = turn(turn(x, pos, freq, pairs).cpu(), pos, -freq, pairs)
    both, first, second = pair_sums(x.double(), 64, pairs)
    bound = 3.5 * sine_error(pos, freq, first, second, 128) * both
    diff = (back.double().cpu() - x.double()).abs()
    assert (diff <= bound).all(), "%g of the bound" % float((diff / bound.clamp(min=1e-300)).max())


@pytest.mark.parametrize("pairs", [False, True])
def test_frequencies_that_are_no_numbers(pairs):
    """Their pairs come out NaN at any position, the others as they should."""
    rng = np.random.default_rng(7)
    pos = np.array([0, 1, -3, 5000, (1 << 31) - 1, -(1 << 31)])
    freq = np.float32(frequencies("mixed", 32, rng))
    bad = {0: np.nan, 5: np.inf, 17: -np.inf, 31: -np.nan}
    for i, f in bad.items():
        freq[i] = f
    x = torch.from_numpy(rng.standard_normal((len(pos), 2, 64))).float()
    got = turn(x, pos, freq, pairs).cpu()
    gone = torch.zeros(64, dtype=torch.bool)
    for i in bad:
        gone[[2 * i, 2 * i + 1] if pairs else [i, i + 32]] = True
    assert torch.isnan(got[..., gone]).all()
    fine = np.where(np.isfinite(freq), freq, 0)
    want = x.double()
    near(torch.where(gone, x, got).cuda(), want, pos, fine, pairs, 2.0 ** -24)


def nearest_e4m3(y):
    """The nearest e4m3 value (ties to even), 448 at most, NaN as NaN."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 1e6)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.frexp(a)[1] - 1, -6)
        v = np.minimum(np.rint(a / 2.0 ** (e - 3.0)) * 2.0 ** (e - 3.0), 448.0)
    return np.where(np.isnan(y), np.nan, np.copysign(v, y))


def stored(v, scale, dt):
    """Values of the e4m3 pages that rows v [t, heads, 64] leave (as v, and as k that is not turned)."""
    t, heads, d = v.shape
    v, scale = v.to(dt).cuda(), torch.as_tensor(np.asarray(scale, np.float32)).cuda()
    kp, vp = (torch.zeros((t, 1, heads, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    binding.rpa_append_rope(None, v, v, None, torch.arange(t, device="cuda"), None, None, kp, vp, k_scale=scale, v_scale=scale)
    assert torch.equal(kp, vp)
    return e4m3(vp[:, 0]).numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_e4m3_quotients_beyond_32_bits(dtype):
    """At most 448 where the quotient overflows; zeros stay zeros under scales whose reciprocal does; infinities, NaN."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    large = [1e37, -1e37, 3e38, -3e38, 1e30, 0.0, -0.0, float("inf"), -float("inf"), float("nan"), 2.0 ** -126, -2.0 ** -133]
    ratios = [0.0, 1.0, -1.0, 3.0, 17.0, -19.0, 448.0, 500.0, -1e5, 2.0 ** -3, 1.5, 208.0]
    scales = [0.01, 1e-30, 2.0 ** -64, 2.0 ** -65, 2.0 ** -126, 2.0 ** -127, 2.0 ** -128, 2.0 ** -130, 1.0, 1e30, 2.0 ** 126, 3e38]
    x = torch.zeros((2, len(scales), 64), dtype=torch.float64)
    x[0, :, :len(large)] = torch.tensor(large, dtype=torch.float64)
    for h, s in enumerate(scales):
        x[1, h, :len(ratios)] = torch.tensor(ratios, dtype=torch.float64) * s
    x = x.clamp(-3.3e38, 3.3e38).where(~torch.isinf(x), x).to(dt)
    s = np.float64(np.float32(scales))[None, :, None]
    with np.errstate(over="ignore"):
        y = x.double().numpy() / s
    got = stored(x, scales, dt)
    # (Ties are decided by the quotient's roundings, two of 2^-24.)
    low, high = nearest_e4m3(y * (1 - 2.0 ** -22 * np.sign(y))), nearest_e4m3(y * (1 + 2.0 ** -22 * np.sign(y)))
    nan = np.isnan(y)
    assert np.array_equal(np.isnan(got), nan)
    ok = nan | ((got >= low) & (got <= high))
    assert ok.all(), [(x[tuple(i)].item(), scales[i[1]], got[tuple(i)]) for i in np.argwhere(~ok)[:5]]
    # The listed ratios are exact, ties among them.
    exact = nearest_e4m3(np.array(ratios))
    for h in range(len(scales)):
        kept = x[1, h, :len(ratios)].double().numpy() == np.array(ratios) * s[0, h, 0]
        assert np.array_equal(got[1, h, :len(ratios)][kept], exact[kept]), scales[h]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_e4m3_quotients_of_any_size(dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(8)
    scales = np.float32(2.0 ** rng.uniform(-140, 127, 40))
    x = rng.choice([-1.0, 1.0], (30, 40, 64)) * scales[None, :, None].astype(np.float64) * 2.0 ** rng.uniform(-12, 11, (30, 40, 64))
    x[::3] = rng.choice([-1.0, 1.0], x[::3].shape) * 2.0 ** rng.uniform(-140, 127.9, x[::3].shape)
    x = torch.from_numpy(x.clip(-3.3e38, 3.3e38)).to(dt)
    y = x.double().numpy() / scales.astype(np.float64)[None, :, None]
    got = stored(x, scales, dt)
    low, high = nearest_e4m3(y * (1 - 2.0 ** -22 * np.sign(y))), nearest_e4m3(y * (1 + 2.0 ** -22 * np.sign(y)))
    ok = (got >= low) & (got <= high)
    assert ok.all(), [(x[tuple(i)].item(), scales[i[1]], got[tuple(i)]) for i in np.argwhere(~ok)[:5]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 256])
def test_rows_of_the_cache_turned_further_in_place(d, dtype):
    """Rows that are the slots they go to: the same bits as from a copy."""
    t, heads = 300, 3
    pages = [torch.randn((t // 4, 4, heads, d), device="cuda").to(dtype) for _ in range(2)]
    rows = [p.view(t, heads, d) for p in pages]
    pos, slots = i32(np.arange(t) * 37 - 5000), torch.arange(t, device="cuda")
    freq = torch.tensor(frequencies("mixed", d // 2, np.random.default_rng(9)), dtype=torch.float32, device="cuda")
    want = [p.clone() for p in pages]
    binding.rpa_append_rope(None, rows[0].clone(), rows[1].clone(), pos, slots, freq, None, *want)
    binding.rpa_append_rope(None, *rows, pos, slots, freq, None, *pages)
    for p, w in zip(pages, want):
        assert torch.equal(p.view(torch.uint8), w.view(torch.uint8))
