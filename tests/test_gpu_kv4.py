"""The 4-bit KV cache on the GPU: write and read against the format's
definition, byte for byte, and attention over 4-bit pages against the float64
oracle on the values the pages stand for.

Bound on an attention output, from the arithmetic (eps / 2 is half a step
relative to the value): the output's rounding to bf16 (2^-8 |ref|); the
probabilities' rounding for the second product (f16 2^-11 on the split-KV
kernel, bf16 2^-8 on prefill) times A = sum_j p_j |v_j|; and the scores' fp32
error ds, which moves each p_j by 2 ds at most (numerator and denominator):
2 ds A, with ds = (D + 2) 2^-23 sm_scale |q| |k| (D products and their sums, a
step each) plus 2^-22 twice for the exponential and the logit scale's
rounding over scores below 2^5: together below 2^-16 A more.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from ragged_paged_attention_rpa_gb300 import binding, build, workloads

from .test_gpu_parity import unseen_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(shape, seed, bf16=True):
    """Rows of all magnitudes: normal times powers of two, zeros and exact ties
    among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 6, shape[:-1] + (1,)))
    x[rng.random(shape) < 0.05] = 0.0
    flat = x.reshape(-1, 16)
    n = max(1, len(flat) // 8)
    flat[:n] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.75, -5.0], (n, 16))
    flat[:n, 0] = 6.0
    x = torch.from_numpy(x.astype(np.float32))
    return x.to(torch.bfloat16) if bf16 else x


def pools(n, hkv, p, d, fill=0):
    one = lambda last: torch.full((n, hkv, p, last), fill, dtype=torch.uint8, device="cuda")
    return [one(d // 2), one(d // 2), one(d // 16), one(d // 16)]


SHAPES = [
    # (tokens, Hkv, D, P, pool pages)
    (1, 1, 64, 16, 1), (5, 3, 64, 32, 3), (37, 2, 128, 16, 5), (300, 8, 128, 64, 9),
    (130, 1, 256, 128, 4), (64, 4, 256, 256, 2), (2000, 2, 64, 16, 200),
]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_and_read(shape, bf16):
    """Codes and scales equal the definition's; slots of no token, and read
    rows of padding, stay as they were; values read back are the stored ones."""
    t, hkv, d, p, n = SHAPES[shape]
    rng = np.random.default_rng(shape)
    slots = rng.permutation(n * p)[:t].astype(np.int64)
    pad = rng.random(t) < 0.1
    slots[pad] = -1
    k, v = rows((t, hkv, d), 2 * shape, bf16), rows((t, hkv, d), 2 * shape + 1, bf16)
    pool = pools(n, hkv, p, d, fill=0xA5)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.rpa_write_kv4(k.cuda(), v.cuda(), *pool, cuda(slots), ws)
    for x, codes, scales in ((k, pool[0], pool[2]), (v, pool[1], pool[3])):
        want_c = np.full((n, hkv, p, d // 2), 0xA5, np.uint8)
        want_s = np.full((n, hkv, p, d // 16), 0xA5, np.uint8)
        c, s = workloads.kv4_encode(x.float().numpy())
        live = slots >= 0
        want_c[slots[live] // p, :, slots[live] % p] = c[live]
        want_s[slots[live] // p, :, slots[live] % p] = s[live]
        assert np.array_equal(scales.cpu().numpy(), want_s)
        assert np.array_equal(codes.cpu().numpy(), want_c)
    for dt in (torch.bfloat16, torch.float32):
        ko = torch.full((t, hkv, d), 7.0, dtype=dt, device="cuda")
        vo = ko.clone()
        binding.rpa_read_kv4(*pool, cuda(slots), ko, vo, ws)
        for x, got in ((k, ko), (v, vo)):
            want = oracle.decode_kv4(*workloads.kv4_encode(x.float().numpy()))
            want[slots < 0] = 7.0
            assert np.array_equal(got.float().cpu().numpy(), want)
    assert binding.rpa_get_device_error(ws) == 0


def test_write_of_extreme_values():
    """NaN and infinities (their whole block reads as NaN), the largest and the
    smallest magnitudes, subnormal scales, and float32 values next to ties."""
    x = np.ones((1, 1, 256), np.float32)
    x[0, 0, 3] = np.nan
    x[0, 0, 20] = np.inf
    x[0, 0, 40] = -np.inf
    x[0, 0, 48:64] = 3e38
    x[0, 0, 64:80] = np.exp2(np.arange(16) - 20.0)
    x[0, 0, 80:96] = 1e-40
    x[0, 0, 96:112] = np.nextafter(np.float32([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6] * 2), np.float32(9))
    x[0, 0, 112:128] = np.nextafter(np.float32([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6] * 2), np.float32(0))
    x[0, 0, 127] = 6
    # Scales next to the midpoints of two of theirs.
    for i, m in enumerate(np.float32([6.375, 6.375 * 2 ** 9, 6 * 2.5 * 2 ** -17, 6 * 1.5 * 2 ** -17])):
        x[0, 0, 128 + 32 * i:144 + 32 * i] = np.nextafter(m, np.float32(1e9))
        x[0, 0, 144 + 32 * i:160 + 32 * i] = np.nextafter(m, np.float32(0))
    pool = pools(1, 1, 16, 256)
    binding.rpa_write_kv4(cuda(x), cuda(-x), *pool, cuda(np.array([5], np.int64)))
    for y, codes, scales in ((x, pool[0], pool[2]), (-x, pool[1], pool[3])):
        c, s = workloads.kv4_encode(y)
        assert np.array_equal(scales[0, 0, 5].cpu().numpy(), s[0, 0])
        assert np.array_equal(codes[0, 0, 5].cpu().numpy(), c[0, 0])


def test_slots_outside_the_pool_set_the_error_word():
    pool = pools(2, 1, 16, 64)
    x = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    slots = cuda(np.array([3, 32, 1 << 40], np.int64))
    binding.rpa_write_kv4(x, x, *pool, slots, ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    assert int((pool[0] != 0).sum()) == 32 and int((pool[0][0, 0, 3] != 0).sum()) == 32
    out = torch.zeros_like(x)
    binding.rpa_read_kv4(*pool, slots, out, out.clone(), ws)
    assert binding.rpa_get_device_error(ws) == binding.RPA_DEVERR_PAGE_ID
    # Ones: 1 / 6 lies between the scales 10 / 64 and 11 / 64, nearer the upper;
    # 64 / 11 > 5, so the code is 6: 66 / 64.
    assert bool((out[0] == 66 / 64).all()) and bool((out[1:] == 0).all())


def test_rows_on_16_byte_boundaries():
    """Rows that start 16 but not 32 bytes into a line, written and read."""
    t, hkv, d, p = 9, 3, 64, 16
    for bf16 in (True, False):
        k, v = rows((t, hkv, d), 31, bf16), rows((t, hkv, d), 32, bf16)
        skip = 8 if bf16 else 4
        def off(x):
            flat = torch.zeros(x.numel() + skip, dtype=x.dtype, device="cuda")
            y = flat[skip:].view(x.shape)
            y.copy_(x)
            assert y.data_ptr() % 32 == 16
            return y
        pool = pools(2, hkv, p, d)
        slots = cuda(np.arange(t, dtype=np.int64) * 3)
        binding.rpa_write_kv4(off(k), off(v), *pool, slots)
        ko, vo = off(torch.zeros_like(k)), off(torch.zeros_like(v))
        binding.rpa_read_kv4(*pool, slots, ko, vo)
        for x, y in ((k, ko), (v, vo)):
            want = oracle.decode_kv4(*workloads.kv4_encode(x.float().numpy()))
            assert np.array_equal(y.float().cpu().numpy(), want)


def test_a_pool_beyond_four_gigabytes():
    """Slots whose byte offsets pass 2^32 (codes) and 2^31 (scales): written,
    read back and attended, by the split-KV kernel and through the prefill."""
    hkv, d, p, n = 2, 256, 256, 70000                 # 4.6 GB of codes each, 0.6 GB of scales
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    pool = [torch.empty((n, hkv, p, last), dtype=torch.uint8, device="cuda") for last in (128, 128, 16, 16)]
    t = 300
    k, v, q = (torch.from_numpy(np.random.default_rng(i).standard_normal((t, h, d)).astype(np.float32)).to(torch.bfloat16)
               for i, h in ((1, hkv), (2, hkv), (3, 4)))
    table = np.array([[n - 1, n - 3]], np.int32)
    pos = np.arange(t)
    slots = cuda(table[0, pos // p].astype(np.int64) * p + pos % p)
    binding.rpa_write_kv4(k.cuda(), v.cuda(), *pool, slots)
    ko, vo = torch.empty_like(k, device="cuda"), torch.empty_like(v, device="cuda")
    binding.rpa_read_kv4(*pool, slots, ko, vo)
    held = [oracle.decode_kv4(*workloads.kv4_encode(x.float().numpy())).astype(np.float64) for x in (k, v)]
    assert np.array_equal(ko.float().cpu().numpy(), held[0]) and np.array_equal(vo.float().cpu().numpy(), held[1])
    for new in (1, t):
        cu = np.array([0, new], np.int32)
        plan = binding.rpa_plan(cu, np.array([t], np.int32), None, 4, hkv, d, p, 2, n, kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
        ws = binding.alloc_workspace(plan)
        out = torch.empty((new, 4, d), dtype=torch.bfloat16, device="cuda")
        binding.rpa_forward_kv4(q[t - new:].cuda(), *pool, cuda(table), cuda(cu), cuda(np.array([t], np.int32)), None,
                                d ** -0.5, out, plan, ws)
        assert binding.rpa_get_device_error(ws) == 0
        got = out.float().cpu().numpy()
        for i in range(0, new, 37):
            m = t - new + i + 1
            for h in range(4):
                x = held[0][:m, h // 2] @ q[t - new + i, h].double().numpy() * d ** -0.5
                w = np.exp(x - x.max())
                w /= w.sum()
                ref, mag = w @ held[1][:m, h // 2], w @ np.abs(held[1][:m, h // 2])
                assert (np.abs(got[i, h] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7.9 * mag).all()


def test_refusals_of_the_binding():
    pool = pools(4, 2, 16, 64)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = cuda(np.arange(3, dtype=np.int64))
    write = binding.rpa_write_kv4
    with pytest.raises(TypeError):
        write(k.half(), k.half(), *pool, slots)
    with pytest.raises(TypeError):
        write(k, k.float(), *pool, slots)
    with pytest.raises(TypeError):
        write(k, k, *pool, slots.int())
    with pytest.raises(TypeError):
        write(k.cpu(), k, *pool, slots)
    with pytest.raises(TypeError):
        write(k, k, pool[0].char(), *pool[1:], slots)
    with pytest.raises(ValueError):
        write(k[:2], k, *pool, slots)
    with pytest.raises(ValueError):
        write(k, k, pool[0], pool[1][:3], *pool[2:], slots)
    with pytest.raises(ValueError):
        write(k, k, *pool[:2], pool[2][..., :2], pool[3], slots)
    with pytest.raises(ValueError):
        write(k.transpose(0, 1).contiguous().transpose(0, 1), k, *pool, slots)
    with pytest.raises(ValueError):
        write(k, k, *pool, slots, torch.zeros(64, dtype=torch.uint8, device="cuda"))
    b = batch([1], [40], 4, 2, 64, 16, seed=3)
    r = Kv4Batch(b)
    with pytest.raises(TypeError):
        r.ws = None
        r.call()
    r = Kv4Batch(b)
    r.pool = pools(4, 1, 16, 64)
    with pytest.raises(ValueError):
        r.call()
    r = Kv4Batch(b)
    args = (r.db.page_table, r.db.cu_q_lens, r.db.kv_lens, None, b.sm_scale)
    with pytest.raises(ValueError):     # a pool of fewer pages than the plan's
        binding.rpa_forward_kv4(r.db.q, *pools(1, 2, 16, 64), *args, r.out, r.plan, r.ws)
    with pytest.raises(ValueError):     # too few rows of q, of out, of the table
        binding.rpa_forward_kv4(r.db.q[:0], *r.pool, *args, r.out, r.plan, r.ws)
    with pytest.raises(ValueError):
        binding.rpa_forward_kv4(r.db.q, *r.pool, *args, r.out[:, :2].contiguous(), r.plan, r.ws)
    with pytest.raises(ValueError):
        binding.rpa_forward_kv4(r.db.q, *r.pool, r.db.page_table[:, :1].contiguous(), *args[1:], r.out, r.plan, r.ws)


def test_trace_names_the_kernels():
    b = batch([1] * 4 + [200], [3000, 40, 50, 60, 300], 8, 2, 128, 16, seed=4)
    r = Kv4Batch(b, decode_sms=-1)
    binding.rpa_trace_begin(16)
    r.call()
    names = [n for n, _ in binding.rpa_trace_end()]
    assert names == ["kv4_decode", "kv4_combine", "kv4_expand", "prefill_tc"]


# ---------------------------------------------------------------- attention

def batch(ql, kv, hq, hkv, d, p, win=None, seed=0, **kw):
    return workloads.with_kv4(workloads.make_batch(ql, kv, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                                   page_size=p, windows=win, seed=seed, **kw))


class Kv4Batch:
    def __init__(self, b, **plan_kw):
        self.b = b
        self.db = binding.Batch(b)
        self.pool = [cuda(x) for x in (b.k_fp4, b.v_fp4, b.k_fp4_scale, b.v_fp4_scale)]
        self.plan = binding.rpa_plan(b.cu_q_lens, b.kv_lens, b.window, b.num_q_heads, b.num_kv_heads,
                                     b.head_dim, b.page_size, b.max_pages_per_seq, b.num_pages,
                                     kv_dtype=binding.RPA_DTYPE_FP4_E2M1, **plan_kw)
        self.ws = binding.alloc_workspace(self.plan)
        self.out = torch.full_like(self.db.q, float("nan"))

    def call(self, page_table=None, out=None, ws=None, stream=None):
        db = self.db
        binding.rpa_forward_kv4(db.q, *self.pool, db.page_table if page_table is None else page_table,
                                db.cu_q_lens, db.kv_lens, db.window, self.b.sm_scale,
                                self.out if out is None else out, self.plan,
                                self.ws if ws is None else ws, stream)
        return self.out if out is None else out


def reference(b):
    """Float64 outputs, sum_j p_j |v_j|, and the bound's score error, [rows, D]."""
    k, v = oracle.kv4_pool(b.k_fp4, b.k_fp4_scale), oracle.kv4_pool(b.v_fp4, b.v_fp4_scale)
    q = oracle.bf16_bits_to_f32(b.q)
    meta = (b.page_table, b.cu_q_lens, b.kv_lens, b.window, b.sm_scale)
    ref = oracle.attention(q, k, v, *meta, precision=64)
    mag = oracle.attention(q, k, np.abs(v), *meta, precision=64)
    seen = ~unseen_slots(b)
    kmax = np.sqrt((k[seen].astype(np.float64) ** 2).sum(-1).max())
    qn = np.sqrt((q.reshape(-1, b.head_dim).astype(np.float64) ** 2).sum(-1))[:, None]
    return ref, mag, (b.head_dim + 2) * 2.0 ** -23 * b.sm_scale * qn * kmax


def check(b, got, prefill=True, ref=None):
    ref, mag, ds = reference(b) if ref is None else ref
    got = got.float().cpu().numpy().reshape(-1, b.head_dim).astype(np.float64)
    bound = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -8 if prefill else 2.0 ** -11) + 2 * ds + 2.0 ** -16) * mag
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / np.maximum(bound, 1e-30)).max()
    assert worst <= 1.0, "worst error %.3g of its bound" % worst


DECODE = [
    # (q_lens, kv_lens, Hq, Hkv, D, P, windows)
    ([1], [1], 1, 1, 64, 16, None),
    ([1] * 9, [1, 2, 15, 16, 17, 127, 128, 129, 700], 8, 1, 256, 128, None),
    ([1] * 7, [3, 64, 65, 200, 1000, 5, 40], 8, 2, 128, 32, [0, 16, 0, 100, 0, 2, 9]),
    ([1] * 4, [2000, 37, 513, 90], 4, 2, 128, 16, [1000, 0, 64, 1]),
    ([1] * 4, [129, 4097, 64, 1], 16, 2, 256, 64, None),
    ([1] * 5, [77, 1, 300, 513, 2049], 4, 4, 64, 16, [0, 0, 17, 0, 500]),        # G = 1
    ([1, 0, 1, 0], [77, 5, 300, 0], 6, 2, 64, 16, None),                         # G = 3, empty sequences
    ([1] * 3, [33, 300, 1700], 14, 2, 128, 64, None),                            # G = 7
    ([1] * 3, [33, 300, 1700], 32, 2, 128, 64, [0, 100, 0]),                     # G = 16
    ([1] * 2, [257, 900], 32, 1, 64, 16, None),                                  # G = 32
    ([1] * 2, [257, 900], 40, 1, 128, 16, None),                                 # G = 40
    ([1] * 2, [15000, 9000], 8, 8, 128, 256, None),                              # long, cut over CTAs
    ([1] * 200, [1 + 7 * i % 300 for i in range(200)], 8, 8, 64, 32, None),      # more tiles than one small launch
]
FEW = [
    ([8, 8, 3], [700, 8, 1000], 8, 1, 256, 128, None),
    ([2, 4, 1, 3], [9, 400, 33, 3], 8, 2, 128, 16, [0, 5, 0, 2]),
    ([5, 2, 7], [100, 2, 90], 4, 4, 64, 32, [0, 1, 33]),
    ([3, 3], [300, 1500], 6, 2, 128, 64, None),
    ([16, 1], [64, 64], 1, 1, 64, 16, [16, 0]),
]
PROMPTS = [
    ([100, 1, 37], [400, 50, 37], 8, 1, 256, 128, [64, 0, 1024]),
    ([300], [300], 4, 2, 64, 16, None),
    ([130, 65, 40], [130, 2000, 41], 2, 2, 128, 16, [0, 129, 1]),
    ([257, 8, 1, 1], [300, 900, 5, 1000], 16, 2, 128, 64, [100, 0, 0, 17]),
    ([64], [64], 128, 1, 64, 32, None),                                          # G = 128
    ([33, 0, 34], [33, 4, 500], 3, 3, 256, 256, None),
    ([133, 0, 134], [133, 4, 500], 3, 3, 256, 256, None),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_single_tokens(case):
    ql, kv, hq, hkv, d, p, win = DECODE[case]
    b = batch(ql, kv, hq, hkv, d, p, win, seed=300 + case)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=r.plan.info()["num_prefill_seqs"] > 0)


@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_tokens(case):
    ql, kv, hq, hkv, d, p, win = FEW[case]
    b = batch(ql, kv, hq, hkv, d, p, win, seed=340 + case)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out)


@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompts(case):
    ql, kv, hq, hkv, d, p, win = PROMPTS[case]
    b = batch(ql, kv, hq, hkv, d, p, win, seed=380 + case)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    # More than 128 rows of one sequence always go to the prefill.
    assert max(ql) * hq // hkv <= 128 or r.plan.info()["num_prefill_items"] > 0
    check(b, out)


def test_the_decode_workload():
    """128 requests of 128 to 2048 tokens, 8 heads on one of 256."""
    b = workloads.with_kv4(workloads.decode_batch(pool_pages=1400))
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=False)


@pytest.mark.parametrize("case", [(DECODE, 2), (DECODE, 3), (DECODE, 8), (FEW, 1), (FEW, 2), (PROMPTS, 0), (PROMPTS, 3)])
def test_unseen_slots_may_hold_anything(case):
    """NaN scales (and codes of ones) wherever no query looks: free slots of the
    last page, keys before a window, pages of no sequence."""
    ql, kv, hq, hkv, d, p, win = case[0][case[1]]
    b = batch(ql, kv, hq, hkv, d, p, win, seed=420 + case[1], pool_pages=sum(-(-x // p) for x in kv) + 2)
    mask = unseen_slots(b)
    assert mask.any()
    ref = reference(b)
    for name in ("k_fp4", "v_fp4", "k_fp4_scale", "v_fp4_scale"):
        x = getattr(b, name).copy()
        x.transpose(0, 2, 1, 3)[mask] = 0xFF
        setattr(b, name, x)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, ref=ref)


def test_a_nan_key_reaches_its_rows_only():
    """A stored NaN (a block of K, a block of V) makes NaN what sees it and
    nothing else: the other sequence and the other KV head stay finite."""
    b = batch([1, 1], [100, 100], 4, 2, 128, 16, seed=77)
    ref = reference(b)
    b.k_fp4_scale[b.page_table[0, 2], 1, 3, 0] = 255
    b.v_fp4_scale[b.page_table[1, 5], 0, 0, 7] = 255
    out = Kv4Batch(b).call().float().cpu().numpy()
    assert np.isnan(out[0, 2:]).all() and np.isfinite(out[0, :2]).all()
    assert np.isnan(out[1, :2, 112:]).all() and np.isfinite(out[1, :2, :112]).all() and np.isfinite(out[1, 2:]).all()
    want = ref[0].reshape(out.shape)
    ok = np.isfinite(out)
    assert np.abs(out[ok] - want[ok]).max() < 2e-2


def test_queries_of_all_sizes():
    """Rows of q from 2^-60 to 2^60 (sm_scale brings the logits back): the f16
    the products take them in holds each after its own power of two."""
    b = batch([1] * 6, [40, 50, 60, 300, 17, 5], 8, 2, 128, 16, seed=99)
    q = oracle.bf16_bits_to_f32(b.q)
    for e, s in ((60, 2.0 ** -60), (-60, 2.0 ** 60)):
        c = workloads.Batch(**{**b.__dict__, "q": oracle.round_bf16((q * 2.0 ** e).astype(np.float32)),
                               "sm_scale": b.sm_scale * s})
        check(c, Kv4Batch(c).call(), prefill=False)


@pytest.mark.parametrize("ql", [[1, 1], [40, 50]])
def test_bad_pages_and_lengths(ql):
    """A page id outside the pool sets the error word; its keys count as not
    seen (the oracle over the sequence without them agrees for one token)."""
    b = batch(ql, [200, 100], 8, 2, 128, 16, seed=55)
    r = Kv4Batch(b)
    for bad in (b.num_pages, -1, 1 << 30):
        table = b.page_table.copy()
        table[0, 3] = bad
        out = r.call(page_table=cuda(table))
        assert binding.rpa_get_device_error(r.ws) == binding.RPA_DEVERR_PAGE_ID
        assert bool(torch.isfinite(out).all())
    ok = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, ok)


@pytest.mark.parametrize("sms", [-1, 20])
def test_mixed_batches_side_by_side_and_after_another(sms):
    """The two parts on disjoint SMs or one after the other, and a workspace whose
    scratch holds NaN bytes: the same bound, and the same bits twice."""
    b = batch([1] * 30 + [300, 150], [40 + 97 * i % 1500 for i in range(30)] + [700, 151], 8, 2, 128, 16,
              [0, 200] * 16, seed=61)
    r = Kv4Batch(b, decode_sms=sms)
    assert r.plan.info()["decode_sms"] == max(0, sms)
    r.ws[256:] = 0xFF
    out = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out)
    assert torch.equal(r.call(), out)


def test_a_launch_holds_so_many_tiles():
    """More row tiles than one launch's parameters carry (864): several launches."""
    kv = [1 + 13 * i % 90 for i in range(1000)]
    b = batch([1] * 1000, kv, 4, 2, 64, 16, seed=62)
    r = Kv4Batch(b)
    out = r.call()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out, prefill=False)


def test_rows_behind_the_last_sequence_stay():
    b = batch([1, 4], [100, 40], 8, 1, 128, 16, seed=56)
    r = Kv4Batch(b)
    q = torch.cat([r.db.q, r.db.q])
    out = torch.full_like(q, 3.0)
    binding.rpa_forward_kv4(q, *r.pool, r.db.page_table, r.db.cu_q_lens, r.db.kv_lens, r.db.window,
                            b.sm_scale, out, r.plan, r.ws)
    assert bool((out[5:] == 3.0).all())
    check(b, out[:5])


def test_same_bits_every_time_on_streams_and_in_graphs():
    """Repeats, a side stream, a captured call replayed, and a workspace that
    another plan has used give the same bits."""
    mixed = batch([1] * 40 + [200, 6], [30 + 61 * i % 900 for i in range(40)] + [333, 700], 8, 2, 128, 32, seed=57)
    r = Kv4Batch(mixed)
    want = r.call().clone()
    assert torch.equal(r.call(), want)
    other = batch([1] * 3, [5000, 70, 900], 8, 2, 128, 32, seed=58)
    o = Kv4Batch(other)
    ws = torch.zeros(max(r.ws.numel(), o.ws.numel()), dtype=torch.uint8, device="cuda")
    a = o.call(ws=ws).clone()
    assert torch.equal(r.call(ws=ws), want) and torch.equal(o.call(ws=ws), a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = torch.full_like(want, float("nan"))
    r.call(out=side, stream=s)
    s.synchronize()
    assert torch.equal(side, want)
    g = torch.cuda.CUDAGraph()
    out = torch.full_like(want, float("nan"))
    with torch.cuda.graph(g):
        r.call(out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert binding.rpa_get_device_error(r.ws) == 0


def test_a_step_written_then_attended():
    """The step as it runs: tables from the lengths, the new rows written
    through the slot map, attention over the result, for three steps of one
    graph-captured table build and write; against the float64 oracle on what
    the cache holds of every row."""
    rng = np.random.default_rng(8)
    S, hq, hkv, d, p, width, pool_n = 5, 8, 2, 128, 16, 12, 64
    i32 = lambda a: cuda(np.asarray(a, np.int32))
    kv, table = i32([0] * S), i32(np.full((S, width), -1))
    free, count = i32(rng.permutation(pool_n)), i32([pool_n])
    ws0 = torch.zeros(256, dtype=torch.uint8, device="cuda")
    pool = pools(pool_n, hkv, p, d, fill=0xFF)
    held_k, held_v = ([np.zeros((0, hkv, d), np.float32) for _ in range(S)] for _ in range(2))
    lens = np.zeros(S, np.int64)
    for step, new in enumerate([[30, 1, 0, 64, 7], [1, 1, 5, 1, 1], [1, 1, 1, 1, 1], [1, 40, 1, 0, 3]]):
        new = np.array(new)
        t = int(new.sum())
        cu, slots = i32([0] * (S + 1)), cuda(np.full(t + 3, 7, np.int64))
        k, v = (torch.from_numpy(rng.standard_normal((t + 3, hkv, d)).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
        binding.rpa_build_tables(i32(new), kv, table, free, count, cu, kv, slots, count, p, ws0)
        binding.rpa_write_kv4(k.cuda(), v.cuda(), *pool, slots, ws0)
        lens += new
        starts = np.concatenate([[0], np.cumsum(new)])
        for s in range(S):
            for held, x in ((held_k, k), (held_v, v)):
                c = oracle.decode_kv4(*workloads.kv4_encode(x[starts[s]:starts[s + 1]].float().numpy()))
                held[s] = np.concatenate([held[s], c])
        assert cu.cpu().tolist() == starts.tolist() and kv.cpu().tolist() == lens.tolist()
        q = torch.from_numpy(rng.standard_normal((t, hq, d)).astype(np.float32)).to(torch.bfloat16)
        plan = binding.rpa_plan(starts.astype(np.int32), lens.astype(np.int32), None, hq, hkv, d, p, width, pool_n,
                                kv_dtype=binding.RPA_DTYPE_FP4_E2M1)
        ws = binding.alloc_workspace(plan)
        out = torch.full((t, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        binding.rpa_forward_kv4(q.cuda(), *pool, table, cu, kv, None, d ** -0.5, out, plan, ws)
        assert binding.rpa_get_device_error(ws) == 0 and binding.rpa_get_device_error(ws0) == 0
        got = out.float().cpu().numpy().astype(np.float64)
        for s in range(S):
            for i in range(new[s]):
                n = lens[s] - new[s] + i + 1
                for h in range(hq):
                    x = held_k[s][:n, h // 4].astype(np.float64) @ q[starts[s] + i, h].double().numpy() * d ** -0.5
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    val = held_v[s][:n, h // 4].astype(np.float64)
                    ref, mag = w @ val, w @ np.abs(val)
                    assert (np.abs(got[starts[s] + i, h] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7.9 * mag).all()


ROWS = [
    # (q_lens, kv_lens, Hq, Hkv, D, P, windows): 17 to 128 query rows a sequence
    ([8, 3, 5, 1], [700, 8, 33, 500], 8, 1, 256, 16, None),
    ([8, 8], [2047, 1300], 8, 1, 256, 256, [100, 0]),
    ([5, 13, 1], [65, 130, 3], 8, 2, 128, 16, [0, 7, 0]),
    ([16, 9], [4000, 3001], 4, 1, 128, 32, [0, 1000]),                           # cut over CTAs
    ([4, 6, 16], [127, 600, 1029], 8, 1, 64, 16, [0, 0, 50]),
    ([1, 1, 1], [900, 1, 128], 64, 1, 64, 32, [0, 0, 33]),                       # single tokens, G = 64
    ([1, 1], [513, 31], 128, 1, 256, 64, None),                                  # G = 128: two tiles
    ([2, 1], [300, 20], 57, 1, 128, 64, None),                                   # G = 57: 114 rows
    ([4, 8, 3], [8, 19, 33], 24, 3, 256, 16, None),                              # whole segments of three heads
    ([8, 8], [19, 40], 24, 3, 128, 32, [0, 3]),
]


@pytest.mark.parametrize("case", range(len(ROWS)))
def test_tens_of_rows(case):
    """Tiles of 64 rows: blocks widened once for all of them.  With NaN bytes in
    every unseen slot the bits are the same, and a bad page is reported and
    counts as unseen."""
    ql, kv, hq, hkv, d, p, win = ROWS[case]
    b = batch(ql, kv, hq, hkv, d, p, win, seed=700 + case)
    r = Kv4Batch(b)
    assert r.plan.info()["num_prefill_seqs"] == 0
    out = r.call().clone()
    assert binding.rpa_get_device_error(r.ws) == 0
    check(b, out)
    unseen = unseen_slots(b)
    for name in ("k_fp4_scale", "v_fp4_scale"):
        x = getattr(b, name).copy()
        x.transpose(0, 2, 1, 3)[unseen] = 255
        setattr(b, name, x)
    r2 = Kv4Batch(b)
    assert torch.equal(r2.call(), out)
    table = b.page_table.copy()
    table[0, 0] = b.num_pages
    bad = r2.call(page_table=cuda(table))
    seen = not (win and win[0] > 0 and kv[0] - ql[0] - (win[0] - 1) >= p)
    assert binding.rpa_get_device_error(r2.ws) == (binding.RPA_DEVERR_PAGE_ID if seen else 0)
    assert bool(torch.isfinite(bad).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [3, 7, 14])
def test_rows_that_see_their_first_key_in_different_blocks(d, tokens):
    """Small windows over many positions: the rows of a tile begin in different
    blocks, wherever a block's border lies."""
    kv = [tokens + 20 + 5 * i for i in range(24)] + [1312]
    b = batch([tokens] * 25, kv, 1, 1, d, 16, [17, 2, 5, 33, 9] * 5, seed=800 + tokens)
    for kw in ({}, {"num_sms": 1}):
        r = Kv4Batch(b, **kw)
        out = r.call()
        assert binding.rpa_get_device_error(r.ws) == 0
        check(b, out)


@pytest.mark.parametrize("d,tokens", [(64, 5), (64, 12), (128, 5), (128, 12), (128, 40), (256, 6), (256, 30)])
def test_a_nan_query_reaches_its_row_only(d, tokens):
    b = batch([tokens, tokens], [300, 90], 1, 1, d, 16, seed=900 + tokens)
    ref = reference(b)
    rows = [1, tokens + 2]
    b.q[rows, 0, 3] = 0x7FC0
    r = Kv4Batch(b)
    out = r.call().clone()
    assert r.plan.info()["num_prefill_seqs"] == 0
    assert bool(torch.isnan(out[rows]).all())
    keep = np.ones(2 * tokens, bool)
    keep[rows] = False
    got = out.float().cpu().numpy().reshape(-1, d).astype(np.float64)
    got[rows] = ref[0][rows]
    assert np.isfinite(got[keep]).all()
    check(b, torch.from_numpy(got), ref=ref)
