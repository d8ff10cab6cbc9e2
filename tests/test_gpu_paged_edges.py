"""GPU tests of the paged KV cache where its calls can go wrong without a fault: what an earlier kernel
leaves in shared memory, weights far below the largest, pages that were given away.

References and tolerances as in test_gpu_paged.py; what differs is derived beside each check.
"""
import numpy as np
import pytest
import torch

import fp8_quantization_amax_b200 as fq
import paged_reference as ref
from helpers import assert_codes_equal, dev, dev_bf16, host
from test_gpu_paged import Cache, append_case, attend, bf16

#: weights are rounded to f16 after a factor that makes a row's largest 2^LIFT at least
LIFT = 9

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available()
    assert fq.device_status() == 0
    yield
    assert fq.device_status() == 0


# ------------------------------------------------------------------ append

def nan_in_shared_memory():
    """A call that leaves the NaN word 0xFFFFFFFF in some 200 KB of every SM's shared memory: attention
    copies codes of 0xFF and scales of NaN through it, one block to an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    codes = torch.full((1, 16, 8, 128), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((8, 16), -1, dtype=torch.int32, device="cuda").view(torch.float32)
    table = torch.zeros((sms, 8), dtype=torch.int32, device="cuda")
    lens = torch.full((sms,), 128, dtype=torch.int32, device="cuda")
    q = dev_bf16(bf16(np.random.default_rng(0), sms, 8, 128))
    return lambda: fq.fp8_attention_paged(q, codes, codes, scales, scales, table, lens, 0, 3)


@pytest.mark.parametrize("d", [16, 32, 48, 80, 96, 112, 160, 192, 240])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_after_nan_in_shared_memory(d, interleaved, monkeypatch):
    """Norm and a scale per token, heads that do not fill a power of two: the places past head_dim count as zeros
    whatever an earlier kernel left behind."""
    before, append = nan_in_shared_memory(), fq.fp8_kv_append

    def after_nan(*a, **kw):
        before()
        return append(*a, **kw)
    monkeypatch.setattr(fq, "fp8_kv_append", after_nan)
    for rot in (0, d // 2 // 8 * 8, d):
        append_case(d + rot, 700, 3, 3, d, 24, 0, 3, rot, interleaved, True)


def test_append_given_scales_of_every_kind(orc):
    """All bf16 inputs by scales at the borders of the kernel's division (2^-68, 2^-60, 2^100, 2^119), tiny, huge,
    negative, infinite and NaN: FP8 of the fp32 quotient, and signed zeros for a scale of zero."""
    s = np.array([1.0, 0.3, -0.5, -3e-3, 0.0, -0.0, np.inf, -np.inf, np.nan, 1e-40, -1e-40, 1e-45, 3e38, -3e38, 2.0 ** -126,
                  2.0 ** -69, 2.0 ** -68, 2.0 ** -60, 2.0 ** 100, 2.0 ** 101, 2.0 ** 119, 2.0 ** 120], np.float32)
    H, D, T = len(s), 256, 256
    x = np.broadcast_to(np.arange(T * D).astype(np.uint16).reshape(T, 1, D), (T, H, D))
    xf = (x.astype(np.uint32) << 16).view(np.float32)
    with np.errstate(all="ignore"):
        q = np.where(s[None, :, None] == 0, np.copysign(np.float32(0), xf), xf / s[None, :, None]).astype(np.float32)
    for fmt in (0, 1):
        k = torch.zeros((T // 16, 16, H, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros_like(k)
        fq.fp8_kv_append(None, dev_bf16(x), dev_bf16(x), torch.arange(T, device="cuda"), k, v, dev(s), dev(s), fmt, 1)
        torch.cuda.synchronize()
        want = orc.encode(np.ascontiguousarray(q).reshape(-1), fmt).reshape(T, H, D)
        for h in range(H):
            assert_codes_equal(host(v).reshape(T, H, D)[:, h], want[:, h], fmt, f"scale {s[h]}")
        assert torch.equal(k, v)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("gran", [1, 3])
@pytest.mark.parametrize("below", [22.0, 24.0, 25.6, 27.0])
def test_attention_keeps_weights_far_below_the_largest(gran, below):
    """One token takes nearly all the weight and its V is zero, so the others are the whole result; each
    request is read by one warp a head.  A weight's error is 2^-11 of it, or 2^-25 where it is subnormal in f16,
    the row's largest being 2^LIFT at least (the tolerance's second line)."""
    rng = np.random.default_rng(int(below))
    B, H, G, D, size, n = torch.cuda.get_device_properties(0).multi_processor_count, 16, 2, 64, 16, 8192
    P = n // size
    k = rng.integers(0, 256, (n, H, D)).astype(np.uint8)
    k[(k & 0x7F) >= 0x78] ^= 0x40                             # moderate codes
    k[:, :, 0] = 0
    k[5] = 0
    k[5, :, 0] = 0x38                                         # 1.0
    v = rng.integers(0x30, 0x41, (n, H, D)).astype(np.uint8)  # 0.5 .. 2
    v[5] = 0
    shape = fq.kv_page_scale_shape(P, size, H, gran)
    ks = np.full(shape, below * np.log(2.0), np.float32)
    vs = np.ones(shape, np.float32)
    if gran == 3:
        vs = np.exp2(rng.uniform(-2, 2, shape)).astype(np.float32)
        vs[:, 5] = 1.0
    x = (rng.standard_normal((H * G, D)) * 2e-5).astype(np.float32)
    x[:, 0] = 1.0
    qb = (x.view(np.uint32) >> 16).astype(np.uint16)
    table = np.broadcast_to(np.arange(P, dtype=np.int32), (B, P))
    cache = [dev(c.reshape(P, size, H, D)) for c in (k, v)]
    out, lse = fq.fp8_attention_paged(dev_bf16(np.broadcast_to(qb, (B, H * G, D))), *cache, dev(ks), dev(vs), dev(table),
                                      dev(np.full(B, n, np.int32)), 0, gran, scale=1.0)
    torch.cuda.synchronize()
    val, q = ref.decode_table(0), ref.bf16_to_f64(qb)
    for h in range(H):
        slots = np.arange(n)
        kk = val[k[:, h]] * ref.token_scale(ks, gran, slots, h)[:, None]
        sv = ref.token_scale(vs, gran, slots, h)
        z = q[h * G:(h + 1) * G] @ kk.T
        dz = (np.abs(q[h * G:(h + 1) * G]) @ np.abs(kk.T) * (D + 8) * 2.0 ** -22 + np.abs(z) * 2.0 ** -21).max(1)[:, None]
        p = np.exp(z - z.max(1, keepdims=True))
        tot = p.sum(1, keepdims=True)
        want = p @ (val[v[:, h]] * sv[:, None]) / tot
        tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * dz + 2.0 ** -19) \
            + n * 2.0 ** -25 * 2.0 ** -LIFT * (p * sv).max(1, keepdims=True) / tot * 2.0
        assert (tol < 0.1 * want).all()                       # a lost tail shows
        for b in (0, 1, B - 1):
            got = ref.bf16_to_f64(host(out[b, h * G:(h + 1) * G]))
            assert (np.abs(got - want) <= tol).all(), (h, b, (np.abs(got - want) / want).max())
            got = host(lse[b, h * G:(h + 1) * G]).astype(np.float64)
            lw = np.log(tot[:, 0]) + z.max(1)
            assert (np.abs(got - lw) <= dz[:, 0] + 2.0 ** -20 * (1 + np.abs(lw))).all()


@pytest.mark.parametrize("gran", [2, 3])
def test_attention_scales_of_either_sign(gran):
    """Scales of tokens may be negative, as those of heads: their magnitude is what a weight is brought to."""
    rng = np.random.default_rng(gran)
    c = Cache(rng, [300, 0, 77], 2, 64, 16, 0, gran)
    for s, d in ((c.ks, c.dks), (c.vs, c.dvs)):
        s *= np.where(rng.random(s.shape) < 0.5, -1.0, 1.0).astype(np.float32)
        d.copy_(dev(s))
    qb = bf16(rng, 3, 8, 64)
    out, lse = c.run(dev_bf16(qb))
    torch.cuda.synchronize()
    c.check(qb, out, lse, 0.125)
    # all of them negative: minus the result of their magnitudes
    c.dvs.copy_(dev(-np.abs(c.vs)))
    neg, _ = c.run(dev_bf16(qb))
    c.dvs.copy_(dev(np.abs(c.vs)))
    pos, _ = c.run(dev_bf16(qb))
    torch.cuda.synchronize()
    assert torch.equal(neg[[0, 2]], -pos[[0, 2]])


@pytest.mark.parametrize("seed,lens,heads,group,d,size,fmt,gran,window,sinks,layout", [
    (251924, [9, 1, 9, 9, 1], 11, 9, 16, 5, 1, 3, 0, 0, "htd"),
    (238364, [1, 0, 5, 9, 9, 1], 33, 17, 16, 16, 0, 3, 0, 0, "thd"),
    (833896, [1, 0, 2, 2, 1, 0, 2, 1, 2, 2, 1], 11, 17, 16, 16, 1, 2, 4, 15, "thd"),
    (363082, [613, 1, 296, 289, 75, 613], 4, 24, 16, 128, 1, 2, 3, 16, "htd"),
    (967120, [1] * 24, 8, 16, 16, 128, 1, 3, 0, 0, "thd"),
    (7, [1] * 40, 16, 1, 48, 32, 1, 2, 0, 0, "htd"),
    (8, list(range(60)), 16, 3, 48, 16, 1, 3, 8, 17, "thd"),
])
def test_attention_lse_of_few_tokens(seed, lens, heads, group, d, size, fmt, gran, window, sinks, layout):
    """The sum of few weights near 1 is what their logarithm is taken of: factors for f16 do not enter it, and a
    sum far from 1 (V's scales of tokens are in the reference) meets the reference before the logarithm."""
    attend(seed, lens, heads, group, d, size, fmt, gran, window, sinks, layout)


@pytest.mark.parametrize("most", [511, 512, 513, 768, 769])
@pytest.mark.parametrize("heads,group,d", [(4, 4, 256), (8, 12, 128), (1, 16, 256), (2, 3, 160)])
def test_attention_wide_heads_spread(heads, group, d, most):
    """Blocks of 8 warps around the lengths up to which heads are spread and requests stay whole."""
    attend(most, [most, 3, most // 2], heads, group, d, 16, 0, 1, max_pages=-(-most // 16))
    attend(most + 1, [most], heads, group, d, 24, 1, 3, max_pages=-(-most // 24))


@pytest.mark.parametrize("heads,most", [(16, 64), (16, 128), (16, 129), (8, 256), (8, 257), (5, 384), (5, 400)])
@pytest.mark.parametrize("gran", [0, 3])
def test_attention_many_short_requests(heads, most, gran):
    """More requests than blocks, around the lengths up to which they stay whole."""
    rng = np.random.default_rng(most)
    lens = [int(n) for n in rng.integers(0, most + 1, 200)]
    lens[7] = most
    attend(heads, lens, heads, 1, 64, 16, 0, gran, max_pages=-(-most // 16))


# ------------------------------------------------------------------ pages

def update(table, lens, added, free, count, size, max_tokens):
    """One step on copies -> (slots, served, lens, list of free pages, table, whole list)."""
    t, f, c = dev(np.array(table, np.int32)), dev(np.array(free, np.int32)), dev(np.array([count], np.int32))
    slots, _, _, served, lens_out, _ = fq.fp8_kv_pages_update(t, dev(np.array(lens, np.int32)), dev(np.array(added, np.int32)),
                                                              f, c, size, max_tokens)
    torch.cuda.synchronize()
    n = int(host(c)[0])
    return host(slots), host(served).tolist(), host(lens_out).tolist(), host(f)[:n].tolist(), host(t)


@pytest.mark.parametrize("B", [4, 1300])
def test_pages_given_away_before_are_not_given_back(B):
    """Pages out of a window's sight were recycled early and are marked in the table: a request's end gives
    back the others, in order, and they alone count for the list's room."""
    table = np.full((B, 6), -1, np.int32)
    lens, added = np.zeros(B, np.int32), np.zeros(B, np.int32)
    table[0, :4], lens[0], added[0] = [-1, -1, 5, 6], 14, -1
    table[1, :2], lens[1] = [7, 0], 8
    table[B - 1, :6], lens[B - 1], added[B - 1] = [-1, 3, -2 ** 31, 4, -7, 2], 24, -1
    slots, served, n, free, _ = update(table, lens, added, [1, 8, 0, 0, 0, 0, 0], 2, 4, 0)
    assert free == [1, 8, 5, 6, 3, 4, 2] and n[0] == n[B - 1] == 0 and n[1] == 8
    assert fq.device_status() == 0
    # nothing but marked entries, and a list with no room left
    table[0, :4], table[B - 1, :6] = -1, -1
    *_, free, _ = update(table, lens, added, [1, 8], 2, 4, 0)
    assert free == [1, 8] and fq.device_status() == 0
    # more than the list holds, behind marked entries: the first ones fill it, the rest is reported
    table[B - 1, :6] = [-1, 3, -1, 4, -1, 2]
    *_, free, _ = update(table, lens, added, [1, 8, 0, 0], 2, 4, 0)
    assert free == [1, 8, 3, 4] and fq.device_status() == 4


def test_pages_given_away_among_many_given_back():
    """More than a thousand pages given back in one step, a few of them marked."""
    rng = np.random.default_rng(1)
    B, width, size = 90, 60, 2
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    table[rng.random((B, width)) < 0.05] = -1
    lens = rng.integers(0, width * size + 1, B).astype(np.int32)
    added = np.where(rng.random(B) < 0.8, -1, 0).astype(np.int32)
    want = [int(p) for b in range(B) if added[b] < 0 for p in table[b, :-(-lens[b] // size)] if p >= 0]
    *_, free, _ = update(table, lens, added, np.zeros(B * width, np.int32), 0, size, 0)
    assert free == want and len(want) > 1024                  # more than a thread block takes at once


@pytest.mark.parametrize("max_tokens", [40, 5000])
def test_pages_marked_entries_take_no_token(max_tokens):
    """A free list, or a request's last page, that holds no page: the tokens have slot -1 and it is reported."""
    size = 4
    slots, _, _, _, table = update([[2, -1, -1, -1]], [3], [9], [9, 8, -5, 7], 4, size, max_tokens)
    assert fq.device_status() == 4
    assert slots[:9].tolist() == [11, 28, 29, 30, 31, -1, -1, -1, -1] and (slots[9:] == -1).all()
    assert table[0].tolist() == [2, 7, -1, -1]
    slots, _, _, _, _ = update([[2, -3, -1, -1]], [6], [4], [9, 8, 7], 3, size, max_tokens)
    assert fq.device_status() == 4
    assert slots[:4].tolist() == [-1, -1, 28, 29]


# ------------------------------------------------------------------ together

def test_steps_back_to_back_equal_steps_apart():
    """Decoding steps one after another without a pause (each kernel starts while its predecessor writes what it
    reads) against the same steps with the device idle between any two calls."""
    B, hq, hk, d, size, P, width, steps = 24, 32, 8, 128, 16, 400, 16, 150
    turns, _ = fq.rope_turns(d, device="cuda")
    x = dev_bf16(bf16(np.random.default_rng(3), steps, B, hq + 2 * hk, d))
    added = torch.ones((steps, B), dtype=torch.int32, device="cuda")
    added[40:, 3] = 0
    added[60, 5] = -1
    added[90, 7] = -1
    got = []
    for apart in (False, True):
        kc, vc = (torch.zeros((P, size, hk, d), dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros((hk, P * size), device="cuda") for _ in range(2))
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        free = torch.arange(P, dtype=torch.int32, device="cuda")
        count = torch.tensor([P], dtype=torch.int32, device="cuda")
        out = torch.empty((steps, B, hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((steps, B, hq), device="cuda")
        slots, pos = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        q = torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            for call in (
                    lambda: fq.fp8_kv_pages_update(table, lens, added[i], free, count, size, slots=slots, positions=pos),
                    lambda: fq.fp8_kv_append(x[i, :, :hq], x[i, :, hq:hq + hk], x[i, :, hq + hk:], slots, kc, vc, ks, vs, 0, 3,
                                             positions=pos, turns=turns, q_out=q),
                    lambda: fq.fp8_attention_paged(q, kc, vc, ks, vs, table, lens, 0, 3, out=out[i], lse=lse[i])):
                call()
                if apart:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        got.append((kc, vc, ks, vs, table, lens, free, count, out, lse))
    assert int(host(got[0][5]).max()) == steps and torch.isfinite(got[0][8]).all()
    assert all(torch.equal(a, b) for a, b in zip(*got))
