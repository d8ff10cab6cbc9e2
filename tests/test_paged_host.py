"""Paged KV cache on the host: refusals of the C ABI and the binding, the rotation table and the
attention's division of work.  No call here reaches a kernel."""
import ctypes
import math
import random

import pytest
import torch

import fp8_quantization_amax_b200 as fq

P = ctypes.c_void_p
A, B, MIS, MIS4 = 1 << 20, 1 << 24, (1 << 20) + 8, (1 << 20) + 2
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="dummy device pointers: run on a host without a GPU")


@pytest.fixture(scope="module")
def L():
    from fp8_quantization_amax_b200 import build
    build.build()
    return fq.lib()


def pages(**kw):
    d = dict(k_codes=A, v_codes=B, k_scales=A, v_scales=B, num_pages=4, page_size=16, heads=2, head_dim=64,
             page_stride=2048, token_stride=128, head_stride=64, f=0, g=1)
    d.update(kw)
    return fq._KvPages(*[d[n] for n, _ in fq._KvPages._fields_])


BAD_CACHES = [
    (dict(f=2), 1), (dict(g=4), 1), (dict(g=-1), 1), (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(heads=0), 1),
    (dict(head_dim=0), 1), (dict(head_dim=72), 1), (dict(head_dim=24), 1), (dict(page_stride=2056), 1),
    (dict(token_stride=136), 1), (dict(head_stride=72), 1), (dict(head_dim=272, head_stride=272, token_stride=544), 2),
    (dict(num_pages=1 << 28), 2), (dict(page_size=1 << 31), 2), (dict(heads=1 << 20), 2),
    (dict(page_stride=1 << 35), 2), (dict(page_stride=1 << 62), 2),
    (dict(head_stride=48), 1), (dict(head_stride=0), 1), (dict(token_stride=0), 1), (dict(page_stride=-2048), 1),
    (dict(k_codes=None), 1), (dict(v_codes=None), 1), (dict(k_codes=MIS), 1), (dict(k_scales=None), 1),
    (dict(v_scales=MIS4), 1),
]


def attention_args(cache, **kw):
    d = dict(q=A, q_stride=512, q_heads=8, table=A, batch=3, max_pages=5, lens=A, scale=0.125, window=0, sinks=0, out=B,
             out_stride=512, lse=A, ws=A, ws_bytes=1 << 30, stream=None)
    d.update(kw)
    return [ctypes.byref(cache)] + list(d.values())


def append_args(cache, **kw):
    d = dict(q=A, q_stride=768, q_heads=8, k=A, k_stride=768, v=A, v_stride=768, tokens=3, slots=A, positions=A, turns=A,
             rot=64, interleaved=0, gain=1.0, q_weight=A, k_weight=A, eps=1e-6, q_out=B, q_out_stride=512, stream=None)
    d.update(kw)
    return [ctypes.byref(cache)] + list(d.values())


def update_args(**kw):
    d = dict(table=A, batch=3, max_pages=5, page_size=16, lens=A, added=A, lens_out=A, free=A, num_pages=20, count=A,
             count_out=A, max_tokens=8, slots=A, positions=A, offsets=A, served=A, ws=None, ws_bytes=0, stream=None)
    d.update(kw)
    return list(d.values())


@host_only
@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches_are_refused(L, change, status):
    assert L.fp8_attention_paged(*attention_args(pages(**change))) == status
    assert L.fp8_kv_append(*append_args(pages(**change))) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(q=MIS), 1), (dict(out=None), 1), (dict(out=MIS), 1), (dict(lens=None), 1), (dict(lens=MIS4), 1),
    (dict(table=None), 1), (dict(table=MIS4), 1), (dict(q_stride=508), 1), (dict(out_stride=500), 1), (dict(q_stride=256), 1),
    (dict(q_heads=0), 1), (dict(q_heads=7), 1), (dict(batch=-1), 1), (dict(max_pages=-1), 1), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(lse=MIS4), 1), (dict(max_pages=1 << 28), 2), (dict(batch=1 << 12, max_pages=1 << 19), 2), (dict(q_heads=1 << 17), 2), (dict(max_pages=500, ws=None, ws_bytes=0), 3),
    (dict(max_pages=500, ws_bytes=100), 3), (dict(max_pages=500, ws=MIS), 3), (dict(batch=0, q=None, out=None), 0),
])
def test_attention_refuses(L, change, status):
    assert L.fp8_attention_paged(*attention_args(pages(), **change)) == status


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(k=(1 << 20) + 4), 1), (dict(slots=MIS4), 1), (dict(k_stride=766), 1), (dict(v_stride=64), 1), (dict(q_stride=256), 1),
    (dict(q_out_stride=100), 1), (dict(positions=None), 1), (dict(turns=None), 1), (dict(rot=60), 1), (dict(rot=72), 1),
    (dict(rot=-8), 1), (dict(tokens=-1), 1), (dict(q_heads=-1), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(q_weight=(1 << 20) + 4), 1), (dict(k_weight=MIS4), 1), (dict(tokens=0, k=None, v=None, slots=None), 0),
])
def test_append_refuses(L, change, status):
    assert L.fp8_kv_append(*append_args(pages(), **change)) == status


@host_only
def test_append_refuses_scales_of_whole_blocks(L):
    assert L.fp8_kv_append(*append_args(pages(g=2))) == 2


@host_only
@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), 1), (dict(max_pages=-1), 1), (dict(page_size=0), 1), (dict(num_pages=-1), 1), (dict(max_tokens=-1), 1),
    (dict(table=None), 1), (dict(table=MIS4), 1), (dict(lens=None), 1), (dict(added=None), 1), (dict(lens_out=None), 1),
    (dict(free=None), 1), (dict(count=None), 1), (dict(count_out=None), 1), (dict(slots=None), 1), (dict(slots=MIS4), 1),
    (dict(positions=None), 1), (dict(offsets=None), 1), (dict(served=None), 1), (dict(max_pages=1 << 28), 2),
    (dict(num_pages=1 << 28), 2), (dict(max_tokens=1 << 33), 2), (dict(batch=1 << 20, max_pages=1 << 12), 2),
    (dict(max_tokens=5000), 3), (dict(max_tokens=5000, ws=A, ws_bytes=8), 3), (dict(batch=1025), 3),
])
def test_pages_update_refuses(L, change, status):
    assert L.fp8_kv_pages_update(*update_args(**change)) == status


def test_workspace_sizes(L):
    assert fq.pages_workspace_bytes(1024, 4096) == 0
    assert fq.pages_workspace_bytes(1024, 4097) >= 1024 * 8
    assert fq.pages_workspace_bytes(-1, 5) == 0
    for batch in (1, 9):                                                   # short requests are not divided
        assert fq.attention_workspace_bytes(batch, 64, 32, 8, 128) == 0
        assert fq.attention_workspace_bytes(batch, 1040, 32, 8, 128) > 0
    assert fq.attention_workspace_bytes(1, 4096, 30, 8, 128) == 0          # not a layout
    a = fq.attention_workspace_bytes(1, 4096, 32, 8, 128)
    assert a == fq.attention_workspace_bytes(64, 1 << 20, 32, 8, 128)      # set by the machine, not the lengths


def test_binding_refuses():
    e = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype)  # noqa: E731
    k, s1 = e(4, 16, 2, 64), e(2, dtype=torch.float32)
    q, t, n = e(3, 8, 64, dtype=torch.bfloat16), e(3, 5, dtype=torch.int32), e(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8_attention_paged(q, k, k, s1, s1, t, n)
    with pytest.raises(TypeError):
        fq.fp8_attention_paged(q.float(), k, k, s1, s1, t, n)
    with pytest.raises(TypeError):
        fq.fp8_attention_paged(q, k.float(), k, s1, s1, t, n)
    with pytest.raises(TypeError):
        fq.fp8_attention_paged(q, k, k, s1, s1, t.long(), n)
    with pytest.raises(TypeError):
        fq.fp8_attention_paged(q, k, k, s1.double(), s1, t, n)
    for bad in (dict(q=q[:, :7]), dict(q=q[..., :32]), dict(k=k[:, :, :1]), dict(v=k[:2]), dict(s=e(3, dtype=torch.float32)),
                dict(t=t[:2]), dict(n=n[:2]), dict(gran=0), dict(gran=3), dict(q=q.transpose(1, 2)),
                dict(k=k.transpose(2, 3), v=k.transpose(2, 3)), dict(v=k.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(q=q, k=k, v=k, s=s1, t=t, n=n, gran=1)
        a.update(bad)
        with pytest.raises(ValueError):
            fq.fp8_attention_paged(a["q"], a["k"], a["v"], a["s"], a["s"], a["t"], a["n"], 0, a["gran"])
    x, slots = e(3, 2, 64, dtype=torch.bfloat16), e(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8_kv_append(q, x, x, slots, k, k, s1, s1)
    turns, pos = e(32, dtype=torch.int64), e(3, dtype=torch.int32)
    for bad in (dict(k=x[:2]), dict(v=x[:, :1]), dict(q=q[:2]), dict(slots=slots[:2]), dict(turns=turns),
                dict(turns=turns, positions=pos[:1]), dict(q_weight=e(32, dtype=torch.bfloat16)), dict(q=None, q_out=q),
                dict(q_out=q[:, :4])):
        a = dict(q=q, k=x, v=x, slots=slots)
        a.update(bad)
        with pytest.raises(ValueError):
            fq.fp8_kv_append(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("slots"), k, k, s1, s1, **a)
    free, count = e(20, dtype=torch.int32), e(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_tokens"):
        fq.fp8_kv_pages_update(t, n, n, free, count, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8_kv_pages_update(t, n, n, free, count, 16, 8)
    with pytest.raises(TypeError):
        fq.fp8_kv_pages_update(t, n.long(), n, free, count, 16, 8)
    with pytest.raises(ValueError):
        fq.fp8_kv_pages_update(t, n[:2], n, free, count, 16, 8)


# ------------------------------------------------------------------ rotation table

def turns_of(*a, **kw):
    t, gain = fq.rope_turns(*a, **kw)
    return [x % (1 << 64) / 2.0 ** 64 for x in t.tolist()], gain


@pytest.mark.parametrize("rot", [0, 8, 24, 64, 128, 256])
def test_plain_frequencies(rot):
    got, gain = turns_of(rot, 500000.0)
    assert gain == 1.0 and len(got) == rot // 2
    for i, g in enumerate(got):
        # the table's unit is 2^-64 of a turn (half of it lost in rounding); power and quotient in 53 bits
        want = 500000.0 ** (-2 * i / rot) / (2 * math.pi)
        assert abs(g - want) <= 2.0 ** -64 + want * 2.0 ** -51


def test_stretched_frequencies():
    plain, _ = turns_of(128, 500000.0)
    linear, gain = turns_of(128, 500000.0, fq.ROPE_LINEAR, 8.0)
    assert gain == 1.0 and all(abs(8 * a - b) <= 9 * 2.0 ** -64 + b * 2.0 ** -50 for a, b in zip(linear, plain))
    smooth, gain = turns_of(128, 500000.0, fq.ROPE_SMOOTH, 8.0, 8192.0, 1.0, 4.0)
    assert gain == 1.0
    for f, s in zip(plain, smooth):
        n = 8192.0 * f                                  # turns over the original length
        mix = min(1.0, max(0.0, (n - 1.0) / 3.0))
        # f is read back with an error of 2^-65, times at most 8192 / 3 where it moves the mix
        assert abs(s - f * (mix + (1 - mix) / 8.0)) <= 2.0 ** -64 * (1 + f * 8192) + f * 2.0 ** -48
    ramp, gain = turns_of(128, 10000.0, fq.ROPE_RAMP, 16.0, 4096.0, 1.0, 32.0)
    plain, _ = turns_of(128, 10000.0)
    assert math.isclose(gain, 0.1 * math.log(16.0) + 1.0, rel_tol=1e-6)
    ratio = [r / p for r, p in zip(ramp, plain)]
    # a frequency of 10000^-1 / 2 pi turns keeps 2^-64 / 1e-5 of itself: 6e-15
    assert ratio[0] == 1.0 and math.isclose(ratio[-1], 1 / 16, rel_tol=1e-12)
    assert all(a >= b - 2.0 ** -40 for a, b in zip(ratio, ratio[1:]))
    for i, r in enumerate(ratio):                        # untouched above 32 turns, stretched fully below 1
        n = 4096.0 * plain[i]
        assert n < 40.0 or r == 1.0
        assert n > 0.9 or math.isclose(r, 1 / 16, rel_tol=1e-12)


@pytest.mark.parametrize("args", [(12,), (264,), (-8,), (64, 0.0), (64, -1.0), (64, math.inf), (64, 1e4, 4), (64, 1e4, 1, 0.5),
                                  (64, 1e4, 2, 8.0, 0.0), (64, 1e4, 2, 8.0, 8192.0, 4.0, 1.0), (64, 1.0, 3, 8.0),
                                  (64, 1e4, 1, math.nan)])
def test_rope_refuses(args):
    with pytest.raises(fq.Fp8qError) as e:
        fq.rope_turns(*args)
    assert e.value.status == 1


# ------------------------------------------------------------------ division of the attention's work

def test_attention_split_holds_for_any_batch():
    rng = random.Random(2)
    for _ in range(400):
        lens = [rng.choice((0, 1, 15, 16, 17, rng.randint(0, 3000))) for _ in range(rng.randint(1, 40))]
        for window, sinks in ((0, 0), (1, 0), (1, 1), (rng.randint(1, 600), rng.randint(0, 50)), (100, 10 ** 6)):
            assert fq.check_attention_split(lens, window, sinks, rng.choice((1, 2, 37, 148, 296, 1184))) == 0
    for workers in (1, 2, 3, 37, 148, 1024):
        for n in range(0, 200):
            assert fq.check_attention_split([n], 0, 0, workers) == 0
            assert fq.check_attention_split([n, 16, n], 0, 0, workers) == 0
            assert fq.check_attention_split([n % 17] * 40, 0, 0, workers) == 0
    assert fq.check_attention_split([], 0, 0, 148) == 0
    assert fq.check_attention_split([131072], 0, 0, 296) == 0
    assert fq.check_attention_split([1], -1, 0, 148) == -1
    assert fq.check_attention_split([1], 0, 0, 0) == -1
