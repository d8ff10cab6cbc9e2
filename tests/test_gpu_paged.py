"""GPU tests of the paged KV cache: page bookkeeping, append and attention against plain 64-bit forms.

Tolerances are derived in paged_reference.py and beside each check; integers, V's codes and K's
codes without norm and rotation are exact.
"""
import numpy as np
import pytest
import torch

import fp8_quantization_amax_b200 as fq
import paged_reference as ref
from helpers import assert_codes_equal, assert_f32_bits_equal, dev, dev_bf16, host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean():
    assert torch.cuda.is_available()
    assert fq.device_status() == 0
    yield
    assert fq.device_status() == 0


def bf16(rng, *shape, std=1.0):
    x = (rng.standard_normal(shape) * std).astype(np.float32)
    u = x.view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


# ------------------------------------------------------------------ attention

class Cache:
    """A cache with lens of each request in random pages; all that no request sees holds NaN."""

    def __init__(self, rng, lens, heads, d, size, fmt, gran, layout="thd", spare=2, window=0, sinks=0, max_pages=None):
        B = len(lens)
        held = [-(-n // size) for n in lens]
        P = sum(held) + spare
        width = max_pages or max(1, max(held))
        ids = rng.permutation(P).astype(np.int32)
        table = np.full((B, width), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + held[b]]
            at += held[b]
        S = P * size
        seen = np.zeros(S, bool)
        for b in range(B):
            for t in range(lens[b]):
                if not window or t >= lens[b] - window or t < sinks:
                    seen[table[b, t // size] * size + t % size] = True
        if window:                                   # pages out of sight may have been given away
            for b in range(B):
                for j in range(held[b]):
                    if not seen[table[b, j] * size:(table[b, j] + 1) * size].any():
                        table[b, j] = -1
        codes = []
        for _ in range(2):
            x = rng.integers(0, 256, (P, size, heads, d)).astype(np.uint8)
            x[(x & 0x7F) >= (0x7F if fmt == 0 else 0x7C)] ^= 0x08     # finite codes
            if fmt == 1:
                x[(x & 0x7F) >= 0x60] ^= 0x40                          # a normal spread of exponents
            x.reshape(S, heads, d)[~seen] = 0x7F
            codes.append(x)
        shape = fq.kv_page_scale_shape(P, size, heads, gran)
        scales = [np.exp2(rng.uniform(-12, -4 if fmt == 0 else -8, shape)).astype(np.float32) for _ in range(2)]
        if gran == 3:
            for s in scales:
                s[:, ~seen] = np.nan
        self.k, self.v = codes
        self.ks, self.vs = scales
        self.table, self.lens = table, np.array(lens, np.int32)
        self.fmt, self.gran = fmt, gran

        def place(x):
            if layout == "thd":
                return dev(x)
            if layout == "htd":                      # [page][head][token][dim]
                return dev(x.transpose(0, 2, 1, 3)).transpose(1, 2)
            wide = torch.full((P, size, heads + 1, d + 16), 0x7F, dtype=torch.uint8, device="cuda")
            wide[:, :, :heads, :d] = dev(x)
            return wide[:, :, :heads, :d]
        self.dk, self.dv = place(self.k), place(self.v)
        self.dks, self.dvs = dev(self.ks), dev(self.vs)
        self.dtable, self.dlens = dev(self.table), dev(self.lens)

    def run(self, q, **kw):
        return fq.fp8_attention_paged(q, self.dk, self.dv, self.dks, self.dvs, self.dtable, self.dlens, self.fmt,
                                      self.gran, **kw)

    def check(self, q_bits, out, lse, scale, window=0, sinks=0):
        want, wl, tol, ltol = ref.attention(ref.bf16_to_f64(q_bits), self.k, self.v, self.ks, self.vs, self.table,
                                            self.lens, self.fmt, self.gran, scale, window, sinks)
        got = ref.bf16_to_f64(host(out))
        assert np.isfinite(got).all()
        off = np.abs(got - want) - tol
        assert (off <= 0).all(), f"out: {np.argwhere(off > 0)[:4]} off by {off.max()}, got {got[off > 0][:4]} want {want[off > 0][:4]}"
        got = host(lse).astype(np.float64)
        empty = np.isneginf(wl)
        assert np.array_equal(np.isneginf(got), empty)
        assert (np.abs(got - wl)[~empty] <= ltol[~empty]).all()


def attend(seed, lens, heads, group, d, size, fmt, gran, window=0, sinks=0, layout="thd", scale=None, **kw):
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, heads, d, size, fmt, gran, layout, window=window, sinks=sinks, **kw)
    qb = bf16(rng, len(lens), heads * group, d)
    out, lse = c.run(dev_bf16(qb), window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    c.check(qb, out, lse, d ** -0.5 if scale is None else scale, window, sinks)
    return c, qb, out, lse


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("gran", [0, 1, 2, 3])
@pytest.mark.parametrize("lens", [[1], [0], [15, 16, 17], [33, 0, 100, 1], [500, 3, 0, 64]])
def test_attention_small(fmt, gran, lens):
    attend(len(lens) + gran, lens, 2, 4, 128, 16, fmt, gran)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 8), (1, 9), (1, 16), (1, 17), (1, 40), (2, 7), (3, 4), (4, 12),
                                         (5, 1), (7, 2), (8, 8), (11, 3), (16, 1), (24, 2)])
def test_attention_head_layouts(heads, group):
    attend(heads * 100 + group, [70, 1, 133, 16], heads, group, 64, 16, 0, 1)


@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 256])
def test_attention_head_dims(d, group):
    attend(d, [5, 90, 200], 2, group, d, 16, 0, 3)
    attend(d + 1, [31, 64], 3, group, d, 16, 1, 0)


@pytest.mark.parametrize("size", [1, 3, 5, 8, 16, 24, 32, 48, 128, 1000])
def test_attention_page_sizes(size):
    attend(size, [1, 40, 257, 0, 300], 2, 4, 64, size, 0, 1)
    attend(size + 1, [77, 130], 1, 8, 128, size, 0, 2)
    attend(size + 2, [77, 130], 8, 1, 128, size, 0, 3, layout="htd")


@pytest.mark.parametrize("layout", ["thd", "htd", "wide"])
@pytest.mark.parametrize("gran", [1, 3])
def test_attention_strides(layout, gran):
    attend(3, [100, 17, 301], 4, 4, 128, 16, 0, gran, layout=layout)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (16, 4), (17, 16), (100, 17), (64, 300), (1000, 5), (333, 0)])
@pytest.mark.parametrize("size", [16, 24])
def test_attention_window(window, sinks, size):
    attend(window + sinks, [1, 2, 16, 90, 117, 500, 0, 801], 2, 4, 64, size, 0, 3 if size == 16 else 1, window, sinks)


@pytest.mark.parametrize("lens", [[20000], [9000, 1, 12000, 0, 700], [64] * 300, [0] * 40 + [3000] + [0] * 30,
                                  [1] * 700])
@pytest.mark.parametrize("gran", [1, 3])
def test_attention_shared_requests(lens, gran):
    """Requests divided over many blocks, several requests in one block, more requests than threads."""
    attend(7, lens, 2, 4, 64, 16, 0, gran)


def test_attention_one_head_shared_by_warps():
    attend(1, [3000, 40, 5000], 1, 8, 128, 16, 0, 1)
    attend(2, [3000, 40, 5000], 3, 16, 128, 16, 0, 3)
    attend(3, [3000, 40, 700], 1, 2, 256, 32, 1, 0)


@pytest.mark.parametrize("heads,group,d", [(5, 12, 128), (10, 4, 128), (3, 16, 128), (17, 1, 64), (1, 16, 256), (5, 9, 192),
                                           (9, 12, 256), (2, 40, 160)])
@pytest.mark.parametrize("size", [8, 16, 24])
def test_attention_groups_of_heads(heads, group, d, size):
    """Heads that do not fill a block's warps, wide heads with many query heads; pages of whole and half tiles."""
    attend(heads + d, [70, 1, 333, 16, 0, 1200], heads, group, d, size, 0, 1)
    attend(heads + d, [64, 200], heads, group, d, size, 1, 3)


def test_attention_scale_and_extreme_scores():
    """Scores far apart (one token takes all), tiny and huge queries, scales many octaves apart."""
    rng = np.random.default_rng(5)
    c = Cache(rng, [200, 64], 2, 64, 16, 0, 3)
    for factor in (2.0 ** -60, 1.0, 30.0, 3000.0):
        x = rng.standard_normal((2, 8, 64)).astype(np.float32) * np.float32(factor)
        qb = (x.view(np.uint32) >> 16).astype(np.uint16)
        for scale in (0.125, 1.0):
            out, lse = c.run(dev_bf16(qb), scale=scale)
            torch.cuda.synchronize()
            c.check(qb, out, lse, scale)
    # V's scales from 2^-40 to 2^20: the large ones on tokens of little weight
    c.vs[:] = np.where(np.isnan(c.vs), c.vs, np.exp2(rng.uniform(-40, 20, c.vs.shape))).astype(np.float32)
    c.vs[0, c.table[0, 2] * 16 + 3] = 0.0
    c.dvs.copy_(dev(c.vs))
    qb = bf16(rng, 2, 8, 64)
    out, lse = c.run(dev_bf16(qb), scale=0.3)
    torch.cuda.synchronize()
    c.check(qb, out, lse, 0.3)


def test_attention_rows_of_nan_and_inf_stay_their_own():
    rng = np.random.default_rng(6)
    c = Cache(rng, [100, 100], 2, 64, 16, 0, 1)
    qb = bf16(rng, 2, 8, 64)
    base, _ = c.run(dev_bf16(qb))
    bad = qb.copy()
    bad[0, 1, 5] = 0x7FC0
    out, _ = c.run(dev_bf16(bad))
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 1]).all()
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(out.cpu()[keep], base.cpu()[keep])
    # a visible NaN code reaches its own head and request only
    c.dk[int(c.table[1, 0]), 3, 0, 7] = 0x7F
    out, _ = c.run(dev_bf16(qb))
    torch.cuda.synchronize()
    assert torch.isnan(out[1, :4]).all()
    assert torch.equal(out[0].cpu(), base[0].cpu()) and torch.equal(out[1, 4:].cpu(), base[1, 4:].cpu())


def test_attention_all_zero():
    rng = np.random.default_rng(6)
    c = Cache(rng, [50], 1, 64, 16, 0, 3)
    for t in (c.dk, c.dv):
        t.zero_()
    c.dks.zero_()
    c.dvs.zero_()
    out, lse = c.run(dev_bf16(bf16(rng, 1, 4, 64)))
    torch.cuda.synchronize()
    assert (out == 0).all()
    assert np.allclose(host(lse), np.log(50.0), rtol=1e-6)


def test_attention_outputs_given_strided_and_wide_table():
    rng = np.random.default_rng(9)
    c = Cache(rng, [40, 0, 333], 2, 64, 16, 0, 1, max_pages=37)
    qb = bf16(rng, 3, 8, 64)
    big = torch.zeros(3, 24, 64, dtype=torch.bfloat16, device="cuda")
    big[:, 8:16] = dev_bf16(qb)
    want, wl = c.run(dev_bf16(qb))
    room = torch.full((3, 24, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 8, device="cuda")
    out, l2 = c.run(big[:, 8:16], out=room[:, 16:], lse=lse)
    torch.cuda.synchronize()
    c.check(qb, want, wl, 0.125)
    assert torch.equal(out, want) and torch.equal(lse, wl) and l2 is lse
    assert (room[:, :16] == 7.0).all()


def test_attention_without_pages_or_cache():
    """No table column: nothing is visible.  A cache of no pages: every visible token is reported, and
    counts as zeros."""
    q = dev_bf16(bf16(np.random.default_rng(1), 3, 8, 64))
    s = torch.ones(2, device="cuda")
    lens = torch.tensor([5, 0, 70], dtype=torch.int32, device="cuda")
    k = torch.zeros((2, 16, 2, 64), dtype=torch.uint8, device="cuda")
    out, lse = fq.fp8_attention_paged(q, k, k, s, s, torch.empty((3, 0), dtype=torch.int32, device="cuda"), lens)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all() and fq.device_status() == 0
    none = k[:0]
    out, lse = fq.fp8_attention_paged(q, none, none, s, s, torch.zeros((3, 5), dtype=torch.int32, device="cuda"), lens)
    torch.cuda.synchronize()
    assert fq.device_status() == 4
    assert (out == 0).all() and np.allclose(host(lse)[[0, 2]], np.log([[5.0], [70.0]]), rtol=1e-6)


@pytest.mark.parametrize("lens", [[64], [63], [17, 1], [1, 16, 2], [32, 32], [33] * 9, [65, 3, 64], [5] * 40 + [200]])
@pytest.mark.parametrize("heads", [1, 8])
def test_attention_few_tiles(lens, heads):
    """Around the number of tiles from which a request is divided, with one head's tiles on all warps or few."""
    attend(sum(lens), lens, heads, 4, 64, 16, 0, 1, max_pages=max(-(-n // 16) for n in lens))


@pytest.mark.parametrize("batch,heads,most", [(1, 1, 15), (140, 1, 16), (100, 1, 40), (18, 8, 200), (19, 8, 200), (2, 40, 513),
                                              (1, 8, 512), (5, 3, 300), (149, 1, 30), (1, 200, 100)])
@pytest.mark.parametrize("gran", [1, 3])
def test_attention_heads_spread(batch, heads, most, gran):
    """Few short requests: heads on blocks of their own, blocks of a warp or several, more requests than threads."""
    rng = np.random.default_rng(batch * heads)
    lens = [int(x) for x in rng.integers(0, most + 1, batch)]
    lens[batch // 2] = most
    attend(most, lens, heads, 3, 64, 16, 0, gran, max_pages=-(-most // 16))
    attend(most + 1, lens, heads, 2, 128, 24, 1, gran, 9, 2, max_pages=-(-most // 24))


def test_attention_same_bits_again_and_beside_other_work():
    rng = np.random.default_rng(11)
    c = Cache(rng, [5000, 300, 7000], 8, 128, 16, 0, 1)
    q = dev_bf16(bf16(rng, 3, 32, 128))
    want = c.run(q)
    side, side2 = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    side2.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        with torch.cuda.stream(side):
            got.append(c.run(q))
        with torch.cuda.stream(side2):
            got.append(c.run(q))
        a = torch.randn(2048, 2048, device="cuda")
        (a @ a).sum()
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_attention_in_graphs():
    """Two captured graphs replayed at the same time, on lengths that change between replays."""
    rng = np.random.default_rng(12)
    c = Cache(rng, [2000, 900, 3000], 8, 128, 16, 0, 3)
    qb = bf16(rng, 3, 32, 128)
    q = dev_bf16(qb)
    c.run(q)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(q))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([2000, 900, 3000], [5, 900, 0], [0, 0, 0], [2000, 1, 2999]):
        c.lens = np.array(lens, np.int32)
        c.dlens.copy_(dev(c.lens))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for out, lse in outs:
            c.check(qb, out, lse, 128 ** -0.5)


def test_attention_bad_pages_and_lengths():
    """A page outside the cache is read as zeros, a length beyond the table clipped; both are reported."""
    rng = np.random.default_rng(13)
    c = Cache(rng, [64, 64], 2, 64, 16, 0, 1)
    qb = bf16(rng, 2, 8, 64)
    want, _ = c.run(dev_bf16(qb))
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c.table.copy()
        t[1, 2] = bad
        out, _ = fq.fp8_attention_paged(dev_bf16(qb), c.dk, c.dv, c.dks, c.dvs, dev(t), c.dlens, 0, 1)
        torch.cuda.synchronize()
        assert fq.device_status() == 4
        assert torch.equal(out[0], want[0]) and torch.isfinite(out).all()
    for n in (65, 1 << 20, 2 ** 31 - 1):
        out, _ = fq.fp8_attention_paged(dev_bf16(qb), c.dk, c.dv, c.dks, c.dvs, c.dtable,
                                        dev(np.array([64, n], np.int32)), 0, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    out, lse = fq.fp8_attention_paged(dev_bf16(qb), c.dk, c.dv, c.dks, c.dvs, c.dtable,
                                      dev(np.array([64, -5], np.int32)), 0, 1)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_offsets_beyond_32_bits():
    """Append to and attention over the last pages of a cache of more than 2^32 bytes."""
    P, size, H, D = 300000, 16, 8, 128
    k = torch.empty((P, size, H, D), dtype=torch.uint8, device="cuda")
    v = torch.empty((P, size, H, D), dtype=torch.uint8, device="cuda")
    assert k.numel() > 2 ** 32
    ks = torch.full((H, P * size), float("nan"), device="cuda")
    vs = torch.full((H, P * size), float("nan"), device="cuda")
    rng = np.random.default_rng(1)
    n = 100
    pages = np.array([P - 1, 7, P - 3, P - 2, 0, P // 2, P - 9], np.int32)
    slots = np.array([int(pages[t // size]) * size + t % size for t in range(n)], np.int64)
    kb, vb = bf16(rng, n, H, D), bf16(rng, n, H, D)
    fq.fp8_kv_append(None, dev_bf16(kb), dev_bf16(vb), dev(slots), k, v, ks, vs, 0, 3)
    qb = bf16(rng, 1, 32, D)
    out, _ = fq.fp8_attention_paged(dev_bf16(qb), k, v, ks, vs, dev(pages[None]), dev(np.array([n], np.int32)), 0, 3)
    # the same tokens in a small cache
    P2 = len(pages)
    k2 = k[torch.from_numpy(pages.astype(np.int64)).cuda()].contiguous()
    v2 = v[torch.from_numpy(pages.astype(np.int64)).cuda()].contiguous()
    at = torch.from_numpy((pages.astype(np.int64)[:, None] * size + np.arange(size)).reshape(-1)).cuda()
    out2, _ = fq.fp8_attention_paged(dev_bf16(qb), k2, v2, ks[:, at].contiguous(), vs[:, at].contiguous(),
                                     dev(np.arange(P2, dtype=np.int32)[None]), dev(np.array([n], np.int32)), 0, 3)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.isfinite(out).all()
    c, s = fq.fp8_quantize(dev_bf16(kb).view(n, H * D), 0, fq.GROUP_1x128)
    got = k.view(-1, H * D)[torch.from_numpy(slots).cuda()]
    assert torch.equal(got, c)
    assert torch.equal(ks[:, torch.from_numpy(slots).cuda()], s)


@pytest.mark.parametrize("gran", [0, 1, 2])
@pytest.mark.parametrize("fmt", [0, 1])
def test_attention_reads_what_the_kv_quantizer_writes(gran, fmt):
    import synth
    T, H, D = 512, 8, 128
    kb, vb = synth.kv_70b(seed=2, tokens=T, heads=H, head_dim=D)
    kc, vc, ks, vs = fq.fp8_kv_quantize(dev_bf16(kb), dev_bf16(vb), fmt, gran)
    rng = np.random.default_rng(2)
    qb = bf16(rng, 1, 64, D)
    size = 32
    table = np.arange(T // size, dtype=np.int32)[None]
    lens = np.array([T - 3], np.int32)
    out, lse = fq.fp8_attention_paged(dev_bf16(qb), kc.view(-1, size, H, D), vc.view(-1, size, H, D), ks, vs, dev(table),
                                      dev(lens), fmt, gran)
    torch.cuda.synchronize()
    want, wl, tol, ltol = ref.attention(ref.bf16_to_f64(qb), host(kc).reshape(-1, size, H, D),
                                        host(vc).reshape(-1, size, H, D), host(ks), host(vs), table, lens, fmt, gran,
                                        D ** -0.5, 0, 0)
    assert (np.abs(ref.bf16_to_f64(host(out)) - want) <= tol).all()
    assert (np.abs(host(lse) - wl) <= ltol).all()


# ------------------------------------------------------------------ append

def append_case(seed, T, hq, hk, d, size, fmt, gran, rot=0, interleaved=False, with_norm=False, positions=None,
                pads=(), layout="thd", std=1.0, gain=1.0, base=500000.0, inplace=False):
    rng = np.random.default_rng(seed)
    P = -(-T // size) + 2
    slots = rng.permutation(P * size)[:T].astype(np.int64)
    slots[list(pads)] = -1
    qkv = bf16(rng, T, hq + 2 * hk, d, std=std)
    wq, wk = (bf16(rng, d) if with_norm else None for _ in range(2))
    positions = rng.integers(0, 1 << 20, T).astype(np.int32) if positions is None else np.asarray(positions, np.int32)
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    shape = fq.kv_page_scale_shape(P, size, hk, gran)
    ks, vs = (rng.uniform(0.5, 2.0, shape).astype(np.float32) * np.float32(6.0 * std / ref.FMAX[fmt]) for _ in range(2))
    kc, vc = (rng.integers(0, 256, (P, size, hk, d)).astype(np.uint8) for _ in range(2))
    if layout == "thd":
        dk, dv = dev(kc), dev(vc)
    else:
        dk, dv = (dev(x.transpose(0, 2, 1, 3)).transpose(1, 2) for x in (kc, vc))
    dks, dvs = dev(ks), dev(vs)
    x = dev_bf16(qkv)
    turns = fq.rope_turns(rot, base, device="cuda")[0] if rot else None
    eps = 1e-5
    q = x[:, :hq] if hq else None
    out = fq.fp8_kv_append(q, x[:, hq:hq + hk], x[:, hq + hk:], dev(slots), dk, dv, dks, dvs, fmt, gran,
                           positions=dev(positions) if rot else None, turns=turns, interleaved=interleaved, gain=gain,
                           q_weight=None if wq is None or not hq else dev_bf16(wq), k_weight=None if wk is None else dev_bf16(wk),
                           eps=eps, q_out=q if inplace else None)
    torch.cuda.synchronize()

    def through(part, w):
        y = ref.norm(ref.bf16_to_f64(part), None if w is None else ref.bf16_to_f64(w), eps)
        y, mag = ref.rotate(y, positions, freq, interleaved)
        if rot:
            y[..., :rot] *= gain
            mag[..., :rot] *= gain
        return y, mag
    # fp32 steps: the norm's sum, root and two products, cos and sin (2^-22 of a turn's unit) and the
    # rotation's two products: under 2^-18 of |a| + |b| for a row of up to 256
    SLOP = 2.0 ** -18
    if hq:
        y, mag = through(qkv[:, :hq], wq)
        got = ref.bf16_to_f64(host(out))
        assert (np.abs(got - y) <= np.abs(y) * 2.0 ** -8 + mag * SLOP + 1e-38).all()
    y, mag = through(qkv[:, hq:hq + hk], wk)
    vy = ref.bf16_to_f64(qkv[:, hq + hk:])
    val = ref.decode_table(fmt)
    live = slots >= 0
    for name, want, m, cache, before, dsc, given in (("k", y, mag, dk, kc, dks, ks), ("v", vy, np.abs(vy) * 0, dv, vc, dvs, vs)):
        got = host(cache).reshape(P * size, hk, d)
        sc = host(dsc)
        untouched = np.ones(P * size, bool)
        untouched[slots[live]] = False
        assert np.array_equal(got[untouched], before.reshape(P * size, hk, d)[untouched]), name
        if gran == 3:
            assert np.array_equal(sc[:, untouched].view(np.uint32), given[:, untouched].view(np.uint32))
            s = sc[:, slots[live]].T.astype(np.float64)
            top = np.abs(want[live]).max(-1) / ref.FMAX[fmt]
            assert (np.abs(s - top) <= top * 2.0 ** -23 + m[live].max(-1) / ref.FMAX[fmt] * SLOP + 1e-45).all(), name
        else:
            assert np.array_equal(sc.view(np.uint32), given.view(np.uint32))
            s = np.broadcast_to(given.reshape(1, -1), (int(live.sum()), hk)).astype(np.float64)
        code = val[got[slots[live]]]
        q = np.clip(want[live] / s[..., None], -ref.FMAX[fmt], ref.FMAX[fmt])
        slack = m[live] / s[..., None] * SLOP + np.abs(q) * 2.0 ** -22
        assert np.isfinite(code).all()
        assert (np.abs(code - q) <= np.maximum(np.abs(q) * ref.REL[fmt], ref.SUB[fmt]) + slack).all(), name
    return dict(x=qkv, slots=slots, k=host(dk), v=host(dv), ks=host(dks), vs=host(dvs), hq=hq, hk=hk, d=d, P=P, size=size)


@pytest.mark.parametrize("gran", [0, 1, 3])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [1, 3, 70])
def test_append_small(T, fmt, gran, interleaved):
    append_case(T + gran, T, 8, 2, 128, 16, fmt, gran, 128, interleaved, True, pads=[T // 2] if T > 2 else ())


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_head_dims_and_parts(d, interleaved):
    for rot in sorted({0, 8, d // 2 // 8 * 8, d}):
        append_case(d + rot, 37, 3, 3, d, 24, 0, 3, rot, interleaved, rot != 8)


@pytest.mark.parametrize("hq,hk", [(0, 1), (0, 8), (1, 1), (7, 1), (14, 2), (32, 8), (64, 8), (5, 5)])
def test_append_head_counts(hq, hk):
    append_case(hq + hk, 29, hq, hk, 128, 16, 0, 1, 64, False, True)


def test_append_many_tokens_and_layouts():
    append_case(1, 5000, 4, 2, 64, 16, 0, 3, 64, False, True, pads=range(4000, 4100))
    append_case(2, 5003, 2, 1, 128, 24, 1, 0, 64, True, False, layout="htd")
    append_case(3, 300, 8, 8, 128, 1, 0, 3, 128, False, False, layout="htd")


def test_append_rows_aligned_to_eight_bytes():
    rng = np.random.default_rng(12)
    T, hq, hk, d = 50, 4, 2, 128
    kv = torch.zeros((4, 16, hk, d), dtype=torch.uint8, device="cuda")
    qkv = dev_bf16(bf16(rng, T, hq + 2 * hk, d))
    room = torch.zeros(T * ((hq + 2 * hk) * d + 4) + 4, dtype=torch.bfloat16, device="cuda")
    odd = room[4:].as_strided((T, hq + 2 * hk, d), ((hq + 2 * hk) * d + 4, d, 1))
    odd.copy_(qkv)
    turns, slots = fq.rope_turns(d, device="cuda")[0], torch.randperm(64, device="cuda")[:T]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    got = []
    for x in (qkv, odd):
        k, v = kv.clone(), kv.clone()
        ks, vs = torch.zeros((hk, 64), device="cuda"), torch.zeros((hk, 64), device="cuda")
        out = fq.fp8_kv_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], slots, k, v, ks, vs, 0, 3, positions=pos, turns=turns)
        got.append((out.clone(), k, v, ks, vs))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("T", [16 * 592, 16 * 592 + 1, 3 * 592 - 1, 593])
def test_append_blocks_of_all_sizes(T):
    """Token counts around whole waves of blocks: every token's row is the quantizer's."""
    rng = np.random.default_rng(T)
    x = bf16(rng, T, 1, 128)
    P = -(-T // 16)
    k = torch.zeros((P, 16, 1, 128), dtype=torch.uint8, device="cuda")
    v, s1, s2 = k.clone(), torch.zeros((1, P * 16), device="cuda"), torch.zeros((1, P * 16), device="cuda")
    fq.fp8_kv_append(None, dev_bf16(x), dev_bf16(x), torch.arange(T, device="cuda"), k, v, s1, s2, 0, 3)
    c, s = fq.fp8_quantize(dev_bf16(x).view(T, 128), 0, fq.GROUP_1x128)
    torch.cuda.synchronize()
    assert torch.equal(k.view(-1, 128)[:T], c) and torch.equal(k, v)
    assert torch.equal(s1[0, :T], s.view(-1)) and torch.equal(s1, s2)


def test_append_in_place_equals_apart():
    a = append_case(4, 100, 8, 2, 128, 16, 0, 3, 128, False, True, inplace=True)
    b = append_case(4, 100, 8, 2, 128, 16, 0, 3, 128, False, True)
    assert np.array_equal(a["k"], b["k"]) and np.array_equal(a["v"], b["v"])


def test_append_far_positions_and_gain():
    append_case(5, 64, 4, 2, 128, 16, 0, 3, 128, False, False, positions=(1 << 30) + np.arange(64) * 7919, gain=1.25)
    append_case(6, 64, 4, 2, 64, 16, 0, 3, 64, True, False, positions=2 ** 31 - 1 - np.arange(64))
    append_case(7, 8, 4, 2, 64, 16, 0, 3, 64, False, False, positions=np.zeros(8))


def test_append_codes_equal_the_quantizer(orc):
    """V, and K without norm and rotation: the same bits as fp8_quantize's 1x128 groups; special rows too."""
    rng = np.random.default_rng(8)
    T, H, D, size = 96, 4, 128, 16
    x = bf16(rng, T, H, D)
    x[0, 0] = 0
    x[1, 1, 5] = 0x7FC0
    x[2, 2, 9] = 0x7F80
    x[3, 3] = 0x0003                                     # subnormals only
    x[4, 0, :] = 0x8000
    x[5, 1, 3] = 0x7F7F
    P = T // size
    for fmt in (0, 1):
        k = torch.zeros((P, size, H, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros_like(k)
        ks = torch.zeros((H, P * size), device="cuda")
        vs = torch.zeros_like(ks)
        fq.fp8_kv_append(None, dev_bf16(x), dev_bf16(x), dev(np.arange(T, dtype=np.int64)), k, v, ks, vs, fmt, 3)
        torch.cuda.synchronize()
        c, s = orc.quantize(x.reshape(T, H * D), fmt, orc.GROUP_1x128)
        for codes, scales in ((k, ks), (v, vs)):
            assert_f32_bits_equal(host(scales), s)
            assert_codes_equal(host(codes).reshape(T, H * D), c, fmt)


def test_append_given_scales_saturate_and_vanish():
    rng = np.random.default_rng(9)
    T, H, D, size = 16, 3, 64, 16
    x = bf16(rng, T, H, D, std=100.0)
    x[0, 0, 0], x[0, 0, 1] = 0x7F80, 0xFF80
    x[0, 1, 0] = 0x7F7F
    for fmt in (0, 1):
        s = np.array([1e-30, 1e-3, 0.0], np.float32)
        k = torch.zeros((1, size, H, D), dtype=torch.uint8, device="cuda")
        v = torch.zeros_like(k)
        fq.fp8_kv_append(None, dev_bf16(x), dev_bf16(x), dev(np.arange(T, dtype=np.int64)), k, v, dev(s), dev(s), fmt, 1)
        torch.cuda.synchronize()
        want = np.clip(ref.bf16_to_f64(x[:, :2]) / s[:2, None].astype(np.float64), -ref.FMAX[fmt], ref.FMAX[fmt])
        got = ref.decode_table(fmt)[host(v)[0]]
        assert (np.abs(got[:, :2] - want) <= np.abs(want) * ref.REL[fmt] * 1.001 + ref.SUB[fmt]).all()
        assert np.array_equal(host(v)[0][:, 2], np.where(x[:, 2] & 0x8000, 0x80, 0).astype(np.uint8))
        assert torch.equal(k, v)


def test_append_slots_beyond_the_cache_are_left_out():
    rng = np.random.default_rng(10)
    T, H, D = 8, 2, 64
    k = torch.full((2, 4, H, D), 9, dtype=torch.uint8, device="cuda")
    v = k.clone()
    s = dev(np.ones(1, np.float32))
    x = dev_bf16(bf16(rng, T, H, D))
    slots = np.array([0, 8, -1, 2 ** 40, 3, -2 ** 62, 2 ** 31, 2 ** 32 + 1], np.int64)
    fq.fp8_kv_append(None, x, x, dev(slots), k, v, s, s, 0, 0)
    torch.cuda.synchronize()
    assert fq.device_status() == 4
    touched = (host(k).reshape(8, -1) != 9).any(1)
    assert touched.tolist() == [True, False, False, True, False, False, False, False]


def test_append_nothing():
    k = torch.zeros((1, 16, 2, 64), dtype=torch.uint8, device="cuda")
    s = torch.ones(1, device="cuda")
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    fq.fp8_kv_append(None, x, x, torch.empty(0, dtype=torch.int64, device="cuda"), k, k.clone(), s, s, 0, 0)
    torch.cuda.synchronize()
    assert (k == 0).all()


# ------------------------------------------------------------------ pages

def device_pages(table, lens, free, count):
    return dev(table), dev(lens), dev(free), dev(np.array([count], np.int32))


def check_step(plain, state, added, max_tokens, size, inplace=True):
    want = plain.step(added, max_tokens)
    t, l, f, c = state
    kw = {} if inplace else {"lens_out": torch.empty_like(l), "free_count_out": torch.empty_like(c)}
    got = fq.fp8_kv_pages_update(t, l, dev(np.asarray(added, np.int32)), f, c, size, max_tokens, **kw)
    torch.cuda.synchronize()
    for name, g, w in zip(("slots", "positions", "offsets", "served"), got, want):
        assert np.array_equal(host(g), w), name
    assert np.array_equal(host(got[4]), plain.lens)
    assert int(host(got[5])[0]) == plain.count
    assert np.array_equal(host(t), plain.table)
    assert np.array_equal(host(f)[:plain.count], plain.free[:plain.count])
    if not inplace:
        l.copy_(got[4])
        c.copy_(got[5])
    return got


@pytest.mark.parametrize("B,width,size,pages", [(1, 4, 16, 6), (7, 6, 5, 30), (40, 20, 16, 500), (300, 9, 1, 2000),
                                                (1500, 4, 8, 4000)])
@pytest.mark.parametrize("inplace", [True, False])
def test_pages_random_steps(B, width, size, pages, inplace):
    """Many steps: prompts, single tokens, ends, rows that overflow, the free list running out."""
    rng = np.random.default_rng(B)
    free = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    lens = np.zeros(B, np.int32)
    plain = ref.Pages(table, lens, free, pages, size)
    state = device_pages(table, lens, free, pages)
    for step in range(12):
        kind = rng.random(B)
        added = np.where(kind < 0.15, -1, np.where(kind < 0.5, 1, np.where(kind < 0.6, 0, rng.integers(0, 2 * size + 3, B))))
        check_step(plain, state, added, int(np.maximum(added, 0).sum()) + (step % 3) * 5, size, inplace)
    held = [p for b in range(B) for p in plain.table[b, :-(-plain.lens[b] // size)]]
    assert sorted(held + list(plain.free[:plain.count])) == list(range(pages))   # no page lost or given twice


@pytest.mark.parametrize("n", [4095, 4096, 4097, 20000])
def test_pages_one_and_two_launches(n):
    for B in (1, 3, 1024, 1025):
        size, width = 16, -(-n // 16) + 1
        pages = -(-n // size) + B
        free = np.arange(pages, dtype=np.int32)[::-1].copy()
        table, lens = np.zeros((B, width), np.int32), np.zeros(B, np.int32)
        added = np.zeros(B, np.int64)
        added[0] = n - (B - 1)
        added[1:] = 1
        plain = ref.Pages(table, lens, free, pages, size)
        check_step(plain, device_pages(table, lens, free, pages), added, n, size)


def test_pages_tokens_beyond_max_tokens_are_not_served():
    free = np.arange(20, dtype=np.int32)
    table, lens = np.zeros((3, 6), np.int32), np.array([3, 0, 5], np.int32)
    table[0, 0], table[2, :2] = 18, [17, 19]
    plain = ref.Pages(table, lens, free[:17].copy(), 17, 4)
    plain.free = np.concatenate([free[:17], np.zeros(3, np.int32)])
    state = device_pages(table, lens, plain.free, 17)
    got = check_step(plain, state, [4, 5, 1], 8, 4)
    assert host(got[3]).tolist() == [1, 0, 0]


@pytest.mark.parametrize("B", [3, 1300])
def test_pages_of_a_request_that_is_not_served_stay_free(B):
    """A request without enough pages, then one that needs none: what is on the list stays there."""
    free = np.arange(20, dtype=np.int32)
    table, lens = np.zeros((B, 6), np.int32), np.zeros(B, np.int32)
    table[0, 0], table[B - 1, 0], lens[0], lens[B - 1] = 18, 19, 3, 1
    plain = ref.Pages(table, lens, free, 2, 4)
    added = np.zeros(B, np.int32)
    added[0], added[B - 1] = 20, 2
    got = check_step(plain, device_pages(table, lens, free, 2), added, 22, 4)
    assert int(host(got[5])[0]) == 2 and host(got[3])[[0, B - 1]].tolist() == [0, 1]


def test_pages_nothing_and_empty():
    free, count = torch.arange(4, dtype=torch.int32, device="cuda"), torch.tensor([4], dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = fq.fp8_kv_pages_update(torch.empty((0, 3), dtype=torch.int32, device="cuda"), e, e, free, count, 16, 5)
    torch.cuda.synchronize()
    assert host(got[0]).tolist() == [-1] * 5 and host(got[2]).tolist() == [0] and int(host(count)[0]) == 4
    lens = torch.tensor([7], dtype=torch.int32, device="cuda")
    got = fq.fp8_kv_pages_update(torch.tensor([[2]], dtype=torch.int32, device="cuda"), lens, torch.zeros_like(lens),
                                 free, count, 16, 0)
    torch.cuda.synchronize()
    assert host(got[3]).tolist() == [1] and int(host(lens)[0]) == 7


def test_pages_many_requests_without_tokens():
    B = 1500
    free, count = torch.arange(2000, dtype=torch.int32, device="cuda"), torch.tensor([500], dtype=torch.int32, device="cuda")
    table = torch.arange(500, 2000, dtype=torch.int32, device="cuda").view(B, 1)
    lens, added = torch.full((B,), 3, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    added[7::100] = -1
    got = fq.fp8_kv_pages_update(table, lens, added, free, count, 16, 0)
    torch.cuda.synchronize()
    assert got[0].numel() == 0 and int(host(count)[0]) == 515
    assert host(free)[500:515].tolist() == list(range(507, 2000, 100))
    assert host(lens).tolist() == [0 if b % 100 == 7 else 3 for b in range(B)]


def test_pages_bad_counts_are_clipped_and_reported():
    for lens, count, added in (([40], 4, [-1]), ([-3], 4, [1]), ([0], 9, [1]), ([0], -2, [1]), ([16, 16], 4, [-1, -1])):
        B = len(lens)
        free = torch.arange(4, dtype=torch.int32, device="cuda")
        c = torch.tensor([count], dtype=torch.int32, device="cuda")
        guard = torch.full((B, 4), 1, dtype=torch.int32, device="cuda")
        table = guard[:, :2].contiguous()
        got = fq.fp8_kv_pages_update(table, dev(np.array(lens, np.int32)), dev(np.array(added, np.int32)), free, c, 16, 4)
        torch.cuda.synchronize()
        assert fq.device_status() == 4, (lens, count)
        assert 0 <= int(host(c)[0]) <= 4
        assert (host(got[0]) < 4 * 16).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("gran", [1, 3])
def test_serving_steps_together(gran):
    """Prompts, then decoding steps as a serving program runs them: pages, append, attention, with
    requests that end and begin, against attention over each request's own tokens in 64 bits."""
    rng = np.random.default_rng(3)
    B, hq, hk, d, size, P, width = 5, 8, 2, 64, 16, 40, 12
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    turns, _ = fq.rope_turns(d, 10000.0, device="cuda")
    wq, wk = bf16(rng, d), bf16(rng, d)
    kc, vc = (torch.full((P, size, hk, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = np.full(fq.kv_page_scale_shape(P, size, hk, gran), 0.02, np.float32)
    ks, vs = dev(sc), dev(sc)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = torch.arange(P, dtype=torch.int32, device="cuda")
    count = torch.tensor([P], dtype=torch.int32, device="cuda")
    steps = [[30, 1, 0, 17, 64], [1, 1, 5, 1, 1], [1, 1, 1, -1, 1], [1, 1, 1, 40, -1], [1, 1, 1, 1, 33]]
    history = [[] for _ in range(B)]                 # (k, v) rows of each request, before quantization
    for added in steps:
        T = sum(max(0, a) for a in added)
        pad = 3
        qkv = bf16(rng, T + pad, hq + 2 * hk, d)
        x = dev_bf16(qkv)
        slots, pos, offsets, served, _, _ = fq.fp8_kv_pages_update(table, lens, dev(np.array(added, np.int32)), free, count,
                                                                   size, T + pad)
        q = fq.fp8_kv_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], slots, kc, vc, ks, vs, 0, gran, positions=pos,
                             turns=turns, q_weight=dev_bf16(wq), k_weight=dev_bf16(wk))
        last = (offsets[1:] - 1).clamp(min=0).long()
        out, _ = fq.fp8_attention_paged(q[last].contiguous(), kc, vc, ks, vs, table, lens, 0, gran)
        torch.cuda.synchronize()
        assert host(served).tolist() == [int(a >= 0) for a in added]
        n, tab = host(lens), host(table)
        for b in range(B):
            if added[b] < 0:
                history[b] = []
            at = int(host(offsets)[b])
            p = np.arange(len(history[b]), len(history[b]) + max(0, added[b]))
            rows = qkv[at:at + max(0, added[b])]
            k = ref.rotate(ref.norm(ref.bf16_to_f64(rows[:, hq:hq + hk]), ref.bf16_to_f64(wk), 1e-6), p, freq, False)[0]
            history[b] += list(zip(k, ref.bf16_to_f64(rows[:, hq + hk:])))
            assert n[b] == len(history[b])
            # the codes stand for the request's own tokens: half an E4M3 step, and fp32 steps before it
            for t, (k1, v1) in enumerate(history[b]):
                slot = tab[b, t // size] * size + t % size
                for cache, s, want in ((kc, ks, k1), (vc, vs, v1)):
                    sl = host(s)[:, slot] if gran == 3 else host(s)
                    got = ref.decode_table(0)[host(cache).reshape(P * size, hk, d)[slot]]
                    y = np.clip(want / sl[:, None], -448, 448)
                    assert (np.abs(got - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10) + 448 * 2.0 ** -17).all()
        want, _, tol, _ = ref.attention(ref.bf16_to_f64(host(q))[host(last)], host(kc), host(vc), host(ks), host(vs), tab, n, 0,
                                        gran, d ** -0.5, 0, 0)
        assert (np.abs(ref.bf16_to_f64(host(out)) - want) <= tol).all()


def test_decoding_step_in_a_graph():
    """One decoding step captured once and replayed: lengths, tables and caches advance on the device."""
    rng = np.random.default_rng(4)
    B, hq, hk, d, size, P, width = 3, 8, 2, 64, 4, 30, 10
    turns, _ = fq.rope_turns(d, device="cuda")
    kc, vc = (torch.zeros((P, size, hk, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((hk, P * size), device="cuda") for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = torch.arange(P, dtype=torch.int32, device="cuda")
    count = torch.tensor([P], dtype=torch.int32, device="cuda")
    added = torch.tensor([1, 1, 0], dtype=torch.int32, device="cuda")
    x = torch.zeros((B, hq + 2 * hk, d), dtype=torch.bfloat16, device="cuda")

    def step():
        slots, pos, *_ = fq.fp8_kv_pages_update(table, lens, added, free, count, size, B)
        q = fq.fp8_kv_append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], slots, kc, vc, ks, vs, 0, 3, positions=pos, turns=turns)
        return q, fq.fp8_attention_paged(q, kc, vc, ks, vs, table, lens, 0, 3)[0]
    warm = (lens.clone(), count.clone())
    step()
    lens.copy_(warm[0])
    count.copy_(warm[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, out = step()
    for i in range(20):
        x.copy_(dev_bf16(bf16(rng, B, hq + 2 * hk, d)))
        g.replay()
        torch.cuda.synchronize()
        n = host(lens)
        assert n.tolist() == [i + 1, i + 1, 0]
        want, _, tol, _ = ref.attention(ref.bf16_to_f64(host(q)), host(kc), host(vc), host(ks), host(vs), host(table), n, 0, 3,
                                        d ** -0.5, 0, 0)
        assert (np.abs(ref.bf16_to_f64(host(out)) - want) <= tol).all()
    assert int(host(count)[0]) == P - 2 * 5
