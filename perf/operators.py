"""Measured cases of the paged FP8 KV-cache operators.

Three operators serve one decoding or prefill step of a model whose KV cache is kept as FP8
codes in pages:

  pages      block tables, slots and positions from the requests' lengths (fp8_kv_pages_update)
  append     per-head RMS norm and rotary positions of q and k, k and v quantized into their
             slots (fp8_kv_append)
  attention  attention of one new token per request over its pages (fp8_attention_paged)

listed() and draw() give cases, prepare() a case's inputs on the GPU, run() one pass through
the operator, exact() the same outputs from the definition in 64 bits and work() the bytes and
operations a pass cannot do without.  With `own` false run() computes the plain form with
elementary torch operations in fp32; with `own` true it calls the library.
"""
import math

import torch

own = False

E4M3, E5M2 = 0, 1
PER_TENSOR, PER_HEAD, PER_HEAD_TOK128, PER_TOKEN = 0, 1, 2, 3
FMAX = (448.0, 57344.0)
FLOAT8 = (torch.float8_e4m3fn, torch.float8_e5m2)
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _attention(name, batch, shortest, longest, hq, hk, d, page, fmt, gran, window=0, sinks=0, empty=0):
    return {"name": name, "op": "attention", "batch": batch, "shortest": shortest, "longest": longest, "hq": hq,
            "hk": hk, "d": d, "page": page, "fmt": fmt, "gran": gran, "window": window, "sinks": sinks, "empty": empty}


def _append(name, tokens, hq, hk, d, rot, interleaved, norm, page, fmt, gran, far, stretch, padded=0):
    return {"name": name, "op": "append", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "interleaved": interleaved, "norm": norm, "page": page, "fmt": fmt, "gran": gran, "far": far,
            "stretch": stretch, "padded": padded}


def _pages(name, batch, old, new, page, finished, spare):
    return {"name": name, "op": "pages", "batch": batch, "old": old, "new": new, "page": page, "finished": finished,
            "spare": spare}


def listed():
    return [
        # one request that has just begun: the latency of a call
        _attention("attention 1 x 33", 1, 33, 33, 32, 8, 128, 16, E4M3, PER_HEAD),
        # a decoding batch of ordinary, ragged lengths on the 8B head layout, two rows not in use
        _attention("attention 16 ragged to 4096", 16, 130, 4096, 32, 8, 128, 16, E4M3, PER_HEAD, empty=2),
        # one long context on the 70B head layout (the 131072-token cache), a scale per token and head
        _attention("attention 1 x 131072", 1, 131072, 131072, 64, 8, 128, 64, E4M3, PER_TOKEN),
        # a large batch, E5M2 with one scale per tensor
        _attention("attention 64 ragged to 8192", 64, 2000, 8192, 64, 8, 128, 32, E5M2, PER_TENSOR),
        # long contexts read through a window and a few first tokens; small heads
        _attention("attention window 4096 + 4", 8, 20000, 131072, 64, 8, 64, 16, E4M3, PER_HEAD, window=4096, sinks=4),
        # one key-value head for all queries, wide head, odd page size, a scale per 128 tokens
        _attention("attention one kv head", 7, 999, 30011, 16, 1, 256, 24, E4M3, PER_HEAD_TOK128),
        # one decoding step of a batch: the latency of a call
        _append("append 32 tokens", 32, 32, 8, 128, 128, False, True, 16, E4M3, PER_HEAD, 131072, 1.0),
        # an odd chunk: part of the head rotated, neighbours paired, no norm, some rows padding
        _append("append 777 tokens", 777, 14, 2, 96, 32, True, False, 24, E5M2, PER_TENSOR, 8192, 1.0, padded=9),
        # a prefill chunk on the 8B head layout, a scale per token and head
        _append("append 8192 tokens", 8192, 32, 8, 128, 128, False, True, 16, E4M3, PER_TOKEN, 8192, 1.0),
        # a prefill on the 70B head layout far into a context with stretched positions
        _append("append 16384 tokens", 16384, 64, 8, 128, 128, False, False, 64, E4M3, PER_HEAD, 1000000, 8.0),
        # one decoding step: a token per request, some requests end
        _pages("pages 256 decoding", 256, 8192, 1, 16, 8, 512),
        # prompts of many requests at once
        _pages("pages 96 prompts", 96, 0, 4096, 16, 0, 512),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "append", "append", "pages"))
    page = rng.choice((8, 16, 16, 24, 32, 64, 128))
    if op == "attention":
        hk = rng.choice((1, 2, 4, 5, 8, 8, 8, 16))
        group = rng.choice((1, 2, 3, 4, 6, 8, 8, 12, 16))
        d = rng.choice((64, 80, 96, 128, 128, 128, 192, 256))
        longest = _spread(rng, 1, min(131072, (1 << 28) // (hk * d)))
        most = max(1, min(256, (1 << 28) // (longest * hk * d)))
        batch = _spread(rng, 1, most)
        window = rng.choice((0, 0, 0, _spread(rng, 1, longest)))
        return {k: v for k, v in _attention("", batch, rng.randint(1, longest), longest, hk * group, hk, d, page,
                                            rng.choice((E4M3, E4M3, E5M2)),
                                            rng.choice((PER_TENSOR, PER_HEAD, PER_HEAD_TOK128, PER_TOKEN)), window,
                                            rng.choice((0, 1, 4, 17)) if window else 0,
                                            rng.choice((0, 0, batch // 3))).items() if k != "name"}
    if op == "append":
        hk = rng.choice((1, 2, 4, 8, 8))
        hq = hk * rng.choice((1, 3, 4, 7, 8))
        d = rng.choice((64, 96, 128, 128, 256))
        rot = rng.choice((d, d, d // 2, d // 4 // 8 * 8, 0))
        tokens = _spread(rng, 1, max(1, min(16384, 16384 * 80 * 128 // ((hq + 2 * hk) * d))))
        return {k: v for k, v in _append("", tokens, hq, hk, d, rot, rng.random() < 0.5, rng.random() < 0.5, page,
                                         rng.choice((E4M3, E4M3, E5M2)),
                                         rng.choice((PER_TENSOR, PER_HEAD, PER_TOKEN)), _spread(rng, 100, 1000000),
                                         rng.choice((1.0, 4.0, 8.0)), rng.choice((0, 0, tokens // 5))).items()
                if k != "name"}
    batch = _spread(rng, 1, 1024)
    return {k: v for k, v in _pages("", batch, rng.choice((0, _spread(rng, 1, 8192))),
                                    _spread(rng, 1, max(1, min(8192, 262144 // batch))), page,
                                    rng.choice((0, batch // 7)), rng.choice((-5, 0, 100))).items() if k != "name"}


# ------------------------------------------------------------------ sizes that follow from a case

def _lengths(c):
    """The requests' lengths, in an order that prepare() shuffles: evenly spread, the last ones empty."""
    n = c["batch"] - c["empty"]
    step = (c["longest"] - c["shortest"]) / max(1, n - 1)
    return [int(c["longest"] - round(step * i)) for i in range(n)] + [0] * c["empty"]


def _visible(c, length):
    if c["window"] == 0 or length <= c["window"]:
        return length
    return min(length, c["window"] + c["sinks"])


def _page_lengths(c):
    """(tokens held, tokens added or -1 for a request that ends) of each request, before shuffling."""
    b = c["batch"]
    held = [c["old"] - (c["old"] * i) // (2 * b) for i in range(b)]
    added = [max(1, c["new"] - (c["new"] * i) // (2 * b)) for i in range(b)]
    for i in range(c["finished"]):
        added[(i * b) // c["finished"]] = -1
    return held, added


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    c = case
    if c["op"] == "attention":
        seen = sum(_visible(c, n) for n in _lengths(c))
        scales = {PER_TENSOR: 2, PER_HEAD: 2 * c["hk"], PER_HEAD_TOK128: 2 * c["hk"] * _cdiv(seen, 128),
                  PER_TOKEN: 2 * c["hk"] * seen}[c["gran"]]
        rows = c["batch"] * c["hq"]
        tables = sum(_cdiv(_visible(c, n), c["page"]) for n in _lengths(c)) + c["batch"]
        return {"bytes": 2 * seen * c["hk"] * c["d"] + 4 * scales + 4 * rows * c["d"] + 4 * rows + 4 * tables,
                "flops": 4 * seen * c["hq"] * c["d"]}
    if c["op"] == "append":
        used = c["tokens"] - c["padded"]
        read = 2 * (used * 2 * c["hk"] + c["tokens"] * c["hq"]) * c["d"] + 12 * c["tokens"] + 4 * c["rot"]
        written = 2 * c["tokens"] * c["hq"] * c["d"] + 2 * used * c["hk"] * c["d"]
        scales = 8 * used * c["hk"] if c["gran"] == PER_TOKEN else 0
        return {"bytes": read + written + scales,
                "flops": (c["tokens"] * c["hq"] + used * c["hk"]) * (3 * c["rot"] + (4 * c["d"] if c["norm"] else 0))
                + 2 * used * c["hk"] * c["d"]}
    held, added = _page_lengths(c)
    tokens = sum(max(0, n) for n in added)
    moved = sum(_cdiv(h + max(0, n), c["page"]) - _cdiv(h, c["page"]) if n >= 0 else _cdiv(h, c["page"])
                for h, n in zip(held, added))
    return {"bytes": 12 * tokens + 8 * moved + 20 * c["batch"], "flops": 4 * tokens}


# ------------------------------------------------------------------ inputs

def _frequencies(rot, stretch):
    """Radians per position of each rotated pair, base 500000, positions stretched for long contexts."""
    return [500000.0 ** (-2.0 * i / rot) / stretch for i in range(rot // 2)]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(torch.bfloat16)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=dev)

    if c["op"] == "pages":
        held, added = _page_lengths(c)
        order = shuffled(c["batch"])
        held = torch.tensor(held, dtype=torch.int32, device=dev)[order]
        added = torch.tensor(added, dtype=torch.int32, device=dev)[order]
        widest = _cdiv(int((held + added.clamp(min=0)).max()), c["page"]) + 1
        pages_held = (held + c["page"] - 1) // c["page"]
        need = ((held + added.clamp(min=0) + c["page"] - 1) // c["page"] - pages_held)
        n_held, n_need = int(pages_held.sum()), int(torch.where(added >= 0, need, 0).sum())
        n_free = max(0, n_need + c["spare"])
        ids = shuffled(n_held + n_free).to(torch.int32)
        first = torch.cumsum(pages_held, 0) - pages_held
        col = torch.arange(widest, device=dev)
        table = ids[(first[:, None] + col).clamp(max=max(0, ids.numel() - 1))] if ids.numel() else \
            torch.zeros((c["batch"], widest), dtype=torch.int32, device=dev)
        table = torch.where(col < pages_held[:, None], table, -1).to(torch.int32).contiguous()
        free = torch.full((n_held + n_free,), -1, dtype=torch.int32, device=dev)
        free[:n_free] = ids[n_held:]
        tokens = int(added.clamp(min=0).sum())
        s = {"case": c, "table": table, "lens": held, "added": added, "free": free,
             "free_count": torch.tensor([n_free], dtype=torch.int32, device=dev), "tokens": tokens}
        return _with_outputs(s)

    hk, hq, d, page = c["hk"], c["hq"], c["d"], c["page"]
    if c["op"] == "append":
        t = c["tokens"]
        # the projection's output row holds q, k and v side by side
        qkv = normal(t, hq + 2 * hk, d)
        qkv[:, hq:hq + hk] *= 1.5
        n_pages = _cdiv(t, page) + 3
        slots = shuffled(n_pages * page)[:t].to(torch.int64)
        start = max(0, c["far"] - t)
        positions = torch.arange(start, start + t, dtype=torch.int32, device=dev)
        if c["padded"]:
            slots[t - c["padded"]:] = -1
        cache = [(torch.randn((n_pages, page, hk, d), generator=gen, device=dev) * 40).to(FLOAT8[c["fmt"]]).view(torch.uint8)
                 for _ in range(2)]
        if c["gran"] == PER_TOKEN:
            scales = [torch.rand((hk, n_pages * page), generator=gen, device=dev) + 0.01 for _ in range(2)]
        else:
            n = hk if c["gran"] == PER_HEAD else 1
            scales = [(torch.rand(n, generator=gen, device=dev) + 0.5) * (8.0 / FMAX[c["fmt"]]) for _ in range(2)]
        weights = [normal(d, std=0.1) + 1.0 for _ in range(2)] if c["norm"] else [None, None]
        s = {"case": c, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:], "positions": positions,
             "slots": slots, "k_cache": cache[0], "v_cache": cache[1], "k_scales": scales[0], "v_scales": scales[1],
             "q_weight": weights[0], "k_weight": weights[1],
             "freq": torch.tensor(_frequencies(c["rot"], c["stretch"]), dtype=torch.float64, device=dev)}
        return _with_outputs(s)

    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)[shuffled(c["batch"])]
    held = (lens + page - 1) // page
    widest = max(1, _cdiv(c["longest"], page))
    n_pages = int(held.sum()) + 3
    ids = shuffled(n_pages).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(widest, device=dev)
    table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=n_pages - 1)], -1).to(torch.int32)
    cache, scales = [], []
    for _ in range(2):
        gain = torch.rand(hk, 1, generator=gen, device=dev) * 3 + 0.5
        x = torch.randn((n_pages, page, hk, d), generator=gen, device=dev)
        x *= gain
        if c["gran"] == PER_TENSOR:
            s = (gain.max() * 5.5 / FMAX[c["fmt"]]).reshape(1)
            x /= s
        elif c["gran"] == PER_HEAD:
            s = (gain * 5.5 / FMAX[c["fmt"]]).reshape(hk)
            x /= s[:, None]
        elif c["gran"] == PER_HEAD_TOK128:
            blocks = _cdiv(n_pages * page, 128)
            s = (torch.rand((blocks, hk), generator=gen, device=dev) + 0.5) * gain[:, 0] * (5.5 / FMAX[c["fmt"]])
            x.view(n_pages * page, hk, d).div_(s.repeat_interleave(128, 0)[:n_pages * page, :, None])
        else:
            s = (x.abs().amax(-1) / FMAX[c["fmt"]])
            x /= s[..., None]
            s = s.reshape(n_pages * page, hk).t().contiguous()
        cache.append(x.clamp_(-FMAX[c["fmt"]], FMAX[c["fmt"]]).to(FLOAT8[c["fmt"]]).view(torch.uint8))
        scales.append(s.float().contiguous())
        del x
    # what an earlier request left behind a request's last token may be any code
    tail = (lens % page != 0).nonzero()[:, 0]
    last = table[tail, (lens[tail] // page).long()].long()
    off = torch.arange(page, device=dev) >= (lens[tail] % page)[:, None]
    for x in cache:
        x[last] = torch.where(off[:, :, None, None], torch.tensor(0x7F, dtype=torch.uint8, device=dev), x[last])
    q = normal(c["batch"], hq, d)
    return _with_outputs({"case": c, "q": q, "k_cache": cache[0], "v_cache": cache[1], "k_scales": scales[0],
                          "v_scales": scales[1], "table": table.contiguous(), "lens": lens, "scale": d ** -0.5})


def _with_outputs(s):
    """The buffers a user's program keeps over its steps, and the rotation table in the library's form."""
    c = s["case"]
    dev = "cuda"
    if c["op"] == "pages":
        s["out_lens"] = torch.empty_like(s["lens"])
        s["out_count"] = torch.empty_like(s["free_count"])
        s["out_slots"] = torch.empty(s["tokens"], dtype=torch.int64, device=dev)
        s["out_positions"] = torch.empty(s["tokens"], dtype=torch.int32, device=dev)
        s["out_offsets"] = torch.empty(c["batch"] + 1, dtype=torch.int32, device=dev)
        s["out_served"] = torch.empty(c["batch"], dtype=torch.int32, device=dev)
    elif c["op"] == "append":
        s["q_out"] = torch.empty((c["tokens"], c["hq"], c["d"]), dtype=torch.bfloat16, device=dev)
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in s["freq"].tolist()]
        s["turns"] = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=dev)
    else:
        s["out"] = torch.empty((c["batch"], c["hq"], c["d"]), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((c["batch"], c["hq"]), dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "append": _plain_append, "pages": _plain_pages}[state["case"]["op"]](state)


def _run_own(s):
    import fp8_quantization_amax_b200 as fq
    c = s["case"]
    if c["op"] == "pages":
        fq.fp8_kv_pages_update(s["table"], s["lens"], s["added"], s["free"], s["free_count"], c["page"],
                               slots=s["out_slots"], positions=s["out_positions"], offsets=s["out_offsets"],
                               served=s["out_served"], lens_out=s["out_lens"], free_count_out=s["out_count"])
        return _pages_outputs(s)
    if c["op"] == "append":
        fq.fp8_kv_append(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                         c["fmt"], c["gran"], positions=s["positions"], turns=s["turns"] if c["rot"] else None,
                         interleaved=c["interleaved"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                         q_out=s["q_out"])
        return _append_outputs(s, s["q_out"])
    return fq.fp8_attention_paged(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                  s["lens"], c["fmt"], c["gran"], scale=s["scale"], window=c["window"],
                                  sinks=c["sinks"], out=s["out"], lse=s["lse"])


def _pages_outputs(s):
    return {"table": s["table"], "lens": s["out_lens"], "count": s["out_count"], "slots": s["out_slots"],
            "positions": s["out_positions"], "offsets": s["out_offsets"], "served": s["out_served"], "free": s["free"]}


def _append_outputs(s, q_out):
    kind = FLOAT8[s["case"]["fmt"]]
    out = {"q": q_out, "k": s["k_cache"].view(kind), "v": s["v_cache"].view(kind)}
    if s["case"]["gran"] == PER_TOKEN:
        out["k_scales"], out["v_scales"] = s["k_scales"], s["v_scales"]
    return out


def _plain_pages(s):
    """Requests that end give their pages back first; the others then take pages from the top of
    the free list in order.  A request whose pages or row do not suffice is not served."""
    page, table = s["case"]["page"], s["table"]
    lens, added = s["lens"].long(), s["added"].long()
    ends = added < 0
    new = added.clamp(min=0)
    held = (lens + page - 1) // page
    back = torch.where(ends, held, 0)
    n_back = back.sum()
    col = torch.arange(table.shape[1], device=table.device)
    given = torch.where(ends[:, None] & (col < held[:, None]),
                        s["free_count"] + torch.cumsum(back, 0)[:, None] - back[:, None] + col, s["free"].numel())
    s["free"].copy_(torch.cat((s["free"], s["free"].new_zeros(1))).scatter(0, given.reshape(-1), table.reshape(-1))[:-1])
    total = s["free_count"].long() + n_back
    need = torch.where(ends, 0, (lens + new + page - 1) // page - held)
    fits = (~ends) & (lens + new <= table.shape[1] * page)
    need = torch.where(fits, need, 0)
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= total))
    from_ = upto - need
    take = served[:, None] & (col >= held[:, None]) & (col < (held + need)[:, None])
    at = (total - 1 - from_[:, None] - (col - held[:, None])).clamp(min=0, max=max(0, s["free"].numel() - 1))
    if s["free"].numel():
        table.copy_(torch.where(take, s["free"][at], table))
    used = torch.where(served, upto, 0).max()
    s["out_count"].copy_(total - used)
    s["out_lens"].copy_(torch.where(ends, 0, torch.where(served, lens + new, lens)))
    s["out_served"].copy_(served)
    offsets = torch.cat((new.new_zeros(1), torch.cumsum(new, 0)))
    s["out_offsets"].copy_(offsets)
    who = torch.repeat_interleave(torch.arange(new.numel(), device=table.device), new, output_size=s["tokens"])
    pos = lens[who] + torch.arange(s["tokens"], device=table.device) - offsets[who]
    at = (pos // page).clamp(max=table.shape[1] - 1)
    s["out_positions"].copy_(pos)
    s["out_slots"].copy_(torch.where(served[who], table[who, at].long() * page + pos % page, -1))
    return _pages_outputs(s)


def _plain_append(s):
    c = s["case"]
    rot, fmax, kind = c["rot"], FMAX[c["fmt"]], FLOAT8[c["fmt"]]

    def norm(x, w):
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    def rotate(x):
        if rot == 0:
            return x
        angle = s["positions"].double()[:, None] * s["freq"]
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        out = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        return out

    q = rotate(norm(s["q"].float(), s["q_weight"])).to(torch.bfloat16)
    k = rotate(norm(s["k"].float(), s["k_weight"]))
    v = s["v"].float()
    used = c["tokens"] - c["padded"]
    slots = s["slots"][:used]
    for x, cache, scales in ((k, s["k_cache"], s["k_scales"]), (v, s["v_cache"], s["v_scales"])):
        x = x[:used]
        if c["gran"] == PER_TOKEN:
            by = x.abs().amax(-1) / fmax
            scales[:, slots] = by.t()
        else:
            by = scales.expand(x.shape[1])[None]
        y = torch.where(by[..., None] > 0, x / by[..., None], 0)
        codes = y.clamp(-fmax, fmax).to(kind).view(torch.uint8)
        cache.view(-1, c["hk"], c["d"])[slots] = codes
    return _append_outputs(s, q)


def _plain_attention(s):
    c = s["case"]
    b, hk, group, d, page = c["batch"], c["hk"], c["hq"] // c["hk"], c["d"], c["page"]
    table = s["table"].clamp(min=0).long()
    n = table.shape[1] * page
    slots = (table[:, :, None] * page + torch.arange(page, device=table.device)).reshape(b, n)
    pos = torch.arange(n, device=table.device)
    seen = pos < s["lens"][:, None]
    if c["window"]:
        seen &= (pos >= s["lens"][:, None] - c["window"]) | (pos < c["sinks"])

    def values(cache, scales):
        x = cache.view(-1, hk, d)[slots].view(FLOAT8[c["fmt"]]).float()
        x = torch.where(seen[:, :, None, None], x, 0)
        if c["gran"] == PER_TOKEN:
            x *= scales.t()[slots][..., None]
        elif c["gran"] == PER_HEAD_TOK128:
            x *= scales[slots // 128][..., None]
        else:
            x *= scales.reshape(-1, 1)
        return x

    k = values(s["k_cache"], s["k_scales"])
    q = s["q"].float().reshape(b, hk, group, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    del k
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = values(s["v_cache"], s["v_scales"])
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total == 0, 1, total)
    lse = (torch.log(total) + top)[..., 0]
    return out.reshape(b, c["hq"], d).to(torch.bfloat16), lse.reshape(b, c["hq"])


# ------------------------------------------------------------------ 64 bits

def _decoded(fmt):
    """The value of each of the 256 codes, from the formats' definition."""
    man, bias = (3, 7) if fmt == E4M3 else (2, 15)
    out = []
    for code in range(256):
        e, m = (code & 0x7F) >> man, code & ((1 << man) - 1)
        x = math.ldexp(m / (1 << man), 1 - bias) if e == 0 else math.ldexp(1 + m / (1 << man), e - bias)
        if fmt == E4M3 and code & 0x7F == 0x7F:
            x = math.nan
        if fmt == E5M2 and e == 31:
            x = math.inf if m == 0 else math.nan
        out.append(-x if code & 0x80 else x)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "pages":
        return None
    if c["op"] == "append":
        return _exact_append(s)
    b, hk, d = c["batch"], c["hk"], c["d"]
    group = c["hq"] // hk
    value = _decoded(c["fmt"])
    out = torch.zeros((b, c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, c["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        places = list(range(n)) if not c["window"] else \
            sorted(set(range(min(n, c["sinks"]))) | set(range(max(0, n - c["window"]), n)))
        if not places:
            continue
        at = torch.tensor(places, device="cuda")
        slot = s["table"][i].long()[at // c["page"]] * c["page"] + at % c["page"]
        for h in range(hk):
            kv = []
            for cache, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
                by = {PER_TENSOR: lambda: scales[0], PER_HEAD: lambda: scales[h],
                      PER_HEAD_TOK128: lambda: scales[slot // 128, h],
                      PER_TOKEN: lambda: scales[h, slot]}[c["gran"]]().double().reshape(-1, 1)
                kv.append(value[cache.view(-1, hk, d)[slot, h].int()] * by)
            z = s["q"][i, h * group:(h + 1) * group].double() @ kv[0].t() * s["scale"]
            lse[i, h * group:(h + 1) * group] = torch.logsumexp(z, 1)
            out[i, h * group:(h + 1) * group] = torch.softmax(z, 1) @ kv[1]
    return out, lse


def _exact_append(s):
    c = s["case"]
    t, d, rot, fmax = c["tokens"], c["d"], c["rot"], FMAX[c["fmt"]]
    first = list(range(0, rot, 2)) if c["interleaved"] else list(range(rot // 2))
    second = [i + 1 for i in first] if c["interleaved"] else [i + rot // 2 for i in first]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None] * torch.tensor(_frequencies(rot, c["stretch"]), dtype=torch.float64,
                                                                       device="cuda"))

    def through(x, weight):
        y = x.double()
        if weight is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * weight.double()
        if rot:
            z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": through(s["q"], s["q_weight"])}
    value = _decoded(c["fmt"])
    where = s["slots"] >= 0
    for name, x in (("k", through(s["k"], s["k_weight"])), ("v", s["v"].double())):
        cache = value[s[name + "_cache"].int()]
        scales = s[name + "_scales"].double()
        if c["gran"] == PER_TOKEN:
            by = x.abs().amax(-1) / fmax
            scales[:, s["slots"][where]] = by[where].t()
            out[name + "_scales"] = scales
        else:
            by = scales.expand(c["hk"]).reshape(1, -1)
        # before the rounding to 8 bits: both sides are off by that rounding.  E5M2's steps are too
        # coarse for such a value to say anything
        cache.view(-1, c["hk"], d)[s["slots"][where]] = (x / by[..., None])[where].clamp(-fmax, fmax)
        out[name] = cache if c["fmt"] == E4M3 else None
    return out
