"""Plain 64-bit forms of the paged KV-cache operators for their tests (numpy, no library code)."""
import math

import numpy as np

FMAX = (448.0, 57344.0)
#: half the smallest step of each format (subnormals), and half a step relative to a normal value
SUB = (2.0 ** -10, 2.0 ** -17)
REL = (2.0 ** -4, 2.0 ** -3)


def decode_table(fmt):
    man, bias = (3, 7) if fmt == 0 else (2, 15)
    out = np.empty(256)
    for code in range(256):
        e, m = (code & 0x7F) >> man, code & ((1 << man) - 1)
        x = math.ldexp(m / (1 << man), 1 - bias) if e == 0 else math.ldexp(1 + m / (1 << man), e - bias)
        if (fmt == 0 and code & 0x7F == 0x7F) or (fmt == 1 and e == 31 and m):
            x = math.nan
        elif fmt == 1 and e == 31:
            x = math.inf
        out[code] = -x if code & 0x80 else x
    return out


def bf16_to_f64(u16):
    return (np.asarray(u16, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def token_scale(scales, gran, slots, h):
    """fp32 scales of head h at the given slots."""
    if gran == 0:
        return np.full(len(slots), scales[0], np.float64)
    if gran == 1:
        return np.full(len(slots), scales[h], np.float64)
    if gran == 2:
        return scales[slots // 128, h].astype(np.float64)
    return scales[h, slots].astype(np.float64)


def attention(q, k_codes, v_codes, k_scales, v_scales, table, lens, fmt, gran, scale, window, sinks):
    """-> (out, lse, out's tolerance, lse's tolerance), q float64 [B][Hq][D], codes [pages][size][H][D].

    Tolerance of an element, from the arithmetic: the result's rounding to bf16 (2^-8 of it); with
    A = sum p |v| / sum p, 2^-11 A for the weights' rounding to f16, n 2^-25 of the largest weight
    times scale times code for weights below f16's normal range; twice the score's error (fp32 sums of
    head_dim products, 2^-22 a step with truncating adders; a few roundings of the scaled score and
    its exponential); a few fp32 roundings in the join."""
    B, Hq, D = q.shape
    P, size, H, _ = k_codes.shape
    G = Hq // H
    val = decode_table(fmt)
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, ltol = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        n = int(lens[b])
        tok = np.arange(n)
        if window:
            tok = tok[(tok >= n - window) | (tok < sinks)]
        if tok.size == 0:
            continue
        page = table[b, tok // size].astype(np.int64)
        place = tok % size
        slots = page * size + place
        for h in range(H):
            sk, sv = token_scale(k_scales, gran, slots, h), token_scale(v_scales, gran, slots, h)
            k = val[k_codes[page, place, h]] * sk[:, None]
            code = val[v_codes[page, place, h]]
            v = code * sv[:, None]
            qq = q[b, h * G:(h + 1) * G]
            z = qq @ k.T * scale
            dz = (np.abs(qq) @ np.abs(k.T) * scale * (D + 8) * 2.0 ** -22 + np.abs(z) * 2.0 ** -21).max(1)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            tot = p.sum(1, keepdims=True)
            o = p @ v / tot
            a = p @ np.abs(v) / tot
            small = tok.size * 2.0 ** -25 * (p * sv).max(1) / tot[:, 0] * np.abs(code).max()
            rows = slice(h * G, (h + 1) * G)
            out[b, rows] = o
            tol[b, rows] = np.abs(o) * 2.0 ** -8 + a * (2.0 ** -11 + 2 * dz[:, None] + 2.0 ** -19) + small[:, None] + 1e-38
            lse[b, rows] = np.log(tot[:, 0]) + m[:, 0]
            ltol[b, rows] = dz + 2.0 ** -20 * (1 + np.abs(lse[b, rows]))
    return out, lse, tol, ltol


def rotate(x, positions, freq, interleaved):
    """x [T][H][D] -> rotated, and |a| + |b| of each element's pair (for tolerances)."""
    rot = 2 * len(freq)
    y, mag = x.copy(), np.abs(x)
    if rot:
        ang = positions.astype(np.float64)[:, None, None] * np.asarray(freq)
        c, s = np.cos(ang), np.sin(ang)
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def norm(x, weight, eps):
    return x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


class Pages:
    """The page bookkeeping, one request after another."""

    def __init__(self, table, lens, free, count, size):
        self.table, self.lens, self.free, self.count, self.size = table.copy(), lens.copy(), free.copy(), count, size

    def step(self, added, max_tokens):
        B, P = self.table.shape
        size = self.size
        held = -(-self.lens.astype(np.int64) // size)
        for b in range(B):
            if added[b] < 0:
                for j in range(held[b]):
                    self.free[self.count] = self.table[b, j]
                    self.count += 1
        total, used, wanted = self.count, 0, 0
        slots, pos = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32)
        offsets, served = np.zeros(B + 1, np.int32), np.zeros(B, np.int32)
        at = 0
        for b in range(B):
            n = max(0, int(added[b]))
            offsets[b] = at
            end = at + n
            old = int(self.lens[b])
            if added[b] < 0:
                self.lens[b] = 0
            else:
                fits = old + n <= P * size and end <= max_tokens
                need = -(-(old + n) // size) - int(held[b]) if fits else 0
                wanted += need
                if fits and (need == 0 or wanted <= total):
                    served[b] = 1
                    for j in range(need):
                        self.table[b, held[b] + j] = self.free[total - 1 - (wanted - need + j)]
                    if need:
                        used = wanted
                    self.lens[b] = old + n
            for i in range(n):
                if at + i < max_tokens:
                    pos[at + i] = old + i
                    if served[b]:
                        slots[at + i] = int(self.table[b, (old + i) // size]) * size + (old + i) % size
            at = end
        offsets[B] = at
        self.count = total - used
        return slots, pos, offsets, served
