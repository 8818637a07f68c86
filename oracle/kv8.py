"""The 8-bit paged cache and attention over it in float64 (numpy), from their
definitions: E4M3's values by their bits, the nearest by a search, pages and
sequences one at a time."""
from __future__ import annotations

import numpy as np

EXP_MIN, EXP_MAX = -117, 119


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7F) == 0x7F else (m / 8 * 2.0 ** -6 if e == 0
                                               else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 0x80 else v
    return out


VALUES = e4m3_values()


def to_code(x: np.ndarray) -> np.ndarray:
    """Nearest code (ties to even) of values no larger than 448; NaN and
    infinities to a NaN code."""
    pos = VALUES[:127]
    a = np.abs(x)
    bad = ~np.isfinite(x)
    a = np.where(bad, 0.0, np.minimum(a, 448.0))
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == pos[hi], hi, code)
    code = np.where(bad, 0x7F, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(mag: float) -> int:
    """The least e in [EXP_MIN, EXP_MAX] with 448 * 2^e >= mag."""
    e = EXP_MIN
    while e < EXP_MAX and 448 * 2.0 ** e < mag:
        e += 1
    return e


def write(codes, exps, x, table, start, counts):
    """Append x [B, H, N, D] (float64) to codes [P, H, page, D] uint8 and exps
    [P, H] int8, in place."""
    B, H, N, D = x.shape
    page = codes.shape[2]
    for b in range(B):
        n = N if counts is None else int(counts[b])
        s = int(start[b])
        for slot in range(s // page, -(-(s + n) // page)):
            if n == 0:
                break
            pid = int(table[b, slot])
            lo, hi = max(s, slot * page), min(s + n, (slot + 1) * page)
            r0, r1 = lo - slot * page, hi - slot * page
            for h in range(H):
                new = x[b, h, lo - s:hi - s]
                fin = np.abs(new[np.isfinite(new)])
                e = exponent(float(fin.max()) if fin.size else 0.0)
                if r0 > 0:
                    held = int(exps[pid, h])
                    e = max(e, held)
                    if e > held:
                        codes[pid, h, :r0] = to_code(
                            np.ldexp(VALUES[codes[pid, h, :r0]], held - e))
                codes[pid, h, r0:r1] = to_code(np.ldexp(new, -e))
                exps[pid, h] = e


def read(codes, exps, table, b, n) -> np.ndarray:
    """[H, n, D] float64: the first n positions of sequence b."""
    page = codes.shape[2]
    out = np.empty((codes.shape[1], n, codes.shape[3]))
    for t in range(n):
        pid = int(table[b, t // page])
        out[:, t] = np.ldexp(VALUES[codes[pid, :, t % page]], exps[pid].astype(int)[:, None])
    return out


def attention(q, k, v, see, scale):
    """One sequence and query head in float64: q [N, D] against k, v [n, D],
    row i seeing the first see[i] positions.  Returns o, lse, and the bounds' parts:
    sum p |v| per output, and how far rounding can move a row's scores (fp32 sums
    of D terms, and how the kernels hold the queries)."""
    N, D = q.shape
    o = np.zeros((N, D))
    mag = np.zeros((N, D))
    lse = np.full(N, -np.inf)
    off = np.zeros(N)
    for i in range(N):
        m = int(see[i])
        if m == 0:
            continue
        s = scale * (k[:m] @ q[i])
        top = s.max()
        p = np.exp(s - top)
        z = p.sum()
        lse[i] = top + np.log(z)
        o[i] = (p / z) @ v[:m]
        mag[i] = (p / z) @ np.abs(v[:m])
        top_q = np.abs(q[i]).max()
        # Queries held in fp16 relative to their largest: off by at most 2^-25 of it.
        # Held as two E4M3 terms, scaled so that the largest lies in [128, 256): a value
        # of eight bits is exact while its last bit is at least E4M3's least, 2^-9, so
        # from 2^-2 on (2^-9 of the largest, at the least); smaller ones are off by half
        # that step, 2^-10 (2^-17 of the largest).
        small = np.abs(q[i]) < 2.0 ** -9 * top_q
        off[i] = scale * float(np.max(
            D * 2.0 ** -24 * (np.abs(k[:m]) @ np.abs(q[i])) +
            top_q * (2.0 ** -25 * np.abs(k[:m]).sum(1) + 2.0 ** -17 * np.abs(k[:m]) @ small)))
    return o, lse, mag, off
