"""Oracle of the paged 8-bit KV cache: plain loops and float64, no blocking, no CUDA.

TEST INFRASTRUCTURE ONLY.  e4m3 is spelled out from its definition (sign, four exponent
bits with bias 7, three mantissa bits, subnormals, no infinity, S.1111.111 is NaN) as a
table of its 256 values, and rounding is a search in that table.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def _e4m3_table():
    out = np.empty(256)
    for code in range(256):
        sign, e, m = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            out[code] = np.nan
        else:
            out[code] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return out


E4M3 = _e4m3_table()
_POS = E4M3[:127]                     # 0 .. 448, increasing


def e4m3_encode(x):
    """Codes of float64 values (|x| <= 448 when finite), nearest, ties to the even code; NaN
    and infinities become NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    mid = (_POS[lo] + _POS[hi]) / 2
    code = np.where(a > mid, hi, np.where(a < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(x), code, 0x7F)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def scale_exponent(a):
    """Least e >= -126 with a <= 448 * 2^e."""
    e = -126
    if a > 0:
        e = max(-126, math.frexp(a / E4M3_MAX)[1] - 1)
        while a > E4M3_MAX * 2.0 ** e:
            e += 1
    return e


def block_plan(kv_lens, rows, tables, n_blocks, free, block_size, T):
    """One planning step over Python lists; `free` is the stack (top last).  Changes tables,
    n_blocks and free; returns (slots, kv_lens_out, served)."""
    B = len(kv_lens)
    need = [-(-(kv_lens[b] + rows[b]) // block_size) for b in range(B)]
    loose = []
    for b in range(B):
        for i in range(need[b], n_blocks[b]):
            loose.append(tables[b][i])
            tables[b][i] = -1
        n_blocks[b] = min(n_blocks[b], need[b])
    free += loose[::-1]
    left, wanted, served = len(free), 0, []
    for b in range(B):
        grow = need[b] - n_blocks[b]
        wanted += grow
        served.append(grow == 0 or wanted <= left)
        if served[b]:
            for i in range(n_blocks[b], need[b]):
                tables[b][i] = free.pop()
            n_blocks[b] = need[b]
    slots = []
    for b in range(B):
        for i in range(rows[b]):
            pos = kv_lens[b] + i
            slots.append(tables[b][pos // block_size] * block_size + pos % block_size
                         if served[b] else -1)
    slots += [-1] * (T - len(slots))
    return slots, [kv_lens[b] + (rows[b] if served[b] else 0) for b in range(B)], served


def kv8_append(pool, scale, x, slots, block_size):
    """pool: codes uint8 [N, Hkv, bs, 256], scale: float64 [N, Hkv], both changed; x: float64
    [T, Hkv, 256]; slots: list (-1: skipped)."""
    T, Hkv, _ = x.shape
    t = 0
    while t < T:
        if slots[t] < 0:
            t += 1
            continue
        n, off = slots[t] // block_size, slots[t] % block_size
        end = t + 1
        while end < T and slots[end] == slots[end - 1] + 1 and slots[end] // block_size == n:
            end += 1
        for g in range(Hkv):
            a = np.abs(x[t:end, g])
            e = scale_exponent(float(np.max(np.where(np.isfinite(a), a, 0.0))))
            if off:
                e = max(e, int(math.frexp(scale[n, g])[1]) - 1)
                old = E4M3[pool[n, g, :off]] * scale[n, g]
                pool[n, g, :off] = e4m3_encode(old * 2.0 ** -e)
            pool[n, g, off:off + end - t] = e4m3_encode(x[t:end, g] * 2.0 ** -e)
            scale[n, g] = 2.0 ** e
        t = end


def kv8_keep(pool, scale, tables, kv_lens, rows, keep, block_size):
    """Appends the kept rows' values behind the first kv_lens[b] - rows[b] keys."""
    for b, idx in enumerate(keep):
        base = kv_lens[b] - rows[b]
        place = lambda pos: (tables[b][pos // block_size], pos % block_size)  # noqa: E731
        vals = [E4M3[pool[n, :, o]] * scale[n][:, None]
                for n, o in (place(base + i) for i in idx)]
        if not vals:
            continue
        slots = [n * block_size + o for n, o in (place(base + k) for k in range(len(idx)))]
        # runs of one block each, whether or not the next block lies right behind it
        start = 0
        for k in range(1, len(slots) + 1):
            if k == len(slots) or (base + k) % block_size == 0:
                kv8_append(pool, scale, np.stack(vals[start:k]), slots[start:k], block_size)
                start = k


def kv8_contiguous(pool, scale, tables, kv_lens, block_size):
    """The cache [B, Hkv, max len, 256] in float64 that the tables describe (0 past a length)."""
    B, L = len(kv_lens), max(max(kv_lens), 1)
    out = np.zeros((B, pool.shape[1], L, 256))
    for b in range(B):
        for j0 in range(0, kv_lens[b], block_size):
            n, m = tables[b][j0 // block_size], min(block_size, kv_lens[b] - j0)
            out[b, :, j0:j0 + m] = E4M3[pool[n, :, :m]] * scale[n][:, None, None]
    return out
