"""Oracle of shared blocks (fork, free, compact, copy) and of rotary positions: plain loops and float64.

TEST INFRASTRUCTURE ONLY.  Tables, stacks and counts are Python lists, changed in place.
"""
from __future__ import annotations

import math
from fractions import Fraction



def block_fork(src, dst, lens, kv_lens, tables, n_blocks, free, shares, block_size):
    """`free` is the stack (top last).  Returns (copies, verdicts): "ok", "refused" or "no block" per fork."""
    B, copies, verdicts, left = len(kv_lens), [], [], len(free)
    took = 0
    plan = []
    for f, (s, d) in enumerate(zip(src, dst)):
        n = kv_lens[s] if lens is None and 0 <= s < B else (lens[f] if lens is not None else -1)
        ok = (0 <= s < B and 0 <= d < B and d not in src and dst.count(d) == 1 and 0 <= n <= kv_lens[s]
              and -(-n // block_size) <= n_blocks[s] and n_blocks[d] == 0)
        plan.append((n, ok))
    for (n, ok), s, d in zip(plan, src, dst):
        full, rest = divmod(n, block_size) if ok else (0, 0)
        if not ok:
            verdicts.append("refused")
        elif rest and took >= left:
            verdicts.append("no block")
        else:
            verdicts.append("ok")
        if verdicts[-1] != "ok":
            copies.append([-1, -1, 0])
            continue
        for i in range(full):
            tables[d][i] = tables[s][i]
            shares[tables[s][i]] += 1
        if rest:
            took += 1
            tables[d][full] = free.pop()
            copies.append([tables[s][full], tables[d][full], rest])
        else:
            copies.append([-1, -1, 0])
        n_blocks[d] = full + (rest > 0)
        kv_lens[d] = n
    return copies, verdicts


def block_free(kv_lens, tables, n_blocks, free, shares, block_size):
    loose = []
    for b, n in enumerate(kv_lens):
        keep = min(-(-n // block_size), n_blocks[b])
        for i in range(keep, n_blocks[b]):
            loose.append(tables[b][i])
            tables[b][i] = -1
        n_blocks[b] = keep
    gone = []
    for k, blk in enumerate(loose):
        if shares[blk] == 0 and blk not in loose[k + 1:]:
            gone.append(blk)
        else:
            shares[blk] = max(shares[blk] - 1, 0)
    free += gone[::-1]


def block_compact(tables, n_blocks, free, shares, num_blocks, block_size):
    """Returns (tables, free, shares, new_index, copies), the inputs as they were."""
    is_free = set(free)
    L = num_blocks - len(free)
    holes = [n for n in range(L) if n in is_free]
    movers = [n for n in range(L, num_blocks) if n not in is_free]
    index = [-1 if n in is_free else n for n in range(num_blocks)]
    for a, b in zip(movers, holes):
        index[a] = b
    new = [[index[t] if i < n_blocks[b] else -1 for i, t in enumerate(row)] for b, row in enumerate(tables)]
    moved = [0] * num_blocks
    for n, to in enumerate(index):
        if to >= 0:
            moved[to] = shares[n]
    copies = [[a, b, block_size] for a, b in zip(movers, holes)]
    copies += [[-1, -1, 0]] * (num_blocks // 2 - len(copies))
    return new, list(range(num_blocks - 1, L - 1, -1)), moved, index, copies


def kv8_copy(copies, pools, scales):
    for a, b, rows in copies:
        if a < 0 or b < 0 or rows <= 0:
            continue
        for p in pools:
            p[b, :, :rows] = p[a, :, :rows]
        for s in scales:
            s[b] = s[a]


def _two_pi(bits):
    """2 pi 2^bits as an integer, from 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        term = (1 << (bits + 32)) // n
        total, k = term, 1
        while term:
            term //= n * n
            total += (-1) ** k * (term // (2 * k + 1))
            k += 1
        return total
    return 2 * (16 * atan(5) - 4 * atan(239)) >> 32


_BITS = 200
_TURN = _two_pi(_BITS)


def angle(position, freq):
    """position * freq modulo 2 pi, in exact integers up to the last rounding."""
    a = Fraction(position) * Fraction(float(freq))
    return float(Fraction((a.numerator << _BITS) // a.denominator % _TURN, 1 << _BITS))


def rope(x, positions, inv_freq, interleaved=False, scale=1.0, inverse=False):
    """x float64 [T, H, D], positions [T]."""
    y, half = x.copy(), len(inv_freq)
    for t, pos in enumerate(positions):
        for j, f in enumerate(inv_freq):
            a = angle(int(pos), f) * (-1 if inverse else 1)
            c, s = math.cos(a) * scale, math.sin(a) * scale
            i1, i2 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            y[t, :, i1] = x[t, :, i1] * c - x[t, :, i2] * s
            y[t, :, i2] = x[t, :, i2] * c + x[t, :, i1] * s
    return y
