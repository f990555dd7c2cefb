"""Cases of the paged 8-bit KV cache: block planning, quantising append, attention, keep.

Layouts (D = 256):
  k_pool, v_pool    e4m3 [num_blocks, Hkv, block_size, D]
  k_scale, v_scale  float32 [num_blocks, Hkv], powers of two: a key's value is e4m3 * scale
  block_tables      int32 [B, max_blocks], n_blocks int32 [B]
  free_list         int32 [num_blocks], free_count int32 [1]  (a stack, top at free_count - 1)
"""
import math

import numpy as np
import torch

own = False

D = 256
E4M3_MAX = 448.0
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of 16 sequences: who needs a new block, and where the new rows go.
        dict(name="plan step 16", op="plan", B=16, max_len=32768, rows=1, prompts=0, prompt=0,
             block=64),
        # A busy scheduler step: 256 requests, draft rows for most, eight prompts admitted.
        dict(name="plan admit 8x8192", op="plan", B=256, max_len=32768, rows=8, prompts=8,
             prompt=8192, block=16),
        # The new keys of one decode step.
        dict(name="append step 16", op="append", B=16, rows=1, Hkv=4, max_len=4096, block=64,
             type="bf16"),
        # A prompt's keys and values.
        dict(name="append prompt 8192", op="append", B=1, rows=8192, Hkv=4, max_len=0, block=64,
             type="bf16"),
        # Prompt chunks of several requests behind the keys they hold, odd lengths.
        dict(name="append chunks 12x2731", op="append", B=12, rows=2731, Hkv=2, max_len=4096,
             block=32, type="fp16"),
        # The accepted rows of a draft tree, a small and a large batch.
        dict(name="keep 8", op="keep", B=8, rows=16, Hkv=2, max_len=8192, block=64),
        dict(name="keep 128", op="keep", B=128, rows=32, Hkv=4, max_len=2048, block=32),
        # One short conversation: latency.
        dict(name="decode 1x500", op="decode", B=1, rows=1, ragged=False, tree=False, Hq=24, Hkv=4,
             min_len=500, max_len=500, block=16, type="bf16"),
        # The 27B-shape decode batch.
        dict(name="decode 16x32768", op="decode", B=16, rows=1, ragged=False, tree=False, Hq=24,
             Hkv=4, min_len=1024, max_len=32768, block=64, type="bf16"),
        # Few sequences, long contexts.
        dict(name="decode 2x131071", op="decode", B=2, rows=1, ragged=False, tree=False, Hq=16,
             Hkv=2, min_len=131071, max_len=131071, block=128, type="fp16"),
        # Short chains of drafts.
        dict(name="verify chain 8x4", op="decode", B=8, rows=4, ragged=False, tree=False, Hq=24,
             Hkv=4, min_len=4097, max_len=32768, block=64, type="bf16"),
        # Draft trees of 1 to 32 rows at the 35B shape.
        dict(name="verify tree 8x32", op="decode", B=8, rows=32, ragged=True, tree=True, Hq=16,
             Hkv=2, min_len=4097, max_len=65536, block=64, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "keep", "decode", "decode", "decode"])
    block = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 256), max_len=_log(rng, 64, 32768), rows=_log(rng, 1, 32),
                    prompts=rng.randint(0, 8), prompt=_log(rng, 16, 8192), block=max(block, 16))
    Hq, Hkv = rng.choice([(24, 4), (16, 2), (8, 8), (12, 3), (32, 8), (16, 1)])
    if op == "append":
        rows = _log(rng, 1, 8192)
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 32768 // rows))), rows=rows, Hkv=min(Hkv, 4),
                    max_len=_log(rng, 1, 4096), block=block, type=rng.choice(["bf16", "fp16"]))
    if op == "keep":
        return dict(op=op, B=_log(rng, 1, 128), rows=_log(rng, 1, 48), Hkv=min(Hkv, 4),
                    max_len=_log(rng, 64, 2048), block=block)
    max_len = _log(rng, 64, 65536)
    tree = rng.random() < 0.3
    rows = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 2, 32)])
    B = _log(rng, 1, max(1, min(64, (1 << 21) // (max_len * Hkv), (1 << 27) // (max_len * Hq * rows))))
    return dict(op=op, B=B, rows=rows, ragged=rng.random() < 0.5, tree=tree, Hq=Hq, Hkv=Hkv,
                min_len=max(rows, max_len // 8), max_len=max(rows, max_len), block=block,
                type=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------------------- inputs

def _lens(case, gen, lo, hi):
    return torch.randint(lo, hi + 1, (case["B"],), generator=gen, dtype=torch.int64)


def _rows(case, gen):
    """New rows of each sequence (host); their sum goes by the case alone."""
    B, order = case["B"], torch.randperm(case["B"], generator=gen)
    spread = 1 + torch.arange(B) * case["rows"] // B
    if case["op"] == "plan":
        spread[B - min(case["prompts"], B) :] = case["prompt"]
        return spread[order]
    if case["op"] == "decode" and case["ragged"]:
        spread[-1] = case["rows"]
        return spread[order]
    return torch.full((B,), case["rows"], dtype=torch.int64)


def _i32(x):
    return x.to(device="cuda", dtype=torch.int32)


def _cu(rows):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(rows, 0)])


def _tables(case, lens, most, gen):
    """Random disjoint blocks for `lens` keys per sequence, at most `most` each, and the free rest.
    The pool has room for `most` keys of every sequence."""
    bs, B = case["block"], len(lens)
    need, width = (lens + bs - 1) // bs, -(-most // bs)
    num_blocks, used = B * width + 3, int(need.sum())
    perm = torch.randperm(num_blocks, generator=gen)
    table = torch.full((B, width), -1, dtype=torch.int64)
    table[torch.arange(width)[None, :] < need[:, None]] = perm[:used]
    free = torch.zeros(num_blocks, dtype=torch.int64)
    free[: num_blocks - used] = perm[used:]
    return num_blocks, need, table, free


def _exponent(a):
    """Least e >= -126 with a <= 448 * 2^e, for a >= 0 (float32): a = m * 2^x, 0.5 <= m < 1."""
    m, x = torch.frexp(a)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(a > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def _filled(num_blocks, Hkv, bs, gen, outliers):
    """A pool of N(0, 1) rows (a hundredth of the rows times 8 where `outliers`), quantised a block
    and head at a time."""
    pool = torch.empty((num_blocks, Hkv, bs, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((num_blocks, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * bs * D))
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        x = torch.randn((n, Hkv, bs, D), generator=gen, device="cuda")
        if outliers:
            hit = torch.rand((n, Hkv, bs, 1), generator=gen, device="cuda") < 0.01
            x = torch.where(hit, x * 8, x)
        e = _exponent(x.abs().amax((2, 3)))
        s = torch.exp2(e.float())
        pool[i : i + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scale[i : i + n] = s
    return pool, scale


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, bs = case["op"], case["block"]
    st = dict(case=case, op=op, bs=bs)
    rows = _rows(case, cpu)
    cu = _cu(rows)
    T = int(cu[-1])
    st.update(T=T, cu_rows=_i32(cu), max_rows=int(rows.max()))
    if op == "plan":
        lens = _lens(case, cpu, 0, case["max_len"])
        num_blocks, n_blocks, table, free = _tables(case, lens, case["max_len"] + int(rows.max()), cpu)
        spare = num_blocks - int(n_blocks.sum())
        st.update(kv_lens=_i32(lens), no_rows=_i32(torch.zeros(case["B"] + 1)), n_blocks=_i32(n_blocks),
                  block_tables=_i32(table), free_list=_i32(free), free_count=_i32(torch.tensor([spare])))
        return st
    Hkv = case["Hkv"]
    if op == "append":
        held = _lens(case, cpu, 0, case["max_len"])
        lens, most = held + rows, case["max_len"] + case["rows"]
        t = _TYPES[case["type"]]
        st["k_new"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").to(t)
        st["v_new"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").to(t)
    elif op == "keep":
        most = max(case["rows"], case["max_len"])
        lens = _lens(case, cpu, case["rows"], most)
    else:
        lens = _lens(case, cpu, case["min_len"], case["max_len"])
        lens[0] = case["max_len"]
        lens, most = torch.maximum(lens, rows), case["max_len"]
    num_blocks, _, table, _ = _tables(case, lens, most, cpu)
    st.update(kv_lens=_i32(lens), block_tables=_i32(table))
    st["k_pool"], st["k_scale"] = _filled(num_blocks, Hkv, bs, gen, op == "decode")
    st["v_pool"], st["v_scale"] = _filled(num_blocks, Hkv, bs, gen, False)
    if op == "append":
        b = torch.repeat_interleave(torch.arange(case["B"]), rows)
        pos = held[b] + torch.arange(T) - cu[b]
        st["slots"] = _i32(table[b, pos // bs] * bs + pos % bs)
    elif op == "keep":
        # an accepted root path: a random increasing half of the draft rows
        pick = torch.rand((case["B"], case["rows"]), generator=cpu) < 0.5
        pick[0, 0] = True
        st["keep_idx"] = _i32(torch.nonzero(pick)[:, 1])
        st["cu_keep"] = _i32(_cu(pick.sum(1)))
        st["kept"] = int(pick.sum())
        st["kv_lens_out"] = torch.zeros_like(st["kv_lens"])
    else:
        t, Hq = _TYPES[case["type"]], case["Hq"]
        st["q"] = torch.randn((T, Hq, D), generator=gen, device="cuda").to(t)
        st["g"] = (torch.randn((T, Hq, D), generator=gen, device="cuda") * 2).to(t)
        st["max_kv_len"] = int(lens.max())
        st["out"] = torch.empty_like(st["q"])
        st["tree_mask"] = None
        if case["tree"]:
            # each new row's parent is a random earlier row: its mask is the parent's and itself
            masks = []
            for n in rows.tolist():
                up = [1]
                for i in range(1, n):
                    up.append(up[int(torch.randint(0, i, (1,), generator=cpu))] | (1 << i))
                masks += up
            st["tree_mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
    return st


# ------------------------------------------------------------------------------- plain forms

def _plan_plain(st, cu_rows, T):
    """One planning step, in place: surplus blocks back on the stack, missing ones off it."""
    bs, table, n_blocks = st["bs"], st["block_tables"].long(), st["n_blocks"].long()
    free, fc = st["free_list"].long(), st["free_count"].long()
    lens, cu = st["kv_lens"].long(), cu_rows.long()
    rows = cu[1:] - cu[:-1]
    need = (lens + rows + bs - 1) // bs
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    loose = (col >= need[:, None]) & (col < n_blocks[:, None])
    rank = torch.cumsum(loose.reshape(-1), 0).reshape(loose.shape) - 1
    total = loose.sum()
    # the entries that stay go to a place behind the list, which is cut off again
    at = torch.where(loose, fc + total - 1 - rank, free.numel())
    free = torch.cat([free, free[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:-1]
    table = torch.where(loose, -1, table)
    avail = fc + total
    grow = (need - n_blocks).clamp(min=0)
    after = torch.cumsum(grow, 0)
    served = (after <= avail) | (grow == 0)
    new = (col >= n_blocks[:, None]) & (col < need[:, None]) & served[:, None]
    take = avail - 1 - ((after - grow)[:, None] + col - n_blocks[:, None])
    table = torch.where(new, free[take.clamp(0, free.numel() - 1)], table)
    st["block_tables"].copy_(table)
    st["n_blocks"].copy_(torch.where(served, need, n_blocks))
    st["free_list"].copy_(free)
    st["free_count"].copy_(avail - (grow * served).sum())
    t = torch.arange(T, device="cuda")
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=lens.numel() - 1)
    pos = lens[b] + t - cu[b]
    slots = table[b, pos // bs] * bs + pos % bs
    slots = torch.where(served[b] & (t < cu[-1]), slots, -1)
    return slots.int(), torch.where(served, lens + rows, lens).int()


def _quantise(x, e):
    return (x * torch.exp2(-e.float())).to(torch.float8_e4m3fn)


def _store_plain(st, name, x, slots, first):
    """Rows x [T, Hkv, D] (float32) behind what their blocks hold, one scale per block and head.
    first: each sequence's first row in x; only its block can hold earlier rows that stay."""
    pool, scale, bs = st[name + "_pool"].view(torch.uint8), st[name + "_scale"], st["bs"]
    block, off = slots // bs, slots % bs
    a = torch.zeros_like(scale).index_reduce(0, block, x.abs().amax(-1), "amax")
    begin = torch.full((scale.shape[0],), bs, device="cuda").index_reduce(0, block, off, "amin")[:, None]
    e_new, e_old = _exponent(a), torch.frexp(scale)[1] - 1
    e = torch.where(begin > 0, torch.maximum(e_old, e_new), e_new)
    e = torch.where(begin < bs, e, e_old)
    n, stay = block[first], torch.arange(bs, device="cuda")[None, :] < off[first][:, None]
    old = pool[n].view(torch.float8_e4m3fn).float() * scale[n][..., None, None]
    again = _quantise(old, e[n][..., None, None]).view(torch.uint8)
    pool[n] = torch.where(stay[:, None, :, None], again, pool[n])
    pool[block, :, off] = _quantise(x, e[block][..., None]).view(torch.uint8)
    scale.copy_(torch.exp2(e.float()))


def _append_plain(st):
    slots, first = st["slots"].long(), st["cu_rows"][:-1].long()
    _store_plain(st, "k", st["k_new"].float(), slots, first)
    _store_plain(st, "v", st["v_new"].float(), slots, first)


def _keep_plain(st):
    bs, cu, ck = st["bs"], st["cu_rows"].long(), st["cu_keep"].long()
    base = st["kv_lens"].long() - (cu[1:] - cu[:-1])
    k = torch.arange(st["kept"], device="cuda")
    b = torch.searchsorted(ck, k, right=True) - 1
    at = lambda pos: st["block_tables"].long()[b, pos // bs] * bs + pos % bs  # noqa: E731
    src, dst = at(base[b] + st["keep_idx"].long()), at(base[b] + k - ck[b])
    for name in ("k", "v"):
        bits = st[name + "_pool"].view(torch.uint8)[src // bs, :, src % bs]
        x = bits.view(torch.float8_e4m3fn).float() * st[name + "_scale"][src // bs][..., None]
        _store_plain(st, name, x, dst, ck[:-1].clamp(max=st["kept"] - 1))
    st["kv_lens_out"].copy_(base + ck[1:] - ck[:-1])


def _decode_plain(st):
    bs, cu, lens = st["bs"], st["cu_rows"].long(), st["kv_lens"].long()
    q, table = st["q"].float(), st["block_tables"].long()
    T, Hq, _ = q.shape
    B, Hkv, R = lens.numel(), st["k_pool"].shape[1], st["max_rows"]
    n = -(-st["max_kv_len"] // bs)

    def cache(name):   # [B, Hkv, n * bs, D] in float32
        pages = table[:, :n].clamp(min=0)
        x = st[name + "_pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        return (x * st[name + "_scale"][pages][..., None, None]).transpose(1, 2).reshape(B, Hkv, n * bs, D)

    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    rows = cu[1:] - cu[:-1]
    qp = torch.zeros((B, R, Hq, D), device="cuda")
    qp[b, i] = q
    qp = qp.view(B, R, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * (Hq // Hkv), D)
    s = qp @ cache("k").transpose(-1, -2) * (1.0 / 16.0)
    key = torch.arange(n * bs, device="cuda")
    ends = torch.zeros((B, R), dtype=torch.int64, device="cuda")
    ends[b, i] = (lens - rows)[b] + i + 1
    seen = key < ends[..., None]
    if st["tree_mask"] is not None:
        bits = torch.zeros((B, R), dtype=torch.int64, device="cuda")
        bits[b, i] = st["tree_mask"]
        back = key - (lens - rows)[:, None]
        new = ((bits[..., None] >> back[:, None].clamp(0, 63)) & 1).bool()
        seen = (back < 0)[:, None] | (new & (back >= 0)[:, None] & (key < lens[:, None])[:, None])
    seen = seen[:, None, :, None, :].expand(B, Hkv, R, Hq // Hkv, n * bs).reshape(s.shape)
    s = torch.where(seen, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    del s, seen
    o = (p @ cache("v")) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(B, Hkv, R, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D)[b, i]
    return (o / (1 + torch.exp(-st["g"].float()))).to(st["q"].dtype)


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "plan":
        # a step's rows get their places; all of them are then given back (a request that was
        # cancelled, drafts that were refused)
        slots, lens = _plan_plain(st, st["cu_rows"], st["T"])
        _, back = _plan_plain(st, st["no_rows"], 0)
        return dict(slots=slots, kv_lens=lens, back=back, tables=st["block_tables"],
                    n_blocks=st["n_blocks"], free_count=st["free_count"])
    if st["op"] == "append":
        _append_plain(st)
        return dict(k=st["k_pool"], v=st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    if st["op"] == "keep":
        _keep_plain(st)
        return dict(k=st["k_pool"], v=st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                    kv_lens=st["kv_lens_out"])
    return dict(out=_decode_plain(st))


def _run_own(st):
    import gqa_head_gated_gb300 as G
    if st["op"] == "plan":
        slots, lens = G.block_plan(st["kv_lens"], st["cu_rows"], st["block_tables"], st["n_blocks"],
                                   st["free_list"], st["free_count"], st["bs"], st["T"])
        _, back = G.block_plan(st["kv_lens"], st["no_rows"], st["block_tables"], st["n_blocks"],
                               st["free_list"], st["free_count"], st["bs"], 0)
        return dict(slots=slots, kv_lens=lens, back=back, tables=st["block_tables"],
                    n_blocks=st["n_blocks"], free_count=st["free_count"])
    if st["op"] == "append":
        G.kv8_append(st["k_new"], st["v_new"], st["slots"], st["k_pool"], st["v_pool"],
                     st["k_scale"], st["v_scale"])
        return dict(k=st["k_pool"], v=st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    if st["op"] == "keep":
        G.kv8_keep(st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], st["block_tables"],
                   st["kv_lens"], st["cu_rows"], st["keep_idx"], st["cu_keep"], st["kv_lens_out"])
        return dict(k=st["k_pool"], v=st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                    kv_lens=st["kv_lens_out"])
    if "workspace" not in st:
        st["workspace"] = torch.empty(
            G.kv8_workspace_size(st["kv_lens"].numel(), st["T"], st["q"].shape[1],
                                 st["k_pool"].shape[1], st["max_rows"], st["max_kv_len"]),
            dtype=torch.uint8, device="cuda")
    return dict(out=G.kv8_decode(st["q"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"],
                                 st["g"], st["block_tables"], st["kv_lens"], st["cu_rows"],
                                 tree_mask=st["tree_mask"], max_rows=st["max_rows"],
                                 max_kv_len=st["max_kv_len"], workspace=st["workspace"],
                                 out=st["out"]))


# ------------------------------------------------------------------------------- work, 64 bits

def work(case):
    B, op, bs = case["B"], case["op"], case["block"]
    if op == "plan":
        extra = min(case["prompts"], B)
        T = sum(1 + i * case["rows"] // B for i in range(B - extra)) + extra * case["prompt"]
        moved = T / bs
        # two steps: lengths, row offsets and block counts in, lengths and block counts out; the
        # moved blocks' table and list entries; the rows' slots
        return {"bytes": 4.0 * (2 * 5 * B + 2 * 4 * moved + T), "flops": 0.0}
    if op == "append":
        rows = B * case["rows"] * case["Hkv"] * 2
        return {"bytes": float(rows * D * 3 + B * case["rows"] * 4), "flops": 2.0 * rows * D}
    if op == "keep":
        rows = B * case["rows"] / 2 * case["Hkv"] * 2
        return {"bytes": float(rows * D * 2), "flops": 2.0 * rows * D}
    lens = (case["min_len"] + case["max_len"]) / 2
    rows = (1 + case["rows"]) / 2 if case["ragged"] else case["rows"]
    keys = B * lens
    return {"bytes": float(keys * case["Hkv"] * (2 * D + 8 / bs) + 3 * 2 * B * rows * case["Hq"] * D),
            "flops": float(4.0 * D * keys * rows * case["Hq"])}


def _round8(x):
    """e4m3 of float64 values within +-448, to the nearest, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.rint(x / step) * step


def _store_exact(pool, scale, x, slots, bs):
    """pool: e4m3 values, scale: powers of two, both float64 and changed; x [n, Hkv, D]."""
    slots = np.asarray(slots)
    begin = [i for i in range(len(slots)) if i == 0 or slots[i] // bs != slots[i - 1] // bs]
    for i, j in zip(begin, begin[1:] + [len(slots)]):
        n, off = int(slots[i] // bs), int(slots[i] % bs)
        a = np.abs(x[i:j]).max(axis=(0, 2))
        new = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(a, 2.0 ** -140) / E4M3_MAX)), -126))
        if off:
            keep = np.maximum(new, scale[n])
            pool[n, :, :off] = _round8(pool[n, :, :off] * (scale[n] / keep)[:, None, None])
            new = keep
        scale[n] = new
        pool[n, :, off : off + j - i] = _round8(x[i:j] / new[None, :, None]).transpose(1, 0, 2)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    f64 = lambda x: x.detach().double().cpu().numpy()  # noqa: E731
    bs = st["bs"]
    if case["op"] in ("append", "keep"):
        got = {}
        for name in ("k", "v"):
            pool, scale = f64(st[name + "_pool"].float()), f64(st[name + "_scale"])
            if case["op"] == "append":
                _store_exact(pool, scale, f64(st[name + "_new"]), st["slots"].cpu().numpy(), bs)
            else:
                table, lens = st["block_tables"].cpu().numpy(), st["kv_lens"].cpu().numpy()
                cu, ck = st["cu_rows"].cpu().numpy(), st["cu_keep"].cpu().numpy()
                idx = st["keep_idx"].cpu().numpy()
                for b in range(case["B"]):
                    base, n = lens[b] - (cu[b + 1] - cu[b]), ck[b + 1] - ck[b]
                    if n == 0:
                        continue
                    src = base + idx[ck[b] : ck[b + 1]]
                    x = pool[table[b, src // bs], :, src % bs] * scale[table[b, src // bs]][..., None]
                    dst = base + np.arange(n)
                    _store_exact(pool, scale, x, table[b, dst // bs] * bs + dst % bs, bs)
            got[name], got[name + "_scale"] = pool, scale
        if case["op"] == "keep":
            got["kv_lens"] = None
        return got
    # attention: a sequence and KV head at a time
    q, g = st["q"].double(), st["g"].double()
    cu, lens, table = st["cu_rows"].tolist(), st["kv_lens"].tolist(), st["block_tables"].long()
    out = torch.zeros_like(q)
    Hq, Hkv = case["Hq"], case["Hkv"]
    gqa = Hq // Hkv
    for b in range(case["B"]):
        t0, t1, L = cu[b], cu[b + 1], lens[b]
        base = L - (t1 - t0)
        pages = table[b, : -(-L // bs)]
        see = torch.ones((t1 - t0, L), dtype=torch.bool, device="cuda")
        for i in range(t1 - t0):
            if st["tree_mask"] is None:
                see[i, base + i + 1 :] = False
            else:
                word = int(st["tree_mask"][t0 + i])
                see[i, base:] = torch.tensor([bool(word >> k & 1) for k in range(t1 - t0)], device="cuda")
        for h in range(Hkv):
            k, v = ((st[n + "_pool"].view(torch.uint8)[pages, h].view(torch.float8_e4m3fn).double()
                     * st[n + "_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:L]
                    for n in ("k", "v"))
            for i in range(h * gqa, (h + 1) * gqa):
                s = (q[t0:t1, i] @ k.T) / math.sqrt(D)
                w = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
                out[t0:t1, i] = (w @ v) * torch.sigmoid(g[t0:t1, i])
    return dict(out=out)
