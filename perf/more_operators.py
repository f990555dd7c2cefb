"""Cases of serving over the paged 8-bit KV cache: rotary positions, forks of shared prefixes,
compaction, and the attention of prompt chunks.

Layouts (D = 256):
  q [T, Hq, D], k [T, Hkv, D]   16 bits, token-major; rope also takes slices of a fused projection
  k_pool, v_pool    e4m3 [num_blocks, Hkv, block_size, D]
  k_scale, v_scale  float32 [num_blocks, Hkv], powers of two: a key's value is e4m3 * scale
  block_tables      int32 [B, max_blocks], n_blocks int32 [B]
  free_list         int32 [num_blocks], free_count int32 [1]  (a stack, top at free_count - 1)
  shares            int32 [num_blocks], how many tables hold a block beside the first
"""
import math

import torch

own = False

D = 256
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # The new tokens of one decode step.
        dict(name="rope step 16", op="rope", T=16, Hq=24, Hkv=4, rot=64, interleaved=False,
             fused=False, far=32768, scale=1.0, type="bf16"),
        # A prompt, taken from the output of a fused q/k/v projection.
        dict(name="rope prompt 8192", op="rope", T=8192, Hq=24, Hkv=4, rot=64, interleaved=False,
             fused=True, far=0, scale=1.0, type="bf16"),
        # Chunks of very long contexts, whole heads rotated in neighbouring pairs.
        dict(name="rope chunks 32749 far", op="rope", T=32749, Hq=16, Hkv=2, rot=256,
             interleaved=True, fused=False, far=1000000, scale=1.1386, type="fp16"),
        # Some samples of one short prompt.
        dict(name="fork 8 of 500", op="fork", parents=1, forks=8, len=500, block=16, Hkv=2),
        # Requests that arrive behind a few long shared prefixes.
        dict(name="fork 192 of 4x24001", op="fork", parents=4, forks=192, len=24001, block=64, Hkv=4),
        # A small pool put in order after half of its requests ended.
        dict(name="compact 16x2000", op="compact", B=16, max_len=2000, block=64, Hkv=2),
        # A large one with small blocks.
        dict(name="compact 256x6000", op="compact", B=256, max_len=6000, block=16, Hkv=4),
        # A short first prompt: latency.
        dict(name="prefill 1x100", op="prefill", B=1, rows=100, ragged=False, context=0, Hq=24, Hkv=4,
             block=16, type="bf16"),
        # The 27B-shape prompt.
        dict(name="prefill 1x8192", op="prefill", B=1, rows=8192, ragged=False, context=0, Hq=24,
             Hkv=4, block=64, type="bf16"),
        # The 35B-shape chunk of a long prompt.
        dict(name="prefill 2048 at 30720", op="prefill", B=1, rows=2048, ragged=False, context=30720,
             Hq=16, Hkv=2, block=64, type="bf16"),
        # Chunks of several requests, odd lengths, behind what each holds.
        dict(name="prefill ragged 12x1501", op="prefill", B=12, rows=1501, ragged=True, context=9973,
             Hq=24, Hkv=4, block=16, type="fp16"),
        # The next turns of long conversations: few rows, many keys.
        dict(name="prefill turns 4x37 at 65000", op="prefill", B=4, rows=37, ragged=True, context=65000,
             Hq=16, Hkv=2, block=128, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "fork", "compact", "prefill", "prefill", "prefill"])
    block = rng.choice([16, 32, 64, 128])
    Hq, Hkv = rng.choice([(24, 4), (16, 2), (8, 8), (12, 3), (32, 8), (16, 1)])
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 24000), Hq=min(Hq, 24), Hkv=min(Hkv, 4),
                    rot=rng.choice([32, 64, 128, 256]), interleaved=rng.random() < 0.5,
                    fused=rng.random() < 0.5, far=_log(rng, 1, 1000000),
                    scale=rng.choice([1.0, 1.2]), type=rng.choice(["bf16", "fp16"]))
    if op == "fork":
        parents = rng.randint(1, 4)
        return dict(op=op, parents=parents, forks=_log(rng, parents, 192), len=_log(rng, 40, 24000),
                    block=block, Hkv=min(Hkv, 4))
    if op == "compact":
        return dict(op=op, B=_log(rng, 4, 256), max_len=_log(rng, 100, 6000), block=block,
                    Hkv=min(Hkv, 4))
    rows = _log(rng, 1, 4096)
    context = rng.choice([0, _log(rng, 1, 65000)])
    most = int(8e8 / (rows * (context + rows) * Hq))
    B = _log(rng, 1, max(1, min(32, most)))
    if most < 1:
        context = max(0, int(8e8 / (rows * Hq)) - rows)
    return dict(op=op, B=B, rows=rows, ragged=rng.random() < 0.5, context=context, Hq=Hq, Hkv=Hkv,
                block=block, type=rng.choice(["bf16", "fp16"]))


def _rows_and_contexts(case):
    """Rows and held keys of each sequence, by the case alone."""
    B = case["B"]
    if not case["ragged"]:
        return [case["rows"]] * B, [case["context"]] * B
    rows = [max(1, case["rows"] * (i + 1) // B) for i in range(B)]
    held = [case["context"] - case["context"] * ((5 * i) % B) // (2 * B) for i in range(B)]
    return rows, held


# ------------------------------------------------------------------------------- inputs

def _i32(x):
    return torch.as_tensor(x).to(device="cuda", dtype=torch.int32)


def _shuffled(n, cpu):
    return torch.randperm(n, generator=cpu)


def _codes(shape, gen):
    """Random e4m3 codes without NaN."""
    x = torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8, device="cuda")
    return torch.where((x & 0x7F) == 0x7F, x - 1, x).view(torch.float8_e4m3fn)


def _scales(shape, gen):
    return torch.exp2(torch.randint(-9, -3, shape, generator=gen, device="cuda").float())


def _filled(num_blocks, Hkv, bs, gen, outliers):
    """A pool of N(0, 1) rows (a hundredth of the rows times 8 where `outliers`), quantised a block
    and head at a time by the least power of two that holds it."""
    pool = torch.empty((num_blocks, Hkv, bs, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((num_blocks, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * bs * D))
    for i in range(0, num_blocks, step):
        n = min(step, num_blocks - i)
        x = torch.randn((n, Hkv, bs, D), generator=gen, device="cuda")
        if outliers:
            hit = torch.rand((n, Hkv, bs, 1), generator=gen, device="cuda") < 0.01
            x = torch.where(hit, x * 8, x)
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0)))
        pool[i : i + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
        scale[i : i + n] = s
    return pool, scale


def _tables(need, width, num_blocks, cpu):
    """Random disjoint blocks, need[b] of them for sequence b, and the stack of the free ones."""
    perm, used = _shuffled(num_blocks, cpu), int(need.sum())
    table = torch.full((len(need), width), -1, dtype=torch.int64)
    table[torch.arange(width)[None, :] < need[:, None]] = perm[:used]
    free = torch.full((num_blocks,), -1, dtype=torch.int64)
    free[: num_blocks - used] = perm[used:]
    return table, free


def _prepare_rope(case, cpu, gen, st):
    T, Hq, Hkv, t = case["T"], case["Hq"], case["Hkv"], _TYPES[case["type"]]
    if case["fused"]:    # one projection's output: q, k and v side by side
        x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen, device="cuda").to(t)
        st["q"], st["k"] = x[:, :Hq], x[:, Hq : Hq + Hkv]
    else:
        st["q"] = torch.randn((T, Hq, D), generator=gen, device="cuda").to(t)
        st["k"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").to(t)
    first = torch.randint(0, case["far"] + 1, (1,), generator=cpu) if case["far"] else torch.zeros(1)
    st["positions"] = _i32(first.long() + torch.arange(T))
    j = torch.arange(0, case["rot"], 2, dtype=torch.float64)
    st["inv_freq"] = (1e7 ** (-j / case["rot"])).float().cuda()


def _prepare_fork(case, cpu, gen, st):
    """Parents with their blocks, and children that the last pass forked from them."""
    P, F, bs = case["parents"], case["forks"], case["block"]
    B, width = P + F, -(-case["len"] // bs) + 2
    lens = torch.tensor([case["len"] - 3 * p for p in range(P)] + [0] * F)
    need = (lens + bs - 1) // bs
    num_blocks = int(need.sum()) + F + 5
    table, free = _tables(need, width, num_blocks, cpu)
    src = torch.arange(F) % P
    part = 0.75 + 0.25 * torch.rand(F, generator=cpu, dtype=torch.float64)
    fork_lens = (lens[src] * part).long().clamp(min=1)
    fork_lens = torch.where(fork_lens % bs == 0, fork_lens - 1, fork_lens).clamp(min=1)
    shares = torch.zeros(num_blocks, dtype=torch.int64)
    n_blocks, top = need.clone(), num_blocks - int(need.sum())
    for f in range(F):
        full = int(fork_lens[f]) // bs
        table[P + f, :full] = table[src[f], :full]
        shares[table[P + f, :full]] += 1
        table[P + f, full] = free[top - 1 - f]
        n_blocks[P + f] = full + 1
    st.update(src=_i32(src), dst=_i32(P + torch.arange(F)), fork_lens=_i32(fork_lens),
              ended=_i32(lens), kv_lens=_i32(torch.cat([lens[:P], fork_lens])),
              block_tables=_i32(table), n_blocks=_i32(n_blocks), free_list=_i32(free),
              free_count=_i32([top - F]), shares=_i32(shares))
    return num_blocks


def _prepare_compact(case, cpu, gen, st):
    """A pool after a while: random blocks, half of the requests ended, some blocks shared."""
    B, bs = case["B"], case["block"]
    lens = torch.tensor([max(1, case["max_len"] * (b + 1) // B) for b in range(B)])
    lens[::2] = 0
    need = (lens + bs - 1) // bs
    num_blocks = 2 * int(need.sum()) + 7
    table, free = _tables(need, -(-case["max_len"] // bs) + 1, num_blocks, cpu)
    shares = torch.zeros(num_blocks, dtype=torch.int64)
    n_blocks = need.clone()
    for b in range(0, B - 1, 8):     # ended ones whose places took a prefix of their neighbour's
        n = int(need[b + 1]) // 2
        table[b, :n] = table[b + 1, :n]
        shares[table[b, :n]] += 1
        n_blocks[b] = n
    st.update(block_tables=_i32(table), n_blocks=_i32(n_blocks), free_list=_i32(free),
              free_count=_i32([num_blocks - int(need.sum())]), shares=_i32(shares),
              live=int(need.sum()))
    return num_blocks


def _prepare_prefill(case, cpu, gen, st):
    bs, t = case["block"], _TYPES[case["type"]]
    rows, held = _rows_and_contexts(case)
    order = _shuffled(case["B"], cpu).tolist()
    rows, held = [rows[i] for i in order], [held[i] for i in order]
    lens = torch.tensor(rows) + torch.tensor(held)
    need = (lens + bs - 1) // bs
    num_blocks = int(need.sum()) + 3
    table, _ = _tables(need, int(need.max()) + 1, num_blocks, cpu)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    shape = (cu[-1], case["Hq"], D)
    st.update(rows=rows, lens=lens.tolist(), cu=cu, cu_rows=_i32(cu), kv_lens=_i32(lens),
              block_tables=_i32(table), max_rows=max(rows), max_kv_len=int(lens.max()))
    st["q"] = torch.randn(shape, generator=gen, device="cuda").to(t)
    st["g"] = (torch.randn(shape, generator=gen, device="cuda") * 2).to(t)
    st["out"] = torch.empty_like(st["q"])
    st["k_pool"], st["k_scale"] = _filled(num_blocks, case["Hkv"], bs, gen, True)
    st["v_pool"], st["v_scale"] = _filled(num_blocks, case["Hkv"], bs, gen, False)


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case, op=case["op"], bs=case.get("block"))
    if case["op"] == "rope":
        _prepare_rope(case, cpu, gen, st)
    elif case["op"] == "prefill":
        _prepare_prefill(case, cpu, gen, st)
    else:
        make = _prepare_fork if case["op"] == "fork" else _prepare_compact
        num_blocks = make(case, cpu, gen, st)
        for name in ("k", "v"):
            st[name + "_pool"] = _codes((num_blocks, case["Hkv"], st["bs"], D), gen)
            st[name + "_scale"] = _scales((num_blocks, case["Hkv"]), gen)
    return st


# ------------------------------------------------------------------------------- plain forms

def _rope_plain(st):
    case = st["case"]
    half = case["rot"] // 2
    a = st["positions"].double()[:, None] * st["inv_freq"].double()[None, :]
    c = (torch.cos(a) * case["scale"]).float()[:, None]
    s = (torch.sin(a) * case["scale"]).float()[:, None]

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            a, b = y[..., 0 : case["rot"] : 2], y[..., 1 : case["rot"] : 2]
            r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half : case["rot"]]
            r = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([r, y[..., case["rot"] :]], -1).to(x.dtype)

    return dict(q=turn(st["q"]), k=turn(st["k"]))


def _free_plain(st, lens):
    """Every sequence keeps the blocks of lens[b] keys; the rest lose an owner, and a block without
    one goes on the stack with its last entry in (sequence, place) order."""
    bs, table, n_blocks = st["bs"], st["block_tables"].long(), st["n_blocks"].long()
    free, fc, shares = st["free_list"].long(), st["free_count"].long(), st["shares"].long()
    N, n = free.numel(), table.numel()
    keep = torch.minimum((lens.long() + bs - 1) // bs, n_blocks)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    loose = ((col >= keep[:, None]) & (col < n_blocks[:, None])).reshape(-1)
    blk = torch.where(loose, table.reshape(-1), N)      # N: a place behind the pool
    left = torch.cat([shares, shares[:1]]).scatter_add(0, blk, -torch.ones_like(blk))
    entry = torch.arange(n, device="cuda")
    last = torch.full((N + 1,), -1, device="cuda").scatter_reduce(0, blk, entry, "amax")
    gone = loose & (left[blk] < 0) & (last[blk] == entry)
    rank, total = torch.cumsum(gone, 0) - 1, gone.sum()
    at = torch.where(gone, fc + total - 1 - rank, N)
    free = torch.cat([free, free[:1]]).scatter(0, at, blk)[:-1]
    st["free_list"].copy_(free)
    st["free_count"].copy_(fc + total)
    st["shares"].copy_(left[:-1].clamp(min=0))
    st["block_tables"].copy_(torch.where(loose, -1, table.reshape(-1)).view_as(table))
    st["n_blocks"].copy_(keep)


def _fork_plain(st):
    bs, table = st["bs"], st["block_tables"].long()
    src, dst, lens = st["src"].long(), st["dst"].long(), st["fork_lens"].long()
    full, rest = lens // bs, lens % bs
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    tail = rest > 0
    rank = torch.cumsum(tail, 0) - 1
    top = st["free_count"].long() - 1 - rank
    new = torch.where(tail, st["free_list"].long()[top.clamp(min=0)], -1)
    old = table[src, full.clamp(max=table.shape[1] - 1)]
    shared = col < full[:, None]
    rows = torch.where(shared, table[src], -1)
    N = st["shares"].numel()
    add = torch.cat([st["shares"].long(), torch.zeros(1, dtype=torch.int64, device="cuda")])
    add = add.scatter_add(0, torch.where(shared, rows, N).reshape(-1), shared.reshape(-1).long())
    table[dst] = torch.where((col == full[:, None]) & tail[:, None], new[:, None], rows)
    n_blocks, kv_lens = st["n_blocks"].long(), st["kv_lens"].long()
    n_blocks[dst] = full + tail
    kv_lens[dst] = lens
    st["block_tables"].copy_(table)
    st["n_blocks"].copy_(n_blocks)
    st["kv_lens"].copy_(kv_lens)
    st["shares"].copy_(add[:-1])
    st["free_count"].copy_(st["free_count"].long() - tail.sum())
    return torch.stack([torch.where(tail, old, -1), new, rest], 1).int()


def _copy_plain(st, copies):
    at, to, rows = copies.long().unbind(1)
    keep = torch.arange(st["bs"], device="cuda")[None, :] < rows[:, None]
    for name in ("k", "v"):
        pool, scale = st[name + "_pool"].view(torch.uint8), st[name + "_scale"]
        pool[to] = torch.where(keep[:, None, :, None], pool[at], pool[to])
        scale[to] = scale[at]


def _compact_plain(st):
    """Live blocks at or behind the number of live ones go to the free places before it, in order."""
    table, n_blocks = st["block_tables"].long(), st["n_blocks"].long()
    free, shares = st["free_list"].long(), st["shares"].long()
    N, device = free.numel(), free.device
    fc = st["free_count"].long()
    n = torch.arange(N, device=device)
    listed_free = torch.where(n < fc, free, N)
    is_free = torch.zeros(N + 1, dtype=torch.bool, device=device).scatter(0, listed_free, n >= 0)[:-1]
    low = n < N - fc
    hole, mover = is_free & low, ~is_free & ~low
    M = N // 2
    none = torch.full((M + 1,), -1, device=device)
    at = none.scatter(0, torch.where(mover, torch.cumsum(mover, 0) - 1, M), n)[:-1]
    to = none.scatter(0, torch.where(hole, torch.cumsum(hole, 0) - 1, M), n)[:-1]
    used = torch.arange(M, device=device) < hole.sum()
    copies = torch.stack([torch.where(used, at, -1), torch.where(used, to, -1),
                          torch.where(used, st["bs"], 0)], 1)
    index = torch.where(is_free, -1, n)
    index = torch.cat([index, index[:1]]).scatter(0, torch.where(used, at, N), to)[:-1]
    held = torch.arange(table.shape[1], device=device)[None, :] < n_blocks[:, None]
    tables = torch.where(held, index[table.clamp(min=0)], -1)
    moved = torch.zeros(N + 1, dtype=torch.int64, device=device)
    moved = moved.scatter(0, torch.where(index >= 0, index, N), shares)[:-1]
    return (tables.int(), (N - 1 - n).int(), moved.int(), index.int(), copies.int())


def _prefill_plain(st):
    case, bs = st["case"], st["bs"]
    Hkv, Hq = case["Hkv"], case["Hq"]
    outs = []
    for b, (r, L) in enumerate(zip(st["rows"], st["lens"])):
        pages = st["block_tables"][b, : -(-L // bs)].long()

        def cache(name):   # [Hkv, L, D] in float32
            x = st[name + "_pool"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
            x = x * st[name + "_scale"][pages][..., None, None]
            return x.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]

        q = st["q"][st["cu"][b] : st["cu"][b] + r].float()
        q = q.view(r, Hkv, Hq // Hkv, D).transpose(0, 1).reshape(Hkv, -1, D)
        s = (q @ cache("k").transpose(-1, -2) * (1.0 / 16.0)).view(Hkv, r, Hq // Hkv, L)
        ends = L - r + torch.arange(r, device="cuda") + 1
        unseen = torch.arange(L, device="cuda")[None, :] >= ends[:, None]
        s.masked_fill_(unseen[None, :, None, :], float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        del s
        total = p.sum(-1, keepdim=True)
        o = (p.view(Hkv, -1, L) @ cache("v")).view(Hkv, r, Hq // Hkv, D) / total
        outs.append(o.transpose(0, 1).reshape(r, Hq, D))
    o = torch.cat(outs)
    return (o / (1 + torch.exp(-st["g"].float()))).to(st["q"].dtype)


def _pools(st):
    return dict(k=st["k_pool"], v=st["v_pool"], k_scale=st["k_scale"], v_scale=st["v_scale"])


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "rope":
        return _rope_plain(st)
    if st["op"] == "prefill":
        return dict(out=_prefill_plain(st))
    if st["op"] == "fork":
        # the children of the last pass end, and as many new requests take their places
        _free_plain(st, st["ended"])
        copies = _fork_plain(st)
        _copy_plain(st, copies)
        return dict(copies=copies, tables=st["block_tables"], n_blocks=st["n_blocks"],
                    kv_lens=st["kv_lens"], free_list=st["free_list"],
                    free_count=st["free_count"], shares=st["shares"], **_pools(st))
    tables, free_list, shares, index, copies = _compact_plain(st)
    at, to, rows = copies.long().unbind(1)
    keep = to >= 0
    _copy_plain(st, copies[keep])
    return dict(tables=tables, free_list=free_list, shares=shares, index=index, copies=copies,
                **_pools(st))


def _run_own(st):
    import gqa_head_gated_gb300 as G
    if st["op"] == "rope":
        case = st["case"]
        q, k = G.rope(st["q"], st["k"], st["positions"], st["inv_freq"],
                      interleaved=case["interleaved"], scale=case["scale"])
        return dict(q=q, k=k)
    pools = (st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"])
    if st["op"] == "fork":
        G.block_free(st["ended"], st["block_tables"], st["n_blocks"], st["free_list"],
                     st["free_count"], st["shares"], st["bs"])
        copies = G.block_fork(st["src"], st["dst"], st["fork_lens"], st["kv_lens"],
                              st["block_tables"], st["n_blocks"], st["free_list"],
                              st["free_count"], st["shares"], st["bs"])
        G.kv8_copy(copies, *pools)
        return dict(copies=copies, tables=st["block_tables"], n_blocks=st["n_blocks"],
                    kv_lens=st["kv_lens"], free_list=st["free_list"],
                    free_count=st["free_count"], shares=st["shares"], **_pools(st))
    if st["op"] == "compact":
        tables, free_list, shares, index, copies = G.block_compact(
            st["block_tables"], st["n_blocks"], st["free_list"], st["free_count"], st["shares"],
            st["bs"])
        G.kv8_copy(copies, *pools)
        return dict(tables=tables, free_list=free_list, shares=shares, index=index, copies=copies,
                    **_pools(st))
    if "workspace" not in st:
        st["workspace"] = torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8,
                                      device="cuda")
    return dict(out=G.kv8_prefill(st["q"], *pools, st["g"], st["block_tables"], st["kv_lens"],
                                  st["cu_rows"], max_rows=st["max_rows"],
                                  max_kv_len=st["max_kv_len"], workspace=st["workspace"],
                                  out=st["out"]))


# ------------------------------------------------------------------------------- work, 64 bits

def work(case):
    op = case["op"]
    if op == "rope":
        heads = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": float(heads * D * 4 + case["T"] * 4 + case["rot"] * 2),
                "flops": 3.0 * heads * case["rot"]}
    block_bytes = 2 * case["Hkv"] * (case["block"] * D + 4)
    if op == "fork":
        entries = case["forks"] * case["len"] * 0.875 / case["block"]
        # freed and forked: a table's entries out and in and its blocks' counts, twice; tails half
        # full on average
        return {"bytes": float(2 * 4 * 4 * entries + case["forks"] * block_bytes), "flops": 0.0}
    if op == "compact":
        blocks = case["B"] / 2 * case["max_len"] / 2 / case["block"]   # live; half of them move
        N = 2 * blocks
        table = case["B"] * (case["max_len"] / case["block"] + 1)
        return {"bytes": float(2 * 4 * table + 4 * 7 * N + blocks * block_bytes), "flops": 0.0}
    rows, held = _rows_and_contexts(case)
    pairs = sum(r * h + r * (r + 1) / 2 for r, h in zip(rows, held))
    keys = sum(rows) + sum(held)
    return {"bytes": float(keys * case["Hkv"] * (2 * D + 8 / case["block"])
                           + 3 * 2 * sum(rows) * case["Hq"] * D),
            "flops": 4.0 * D * case["Hq"] * pairs}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    st = prepare(case, seed)
    if case["op"] == "rope":
        out = {}
        angle = torch.outer(st["positions"].double(), st["inv_freq"].double())
        turn = torch.polar(torch.full_like(angle, case["scale"]), angle)[:, None, :]
        for name in ("q", "k"):
            x, n = st[name].double(), case["rot"]
            y = x.clone()
            if case["interleaved"]:
                z = torch.complex(x[..., 0:n:2], x[..., 1:n:2]) * turn
                y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
            else:
                z = torch.complex(x[..., : n // 2], x[..., n // 2 : n]) * turn
                y[..., : n // 2], y[..., n // 2 : n] = z.real, z.imag
            out[name] = y
        return out
    out = torch.empty_like(st["q"], dtype=torch.float64)
    group, bs = case["Hq"] // case["Hkv"], case["block"]
    for b in range(case["B"]):
        L, r, t0 = st["lens"][b], st["rows"][b], st["cu"][b]
        pages = st["block_tables"][b, : -(-L // bs)].long()
        row = torch.arange(r, device="cuda")[:, None]
        hidden = torch.arange(L, device="cuda")[None, :] > L - r + row
        for h in range(case["Hq"]):
            k, v = ((st[n + "_pool"].view(torch.uint8)[pages, h // group].view(torch.float8_e4m3fn).double()
                     * st[n + "_scale"][pages, h // group].double()[:, None, None]).reshape(-1, D)[:L]
                    for n in ("k", "v"))
            s = st["q"][t0 : t0 + r, h].double() @ k.T / math.sqrt(D)
            w = torch.softmax(s.masked_fill_(hidden, float("-inf")), -1)
            out[t0 : t0 + r, h] = w @ v
    return dict(out=out * torch.sigmoid(st["g"].double()))
