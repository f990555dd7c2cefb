"""Paged 8-bit caches for the tests: random disjoint blocks, on the CPU."""
import numpy as np
import torch

import oracle

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def f8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).to(DEV)


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def random_codes(shape, gen):
    """Codes of N(0, 1) values times 64, without NaN: a usual block under its scale."""
    x = torch.randn(shape, generator=gen) * 64
    return oracle.e4m3_encode(x.double().clamp(-448, 448).numpy())


class Cache:
    """B sequences of kv_lens keys in random blocks of one pool; `spare` blocks are free.
    Blocks' rows past a length, and the free blocks, hold NaN."""

    def __init__(self, kv_lens, Hkv, bs, seed, room=0, spare=3, scale_exps=(-7, -5)):
        gen = torch.Generator().manual_seed(seed)
        self.bs, self.Hkv, self.lens = bs, Hkv, list(kv_lens)
        need = [-(-(n + room) // bs) for n in kv_lens]
        self.N = sum(need) + spare
        perm = torch.randperm(self.N, generator=gen).tolist()
        self.max_blocks = max(max(need), 1) + 1
        self.tables, at = [], 0
        for n in need:
            self.tables.append(perm[at:at + n] + [-1] * (self.max_blocks - n))
            at += n
        self.k, self.v = (np.full((self.N, Hkv, bs, 256), 0x7F, dtype=np.uint8) for _ in "kv")
        lo, hi = scale_exps
        self.ks, self.vs = (2.0 ** torch.randint(lo, hi + 1, (self.N, Hkv), generator=gen).double().numpy()
                            for _ in "kv")
        for b, n in enumerate(kv_lens):
            for j in range(0, n, bs):
                m = min(bs, n - j)
                for pool in (self.k, self.v):
                    pool[self.tables[b][j // bs], :, :m] = random_codes((Hkv, m, 256), gen)

    def device(self):
        """k_pool, v_pool, k_scale, v_scale, block_tables on the GPU."""
        return (f8(self.k), f8(self.v), torch.from_numpy(self.ks).float().to(DEV),
                torch.from_numpy(self.vs).float().to(DEV), i32(self.tables))

    def contiguous(self):
        return (oracle.kv8_contiguous(self.k, self.ks, self.tables, self.lens, self.bs),
                oracle.kv8_contiguous(self.v, self.vs, self.tables, self.lens, self.bs))


def rows_qg(T, Hq, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    q = torch.randn(T, Hq, 256, generator=gen).to(dtype)
    g = (torch.randn(T, Hq, 256, generator=gen) * 2).to(dtype)
    return q, g


def cu_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist()
