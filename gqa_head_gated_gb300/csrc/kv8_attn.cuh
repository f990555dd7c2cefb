// Pieces shared by the attention kernels over the paged 8-bit cache (kv8_attn.cu: few rows,
// kv8_wide.cu: many): the schedule, the warp that copies the cache, and its rings.
//
// The key tiles of all (sequence, KV head, row block) segments are laid end to end and cut
// into equal contiguous shares, one per CTA, so ragged lengths cost no tail; the copies run
// ahead across segments.  A share that crosses segments writes one part per piece.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "kv8_attn.h"
#include "kv8_common.cuh"
#include "ptx_sm100.cuh"
#include "tc_common.cuh"

namespace gqa {
namespace {

constexpr int kTile = 128;                       // keys per tile
constexpr int kHalfBytes = kTile * 128;          // 128 keys x 128 dims of K or V
constexpr int kSlotBytes = 2 * kHalfBytes;
constexpr int kScaleRing = 8;      // tiles whose scales are held: see the copies
constexpr int kPieceRing = 8;      // pieces whose descriptions are held: see the copies
// What going on to another segment costs a CTA, in tiles (its end and start, and the first
// tiles, whose references still move), where shares have kLongShare tiles or more (with short
// ones it would only unsettle them: one tile each is best then).  Swept over 1, 3, 5, 7, 9 and
// 12: 16 x 32768 decode (16 rows) 92.2, 89.4, 89.9, 90.7, 90.3, 90.3 us, and over 3, 4 and 5: 88.3,
// 88.6, 88.8 (2 x 131071: 52.8 with each); over 3, 6, 9 and 12:
// chain verify (24 rows) 78.6, 75.5, 74.0, 74.8; over 3, 5 and 8: tree verify (128 rows) 149.8,
// 147.8, 149.4.
template <int MB>
constexpr uint32_t switch_tiles() { return MB == 16 ? 4 : MB <= 32 ? 9 : 5; }
constexpr uint32_t kLongShare = 8;
constexpr int kMaxTileBlocks = kTile / 16;
// Pieces whose rows, limits and masks are held.  prepare() of piece n may run while another
// group still writes the parts of piece n - 2 (a piece n - 1 of one tile makes no group wait for
// the others), but not those of n - 3, which come before the group's tiles of n - 2.  So three
// would do; a power of two keeps the remainder cheap (tree verify 195 us with 3, 172 with 4).
constexpr uint32_t kRowSets = 4;
constexpr float kLSlack = 64.f;    // l's terms stay below 2^64
constexpr int kLongPiece = 64;     // tiles from which on p's references may go down again
constexpr float kNone = -3.0e38f;  // reference of a row that has seen no key

// A run of key tiles of one segment that one CTA takes.
struct Piece {
  int b, g, rb, s;            // sequence, KV head, row block, part (-1: nothing is written)
  int rows, t0, kv_len;       // of the sequence
  int k_lo, k_hi, n_tiles;    // keys that some row of the block sees; 0 tiles: the share's end
};

// The shared memory of the schedule and the copies.
template <int KS, int VS>
struct RingSmem {
  uint8_t k[KS][kSlotBytes];
  uint8_t v[VS][kSlotBytes];
  float scale[kScaleRing][2][kMaxTileBlocks];
  uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS];
  uint64_t sc_full[kScaleRing];
  uint64_t piece_full[kPieceRing];
  Piece piece[kPieceRing];
  int4 seq[kKv8Seqs];                      // first token, rows, keys, tiles
  uint32_t base[kKv8Seqs + 1];             // first position of each sequence's segments
  uint32_t segs[kKv8Seqs + 1];             // segments before each sequence
  uint32_t tmem_base;
  int most;                                // tiles of the longest sequence
  int abort, zero;
};

// This CTA's share [pos, end) of the launch's positions, cut into n_cta shares.
struct Share {
  uint32_t pos, end, n_cta, lead;   // lead: positions of a segment before its tiles
};

// ptx::mbar_wait with the polling loop out of line: the kernel has many waits, and its code
// has to stay small (inlined, they made it 114 KB, whose instruction fetches took thousands
// of cycles wherever a path had not run for a while).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, uint64_t tmo, int* abort) {
  return ptx::mbar_wait(bar, parity, tmo, abort);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint64_t tmo, int* abort) {
  return ptx::mbar_try_wait(ptx::smem_addr(bar), parity) || wait_slow(bar, parity, tmo, abort);
}

// The piece of this CTA's share [.., end) that starts at position `pos`, which moves on behind
// it.  A segment takes `lead` positions before those of its tiles: a CTA that goes on to it
// from another has that much less to do.  `last`: the piece ends its segment.  False: the
// piece has no position of a tile.
template <int MB>
__device__ __forceinline__ bool piece_at(const Kv8AttnArgs& p, const int4* seqs, const uint32_t* base,
                                         uint32_t& pos, const Share& share, Piece& x, bool& last) {
  const uint32_t end = share.end;
  int lo = 0, hi = p.B - 1;   // last sequence that starts at or before pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  const int4 q = seqs[lo];
  x.b = lo;
  x.t0 = q.x;
  x.rows = q.y;
  x.kv_len = q.z;
  const uint32_t len = uint32_t(q.w) + share.lead, n_rb = uint32_t((x.rows * p.gqa + MB - 1) / MB);
  const uint32_t seg = (pos - base[lo]) / len;
  x.g = int(seg / n_rb);
  x.rb = int(seg - uint32_t(x.g) * n_rb);
  const uint32_t start = base[lo] + seg * len, first = start + share.lead;
  const uint32_t from = max(pos, first);
  last = end >= start + len;
  pos = min(end, start + len);
  if (pos <= from) return false;
  // the piece's part: this CTA's place among those that have tiles of the segment
  x.s = 0;
  if (from != first) {
    const unsigned long long W = base[p.B];
    x.s = int(blockIdx.x) - int(((first + 1ull) * share.n_cta - 1) / W);
  }
  x.k_lo = int(from - first) * kTile;
  x.k_hi = x.kv_len;          // a tree row may see up to the last key
  if (p.tree_mask == nullptr) {
    const int last_row = min(x.rows * p.gqa - 1, x.rb * MB + MB - 1) / p.gqa;
    x.k_hi = x.kv_len - x.rows + last_row + 1;
  }
  if (!last) x.k_hi = min(x.k_hi, int(pos - first) * kTile);
  x.n_tiles = x.k_hi > x.k_lo ? (x.k_hi - x.k_lo + kTile - 1) / kTile : 0;
  return true;
}

// log2 of a scale, exactly where it is a normal power of two; 0 gives -inf.  Without a branch.
__device__ __forceinline__ float log2_scale(float s) {
  const uint32_t b = __float_as_uint(s);
  const float e = float(int(b >> 23) - 127), l = __log2f(s);
  return (b & 0x7FFFFFu) == 0u && b - 0x00800000u < 0x7F000000u ? e : l;
}

// Bytes of a 16-byte chunk that are e4m3 NaN become 0; returns whether there was one.
__device__ __forceinline__ bool clear_nan8(uint4& u) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = __vcmpeq4(w[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    w[i] &= ~m;
    any |= m;
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  return any != 0u;
}

// 16-byte chunks c0 .. c1 - 1 of the V row of one key of a landed tile: zeroed, or their NaN
// codes taken out.
__device__ __noinline__ bool clean_v_row(uint8_t* slot, int row, bool zero, int c0 = 0,
                                          int c1 = 16) {
  bool hit = false;
  for (int c = c0; c < c1; ++c) {
    uint4* const a = reinterpret_cast<uint4*>(slot + (c >> 3) * kHalfBytes + row * 128 +
                                              (((c & 7) ^ (row & 7)) << 4));
    if (zero) {
      *a = make_uint4(0u, 0u, 0u, 0u);
    } else {
      uint4 u = *a;
      if (clear_nan8(u)) {
        *a = u;
        hit = true;
      }
    }
  }
  return hit;
}

// Two values to e4m3, and what they leave: (lo, hi) becomes (x - e4m3(x)) * step.
__device__ __forceinline__ uint32_t take_term(float& lo, float& hi, float step) {
  const uint32_t t = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
  const float2 f = from_e4m3x2(t);
  lo = (lo - f.x) * step;
  hi = (hi - f.y) * step;
  return t;
}

// A row's output of one dim: NaN when a key that it sees had a NaN there (`hits`: keys from
// pr_lo on whose V rows had NaN codes taken out).
__device__ __noinline__ float put_back_nan(const Kv8AttnArgs& p, int b, int g,
                                           unsigned long long hits, int pr_lo, int lim, bool tree,
                                           int base, unsigned long long mask, int dim, float o) {
  for (; hits != 0ull; hits &= hits - 1ull) {
    const int key = pr_lo + __ffsll(static_cast<long long>(hits)) - 1;
    if (key >= lim || (tree && key >= base && !((mask >> (key - base)) & 1ull))) continue;
    const int blk = __ldg(p.tables + (long long)b * p.max_blocks + (key >> p.bs_log2));
    if (blk < 0 || blk >= p.num_blocks) continue;
    const size_t row = ((size_t(blk) * p.Hkv + g) << p.bs_log2) + (key & ((1 << p.bs_log2) - 1));
    if ((p.v_pool[row * 256 + dim] & 0x7Fu) == 0x7Fu) o = __int_as_float(0x7FC00000);
  }
  return o;
}

// One thread: the rings' barriers and flags.
template <int KS, int VS>
__device__ __forceinline__ void init_ring(RingSmem<KS, VS>& sm) {
  for (int i = 0; i < KS; ++i) {
    ptx::mbar_init(&sm.k_full[i], 1);
    ptx::mbar_init(&sm.k_empty[i], 1);
  }
  for (int i = 0; i < VS; ++i) {
    ptx::mbar_init(&sm.v_full[i], 1);
    ptx::mbar_init(&sm.v_empty[i], 1);
  }
  for (int i = 0; i < kScaleRing; ++i) ptx::mbar_init(&sm.sc_full[i], 32);
  for (int i = 0; i < kPieceRing; ++i) ptx::mbar_init(&sm.piece_full[i], 1);
  sm.base[0] = 0;
  sm.most = 0;
  sm.abort = 0;
  sm.zero = 0;
}

// All threads, after init_ring and a barrier: waits for the launch's inputs, lays the
// segments out and cuts this CTA's share.
template <int MB, int KS, int VS>
__device__ __forceinline__ Share cut_shares(RingSmem<KS, VS>& sm, const Kv8AttnArgs& p) {
  const int tid = threadIdx.x, lane = tid & 31;
  wait_for_last();
  let_next_start();   // not before: the merge reads lengths and gate ahead of its own wait
  // All of Q is on its way to L2 while the shares are cut (a piece's start reads its rows).
  if (p.b0 == 0) {
    const size_t lines = size_t(p.T) * p.Hq * 4;   // 128 bytes each
    for (size_t i = size_t(blockIdx.x) * blockDim.x + tid; i < lines && i < (size_t(1) << 17);
         i += size_t(gridDim.x) * blockDim.x)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + i * 8));
  }
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int kv = p.kv_lens[b], t0 = p.cu_rows ? p.cu_rows[b] : p.b0 + b;
    const int rows = p.cu_rows ? p.cu_rows[b + 1] - t0 : 1;
    const bool ok = rows >= 0 && rows <= p.max_rows && t0 >= 0 && rows <= p.T - t0 && kv >= rows &&
                    kv <= p.max_kv_len;
    const int tiles = ok && rows > 0 ? (kv + kTile - 1) / kTile : 0;
    sm.seq[b] = make_int4(t0, rows, kv, tiles);
    const uint32_t segs = tiles > 0 ? uint32_t(p.Hkv) * uint32_t((rows * p.gqa + MB - 1) / MB) : 0u;
    sm.base[b + 1] = uint32_t(tiles) * segs;
    sm.segs[b + 1] = segs;
    if (tiles > 0) atomicMax(&sm.most, tiles);
    if (!ok && blockIdx.x == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
  __syncthreads();
  Share x{0, 0, 0, 0};
  if (tid < 32) {   // inclusive sums over the sequences, 32 at a time
    uint32_t run = 0, runs = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      uint32_t v = b0 + lane < p.B ? sm.base[b0 + lane + 1] : 0u;
      uint32_t w = b0 + lane < p.B ? sm.segs[b0 + lane + 1] : 0u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o), t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) {
          v += u;
          w += t;
        }
      }
      if (b0 + lane < p.B) {
        sm.base[b0 + lane + 1] = run + v;
        sm.segs[b0 + lane + 1] = runs + w;
      }
      run += __shfl_sync(0xffffffffu, v, 31);
      runs += __shfl_sync(0xffffffffu, w, 31);
    }
    // (this warp's own writes) each sequence's leads go before its tiles
    __syncwarp();
    if (run >= kLongShare * gridDim.x)
      for (int b = lane; b < p.B; b += 32) sm.base[b + 1] += switch_tiles<MB>() * sm.segs[b + 1];
  }
  __syncthreads();
  const uint32_t W = sm.base[p.B];
  x.lead = W > 0 && W >= kLongShare * gridDim.x + switch_tiles<MB>() * sm.segs[p.B] ? switch_tiles<MB>() : 0;
  x.n_cta = min(gridDim.x, W);
  // Shares so long that no segment needs more than `parts` parts.
  if (sm.most > p.parts)
    x.n_cta = min(x.n_cta, max(1u, uint32_t((unsigned long long)W * uint32_t(p.parts - 2) /
                                            uint32_t(sm.most))));
  if (blockIdx.x < x.n_cta) {
    x.pos = uint32_t((unsigned long long)W * blockIdx.x / x.n_cta);
    x.end = uint32_t((unsigned long long)W * (blockIdx.x + 1) / x.n_cta);
  }
  return x;
}

// The copying warp: publishes the share's pieces, copies their tiles and scales, marks parts
// that no row sees, and counts each segment's parts.
//
// A tile's scales live in a ring of kScaleRing tiles without a release: tile J + 8 is copied
// only once S of tile J + 8 - KS >= J + 5 was issued, which waits for the softmax of tile
// J + 3, so tile J's scales have been read.  So with the pieces' descriptions: a piece has a
// tile at least, so that when piece n + 8 is published the softmax has passed tiles of piece
// n + 8 - KS - 3 and with it piece n.
//
// kLead: V of a tile is copied behind K of the next one, for a kernel whose products of scores
// run further ahead than its V slots do (tree verify 158.6 us without, 156.3 with).
template <int MB, bool kLead, int KS, int VS>
__device__ __forceinline__ void copy_role(RingSmem<KS, VS>& sm, const Kv8AttnArgs& p,
                                          const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const Share& share) {
  static_assert(kScaleRing >= KS + 3 && kPieceRing >= KS + 4, "rings");
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.ctl.timeout_ns;
  const int bs = 1 << p.bs_log2, per_tile = kTile >> p.bs_log2;
  uint32_t J = 0;
  bool ok = true;
  if (lane == 0) {
    ptx::prefetch_tmap(&tmK);
    ptx::prefetch_tmap(&tmV);
  }
  uint32_t n_pieces = 0;
  // V of tile n, a block of this lane's from map row `row`, `bytes` in all
  uint32_t n_v = 0;      // tiles whose V copies are issued
  int v_row = 0;
  uint32_t v_bytes = 0;
  bool v_mine = false;
  const auto copy_v = [&]() -> bool {
    const uint32_t vs = n_v % VS;
    int go = 1;
    if (lane == 0) {
      if (n_v >= VS) go = wait(&sm.v_empty[vs], (n_v / VS - 1) & 1u, tmo, &sm.abort);
      if (go) ptx::mbar_arrive_expect_tx(&sm.v_full[vs], v_bytes);
    }
    if (__shfl_sync(0xffffffffu, go, 0) == 0) return false;
    if (v_mine) {
      uint8_t* const d = sm.v[vs] + lane * bs * 128;
      ptx::tma_load_2d(d, &tmV, &sm.v_full[vs], 0, v_row);
      ptx::tma_load_2d(d + kHalfBytes, &tmV, &sm.v_full[vs], 128, v_row);
    }
    ++n_v;
    return true;
  };
  const auto publish = [&](const Piece& x) {
    if (lane == 0) {
      sm.piece[n_pieces % kPieceRing] = x;
      ptx::mbar_arrive(&sm.piece_full[n_pieces % kPieceRing]);
    }
    ++n_pieces;
  };
  for (uint32_t pos = share.pos; ok && pos < share.end;) {
    Piece x;
    bool last;
    if (!piece_at<MB>(p, sm.seq, sm.base, pos, share, x, last)) continue;
    if (x.s < 0 || x.s >= p.parts) {   // never, with shares as cut above
      if (lane == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
      x.s = -1;
    }
    const int n_rows = min(MB, x.rows * p.gqa - x.rb * MB);
    for (int r = lane; r < n_rows; r += 32) {
      const int pp = x.rb * MB + r, i = pp / p.gqa;
      const size_t row = size_t(x.t0 + i) * p.Hq + x.g * p.gqa + (pp - i * p.gqa);
      if (x.n_tiles == 0 && x.s >= 0)   // no row of the block sees a key of the piece
        p.lse_parts[size_t(x.s) * size_t(p.T) * p.Hq + row] = -INFINITY;
      for (int c = 0; c < 4; ++c)       // Q's rows, which the piece's start will wait for
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + row * 32 + c * 8));
    }
    if (last && lane == 0 && x.s >= 0)
      p.n_parts[(size_t(p.b0 + x.b) * p.Hkv + x.g) * p.max_rb + x.rb] = x.s + 1;
    if (x.n_tiles == 0) continue;
    publish(x);
    const int* const table = p.tables + (long long)x.b * p.max_blocks;
    int at = x.k_lo + lane * bs;   // first key of this lane's block
    int blk = lane < per_tile && at < x.k_hi ? __ldg(table + (at >> p.bs_log2)) : 0;
    for (int j = 0; ok && j < x.n_tiles; ++j) {
      const bool mine = lane < per_tile && at < x.k_hi;
      const bool in = blk >= 0 && blk < p.num_blocks;
      if (mine && !in) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
      // a block outside the pool: past the map's last row, which copies zeros
      const int row = in ? (blk * p.Hkv + x.g) << p.bs_log2 : (p.num_blocks * p.Hkv) << p.bs_log2;
      const uint32_t bytes = uint32_t(__popc(__ballot_sync(0xffffffffu, mine))) * uint32_t(bs) * 256u;
      const int cur = blk;
      at += kTile;
      blk = lane < per_tile && at < x.k_hi ? __ldg(table + (at >> p.bs_log2)) : 0;
      const uint32_t ks = J % KS;
      int go = 1;
      if (lane == 0) {
        if (J >= KS)
          go = wait(&sm.k_empty[ks], (J / KS - 1) & 1u, tmo, &sm.abort);
        if (go) ptx::mbar_arrive_expect_tx(&sm.k_full[ks], bytes);
      }
      ok = __shfl_sync(0xffffffffu, go, 0) != 0;
      if (!ok) break;
      if (mine) {
        uint8_t* const d = sm.k[ks] + lane * bs * 128;
        ptx::tma_load_2d(d, &tmK, &sm.k_full[ks], 0, row);
        ptx::tma_load_2d(d + kHalfBytes, &tmK, &sm.k_full[ks], 128, row);
        const size_t sc = size_t(in ? cur : 0) * p.Hkv + x.g;
        ptx::cp_async4(ptx::smem_addr(&sm.scale[J % kScaleRing][0][lane]), p.k_scale + sc, in ? 4u : 0u);
        ptx::cp_async4(ptx::smem_addr(&sm.scale[J % kScaleRing][1][lane]), p.v_scale + sc, in ? 4u : 0u);
      }
      ptx::cp_async_mbar_arrive(&sm.sc_full[J % kScaleRing]);
      ++J;   // (K of this tile is on its way)
      if (kLead && J > 1) ok = copy_v();
      v_row = row;
      v_bytes = bytes;
      v_mine = mine;
      if (!kLead) ok = copy_v();
    }
  }
  if (kLead && ok && J > 0) ok = copy_v();
  if (ok) {
    Piece none{};
    publish(none);   // (the share's end: no tiles)
  }
  if (!ok && lane == 0) {
    sm.abort = 1;
    record_status(p.ctl.status, GQA_ERR_TIMEOUT);
  }
  ptx::cp_async_wait_all();
  if (lane == 0) {   // every copy has landed before the CTA ends
    for (uint32_t c = J - min(J, uint32_t(KS)); c < J; ++c)
      wait(&sm.k_full[c % KS], (c / KS) & 1u, tmo, &sm.zero);
    for (uint32_t c = n_v - min(n_v, uint32_t(VS)); c < n_v; ++c)
      wait(&sm.v_full[c % VS], (c / VS) & 1u, tmo, &sm.zero);
  }
  __syncwarp();
}

bool encode_pool(EncodeTiledFn fn, CUtensorMap* map, const void* pool, const Kv8AttnArgs& a) {
  const cuuint64_t dims[2] = {256, cuuint64_t(a.num_blocks) * cuuint64_t(a.Hkv) << a.bs_log2};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {128, cuuint32_t(1) << a.bs_log2};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_pools(CUtensorMap* tmK, CUtensorMap* tmV, const Kv8AttnArgs& a) {
  EncodeTiledFn fn = get_encode_fn();
  return fn != nullptr && encode_pool(fn, tmK, a.k_pool, a) && encode_pool(fn, tmV, a.v_pool, a);
}

}  // namespace
}  // namespace gqa
