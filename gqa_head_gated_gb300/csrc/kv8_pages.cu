// Blocks that sequences share: forking a sequence's prefix, freeing, compacting the pool, and copying blocks.
//
// shares[n] counts the tables that hold block n beside the first, so a block that one table holds has 0 and
// block_plan, which hands blocks out and takes back those of one owner, knows nothing of it.
//
//   fork    table[dst][i] = table[src][i], shares + 1, for the full blocks of the prefix; the rows behind them go to
//           a block of the child's own, whose copy is listed
//   free    entries behind ceil(len / bs) lose an owner; a block that has none left goes on the stack, with the last
//           of its entries: the k-th of R such in (sequence, place) order to free_list[fc + R - 1 - k]
//   compact live blocks n >= L (L of them in all) take the free places below L, in order; tables, counts and stack
//           name the new places
//   copy    rows of listed blocks, K and V of every head, with their scales
//
// The first three are integers, bound by latency: one cluster each (compaction's tables, which are large, go to a
// second kernel over the whole GPU), whose barriers keep the steps apart.  A freed block's last entry is found with
// two rounds of atomics on its own count: all entries take one off, and where that leaves it below 0, the largest
// rank among them wins it; results do not hang on the atomics' order.  The copies are bound by memory.
// Measured: 192 forks of 281 to 375 blocks freed, forked and copied again 42 us repeated, the kernels alone and cold 31, 17
// and 7; 8 forks of up to 31 blocks cold 8, 6 and 4.  Compaction of 48,000 places 22 us, its 12,000 copies of 32 KB 117
// (98 % of the copy rate).
#include <cuda_runtime.h>

#include <initializer_list>

#include "kv8_common.cuh"
#include "kv8_scan.cuh"
#include "ptx_sm100.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCtas = 8;       // the portable cluster size
constexpr int kMaxSeqs = 8192;    // sequences, and forks, of a call
constexpr int kWon = 1 << 30;     // entries are fewer
// Entries that a thread has on their way together: entry k0 + kThreads u + tid of a tile is its u-th.  One CTA has few
// (kernels this short are bound by fetching their code: a free of 350 entries 7 us with 4, 16 with 16), a
// cluster many.
constexpr int kFew = 4, kMany = 16;

struct PagesParams {
  const int* src;
  const int* dst;
  const int* lens;
  int* kv_lens;
  int* tables;
  int* n_blocks;
  int* free_list;
  int* free_count;
  int* shares;
  int* copies;
  int F, B, max_blocks, num_blocks, bs_log2;
  LaunchCtl ctl;
};

// Owners of this thread's entries of the tile at k0 (by their exclusive sums, n of them), searched side by side.
template <int kRun>
__device__ __forceinline__ void owners(const int* sums, int n, int k0, int (&b)[kRun]) {
#pragma unroll
  for (int u = 0; u < kRun; ++u) b[u] = 0;
#pragma unroll 1
  for (int s = 1 << (31 - __clz(n)); s > 0; s >>= 1)
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int c = b[u] + s;
      if (c < n && sums[c] <= k0 + kThreads * u + int(threadIdx.x)) b[u] = c;
    }
}

template <int kRun>
__global__ void __launch_bounds__(kThreads, 1) block_fork_kernel(const PagesParams p) {
  constexpr int kTile = kThreads * kRun;
  extern __shared__ int smem[];
  __shared__ int2 part[kThreads / 32];
  int* const s_use = smem;             // B: 1 where it is forked from, + 2 per fork to it
  int* const s_full = s_use + p.B;     // F: full blocks of the prefix, then their exclusive sums
  int* const s_tail = s_full + p.F;    // F: whether rows are left, then those before
  int* const s_len = s_tail + p.F;     // F: keys of the prefix, -1 for a fork that is refused
  const int tid = threadIdx.x, cta = blockIdx.x, per = gridDim.x * kThreads, bs = 1 << p.bs_log2;
  let_next_start();
  for (int b = tid; b < p.B; b += kThreads) s_use[b] = 0;
  __syncthreads();
  wait_for_last();
  for (int f = tid; f < p.F; f += kThreads) {
    const int s = p.src[f], d = p.dst[f];
    if (s >= 0 && s < p.B) atomicOr(&s_use[s], 1);
    if (d >= 0 && d < p.B) atomicAdd(&s_use[d], 2);
  }
  __syncthreads();
  const int fc_read = *p.free_count, fc = min(max(fc_read, 0), p.num_blocks);
  for (int f = tid; f < p.F; f += kThreads) {
    const int s = p.src[f], d = p.dst[f];
    bool ok = s >= 0 && s < p.B && d >= 0 && d < p.B && s_use[d] == 2;
    int len = 0;
    if (ok) {
      const int held = p.kv_lens[s], have = p.n_blocks[s];
      len = p.lens != nullptr ? p.lens[f] : held;
      const long long need = ((long long)len + bs - 1) >> p.bs_log2;
      ok = len >= 0 && len <= held && need <= have && have <= p.max_blocks && p.n_blocks[d] == 0;
    }
    s_full[f] = ok ? len >> p.bs_log2 : 0;
    s_tail[f] = ok && (len & (bs - 1)) != 0;
    s_len[f] = ok ? len : -1;
    if (!ok && cta == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
  __syncthreads();
  const int2 total = scan2<kThreads>(s_full, s_tail, p.F, part);
  ptx::cluster_sync();   // every CTA has read what is changed from here on
  // a fork whose own block the stack has not got takes nothing
  const auto served = [&](int f) {
    return s_len[f] >= 0 && ((s_len[f] & (bs - 1)) == 0 || s_tail[f] < fc);
  };
  for (int k0 = cta * kTile; k0 < total.x; k0 += int(gridDim.x) * kTile) {
    int blk[kRun];
    int* to[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) to[u] = nullptr;
    int f[kRun];
    owners(s_full, p.F, k0, f);
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int k = k0 + kThreads * u + tid;
      if (k >= total.x || !served(f[u])) continue;
      const int i = k - s_full[f[u]];
      blk[u] = p.tables[(long long)p.src[f[u]] * p.max_blocks + i];
      to[u] = p.tables + (long long)p.dst[f[u]] * p.max_blocks + i;
    }
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (to[u] == nullptr) continue;
      *to[u] = blk[u];
      if (blk[u] >= 0 && blk[u] < p.num_blocks) atomicAdd(&p.shares[blk[u]], 1);
      else record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    }
  }
  for (int f = cta * kThreads + tid; f < p.F; f += per) {
    int from = -1, to = -1, rows = 0;
    if (served(f)) {
      const int len = s_len[f], full = len >> p.bs_log2, d = p.dst[f];
      rows = len & (bs - 1);
      p.n_blocks[d] = full + (rows != 0);
      p.kv_lens[d] = len;
      if (rows != 0) {
        from = p.tables[(long long)p.src[f] * p.max_blocks + full];
        to = p.free_list[fc - 1 - s_tail[f]];
        if (to < 0 || to >= p.num_blocks) to = -1;
        p.tables[(long long)d * p.max_blocks + full] = to;
        if (to < 0 || from < 0 || from >= p.num_blocks) {   // nothing to copy, or nowhere
          from = to = -1;
          rows = 0;
          record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
        }
      }
    } else if (s_len[f] >= 0) {
      record_status(p.ctl.status, GQA_ERR_NO_BLOCKS);
    }
    p.copies[3 * f] = from;
    p.copies[3 * f + 1] = to;
    p.copies[3 * f + 2] = rows;
  }
  if (cta == 0 && tid == 0) {
    *p.free_count = fc - min(total.y, fc);
    if (fc != fc_read) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
}

// Sum of the CTA's counts before this thread's, and of all (whole CTA).
__device__ __forceinline__ int2 counts_to(int n, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();   // (the last round's counts have been read)
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  int before = v - n, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  return make_int2(before, all);
}

// Counts a tile's flagged entries (bit u of m: this thread's u-th) in their order: afterwards s_cnt[u * 16 + warp] has
// those before the warp's u-th row.  Returns all (whole CTA).
constexpr int kWarps = kThreads / 32;
static_assert(kMany * kWarps <= kThreads, "a thread scans one count");
template <int kRun>
__device__ __forceinline__ int rank_tile(uint32_t m, int* s_cnt, int* s_warp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();   // (the last tile's counts have been read)
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const uint32_t b = __ballot_sync(0xffffffffu, (m >> u) & 1u);
    if (lane == 0) s_cnt[u * kWarps + warp] = __popc(b);
  }
  __syncthreads();
  const int2 r = counts_to(tid < kRun * kWarps ? s_cnt[tid] : 0, s_warp);
  if (tid < kRun * kWarps) s_cnt[tid] = r.x;
  __syncthreads();
  return r.y;
}
// f(u, rank) for each of this thread's flagged entries.
template <int kRun, typename F>
__device__ __forceinline__ void each_ranked(uint32_t m, const int* s_cnt, F&& f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const bool flag = (m >> u) & 1u;
    const uint32_t b = __ballot_sync(0xffffffffu, flag);
    if (flag) f(u, s_cnt[u * kWarps + warp] + __popc(b & ((1u << lane) - 1u)));
  }
}

// Tells every CTA of the cluster this one's counts; returns the sums before it and of all (whole CTA).
__device__ __forceinline__ int4 counts_before(int2 mine, int2* s_all) {
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (threadIdx.x < uint32_t(ctas)) {
    const uint32_t a = ptx::mapa_shared(ptx::smem_addr(&s_all[cta]), threadIdx.x);
    ptx::st_cluster_u32(a, uint32_t(mine.x));
    ptx::st_cluster_u32(a + 4, uint32_t(mine.y));
  }
  ptx::cluster_sync();
  int4 r = make_int4(0, 0, 0, 0);
  for (int c = 0; c < ctas; ++c) {
    if (c < cta) {
      r.x += s_all[c].x;
      r.y += s_all[c].y;
    }
    r.z += s_all[c].x;
    r.w += s_all[c].y;
  }
  return r;
}

template <int kRun>
__global__ void __launch_bounds__(kThreads, 1) block_free_kernel(const PagesParams p) {
  constexpr int kTile = kThreads * kRun;
  extern __shared__ int smem[];
  __shared__ int2 part[kThreads / 32];
  __shared__ int s_warp[kWarps], s_cnt[kRun * kWarps];
  __shared__ int2 s_all[kMaxCtas];
  int* const s_keep = smem;            // B: blocks that stay
  int* const s_rel = s_keep + p.B;     // B: entries to release, then their exclusive sums
  int* const s_none = s_rel + p.B;     // B (the sums' second array)
  const int tid = threadIdx.x, cta = blockIdx.x, per = gridDim.x * kThreads, bs = 1 << p.bs_log2;
  let_next_start();
  wait_for_last();
  const int fc_read = *p.free_count, fc = min(max(fc_read, 0), p.num_blocks);
  for (int b = tid; b < p.B; b += kThreads) {
    const int len = p.lens[b], have = p.n_blocks[b];
    const bool ok = len >= 0 && have >= 0 && have <= p.max_blocks;
    const int keep = ok ? int(min(((long long)len + bs - 1) >> p.bs_log2, (long long)have)) : have;
    s_keep[b] = keep;
    s_rel[b] = have - keep;
    s_none[b] = 0;
    if (!ok && cta == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
  __syncthreads();
  const int total = scan2<kThreads>(s_rel, s_none, p.B, part).x;
  ptx::cluster_sync();   // every CTA has read the counts
  const auto inside = [&](int blk) { return blk >= 0 && blk < p.num_blocks; };
  // each CTA has a run of the entries, in order
  const int lo = int((long long)total * cta / int(gridDim.x)), hi = int((long long)total * (cta + 1) / int(gridDim.x));
  const bool one = hi - lo <= kTile;   // (its blocks stay in registers)
  int blk[kRun], b[kRun];
  const auto place = [&](int u, int k) {
    return p.tables + ((long long)b[u] * p.max_blocks + s_keep[b[u]] + (k - s_rel[b[u]]));
  };
  const auto blocks = [&](int k0) {
    owners(s_rel, p.B, k0, b);
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int k = k0 + kThreads * u + tid;
      blk[u] = k < hi ? *place(u, k) : -1;
    }
  };
  for (int k0 = lo; k0 < hi; k0 += kTile) {
    blocks(k0);
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (inside(blk[u])) atomicSub(&p.shares[blk[u]], 1);
      else if (k0 + kThreads * u + tid < hi) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    }
  }
  ptx::cluster_sync();
  uint32_t m = 0u;   // entries whose block has no owner left; those that won it
  const auto look = [&](int k0, auto&& is) {
    int left[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) left[u] = inside(blk[u]) ? __ldcg(p.shares + blk[u]) : 0;
    m = 0u;
#pragma unroll
    for (int u = 0; u < kRun; ++u)
      if (is(left[u], k0 + kThreads * u + tid)) m |= 1u << u;
  };
  for (int k0 = lo; k0 < hi; k0 += kTile) {
    if (!one) blocks(k0);
    look(k0, [&](int left, int) { return left < 0; });
#pragma unroll
    for (int u = 0; u < kRun; ++u)
      if ((m >> u) & 1u) atomicMin(&p.shares[blk[u]], -kWon - (k0 + kThreads * u + tid));
  }
  ptx::cluster_sync();
  const auto won = [&](int k0) {
    if (!one) blocks(k0);
    if (!one || __any_sync(0xffffffffu, m != 0u)) look(k0, [&](int left, int k) { return left == -kWon - k; });
  };
  int mine = 0;
  for (int k0 = lo; k0 < hi; k0 += kTile) {
    won(k0);
    mine += rank_tile<kRun>(m, s_cnt, s_warp);
  }
  const int4 c = counts_before(make_int2(mine, 0), s_all);
  int at = c.x;
  for (int k0 = lo; k0 < hi; k0 += kTile) {
    if (!one) won(k0);
    const int n = one ? mine : rank_tile<kRun>(m, s_cnt, s_warp);
    each_ranked<kRun>(m, s_cnt, [&](int u, int rank) {
      const int to = fc + c.z - 1 - (at + rank);
      if (to < p.num_blocks) p.free_list[to] = blk[u];
      p.shares[blk[u]] = 0;
    });
    at += n;
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int k = k0 + kThreads * u + tid;
      if (k < hi) *place(u, k) = -1;
    }
  }
  for (int b = cta * kThreads + tid; b < p.B; b += per)
    if (p.n_blocks[b] > s_keep[b]) p.n_blocks[b] = s_keep[b];
  if (cta == 0 && tid == 0) {
    *p.free_count = min(fc + c.z, p.num_blocks);
    if (fc != fc_read || (long long)fc + c.z > p.num_blocks)
      record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);   // more blocks than there are
  }
}

struct CompactParams {
  const int* tables;
  const int* n_blocks;
  const int* free_list;
  const int* free_count;
  const int* shares;
  int* tables_out;
  int* free_list_out;
  int* shares_out;
  int* index;
  int* copies;
  int B, max_blocks, num_blocks, block_size;
  LaunchCtl ctl;
};

// New places of the blocks, the copies, and the stack.
template <int kRun>
__global__ void __launch_bounds__(kThreads, 1) compact_index_kernel(const CompactParams p) {
  constexpr int kTile = kThreads * kRun;
  __shared__ int s_warp[kWarps], s_cnt[2][kRun * kWarps];
  __shared__ int2 s_all[kMaxCtas];
  const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x, N = p.num_blocks;
  const int per = ctas * kThreads, first = cta * kThreads + tid;
  let_next_start();
  wait_for_last();
  const int fc_read = *p.free_count, fc = min(max(fc_read, 0), N), live = N - fc;
  for (int n = first; n < N; n += per) {
    p.index[n] = n;
    p.shares_out[n] = 0;
  }
  for (int k = first; k < 3 * (N / 2); k += per) p.copies[k] = k % 3 == 2 ? 0 : -1;
  ptx::cluster_sync();
  for (int i = first; i < fc; i += per) {
    const int blk = p.free_list[i];
    if (blk >= 0 && blk < N) p.index[blk] = -1;
  }
  ptx::cluster_sync();
  // free places below `live` and live blocks from there on: each CTA has a run of the pool
  const int lo = int((long long)N * cta / ctas), hi = int((long long)N * (cta + 1) / ctas);
  // this thread's places of the tile at n0: free ones below `live`, and live ones from there on
  uint32_t holes = 0u, movers = 0u;
  const auto look = [&](int n0) {
    int to[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int n = n0 + kThreads * u + tid;
      to[u] = n < hi ? __ldcg(p.index + n) : 0;
    }
    holes = movers = 0u;
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int n = n0 + kThreads * u + tid;
      if (n < hi && to[u] < 0 && n < live) holes |= 1u << u;
      if (n < hi && to[u] >= 0 && n >= live) movers |= 1u << u;
    }
  };
  int2 mine = make_int2(0, 0);
  for (int n0 = lo; n0 < hi; n0 += kTile) {
    look(n0);
    mine.x += rank_tile<kRun>(holes, s_cnt[0], s_warp);
    mine.y += rank_tile<kRun>(movers, s_cnt[1], s_warp);
  }
  const int4 c = counts_before(mine, s_all);
  const bool whole = c.z == c.w && fc == fc_read;   // else a block is on the stack twice, or is not one
  int2 at = make_int2(c.x, c.y);
  for (int n0 = lo; whole && n0 < hi; n0 += kTile) {
    if (hi - lo > kTile) {
      look(n0);
      mine.x = rank_tile<kRun>(holes, s_cnt[0], s_warp);
      mine.y = rank_tile<kRun>(movers, s_cnt[1], s_warp);
    }
    each_ranked<kRun>(holes, s_cnt[0], [&](int u, int rank) { p.copies[3 * (at.x + rank) + 1] = n0 + kThreads * u + tid; });
    each_ranked<kRun>(movers, s_cnt[1], [&](int u, int rank) {
      p.copies[3 * (at.y + rank)] = n0 + kThreads * u + tid;
      p.copies[3 * (at.y + rank) + 2] = p.block_size;
    });
    at.x += mine.x;
    at.y += mine.y;
  }
  for (int n = first; n < N; n += per) p.free_list_out[n] = whole ? N - 1 - n : p.free_list[n];
  ptx::cluster_sync();
  if (whole)
    for (int r = first; r < c.z; r += per) p.index[__ldcg(p.copies + 3 * r)] = __ldcg(p.copies + 3 * r + 1);
  if (!whole && first == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
}

// Tables and counts by the new places.
__global__ void __launch_bounds__(256) compact_tables_kernel(const CompactParams p) {
  let_next_start();
  wait_for_last();
  // (entries and blocks are below 2^30)
  const uint32_t per = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  for (uint32_t n = first; n < uint32_t(p.num_blocks); n += per) {
    const int to = __ldcg(p.index + n);
    if (to >= 0) p.shares_out[to] = p.shares[n];
  }
  const uint32_t width = uint32_t(p.max_blocks), entries = uint32_t(p.B) * width;
  for (uint32_t e = first; e < entries; e += per) {
    const int b = int(e / width), i = int(e - uint32_t(b) * width);
    int out = -1;
    if (i < __ldg(p.n_blocks + b)) {
      const int blk = p.tables[e];
      if (blk >= 0 && blk < p.num_blocks) out = __ldcg(p.index + blk);
      if (out < 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);   // no block, or a free one
    }
    p.tables_out[e] = out;
  }
}

struct CopyParams {
  const int* copies;
  uint4* k_pool;
  uint4* v_pool;
  float* k_scale;
  float* v_scale;
  long long n;            // listed copies
  int num_blocks, Hkv, bs_log2, parts;   // parts: of a block's copy
  LaunchCtl ctl;
};

constexpr int kCopyThreads = 256;
constexpr int kUnroll = 4;
constexpr int kChunk = kCopyThreads * kUnroll;   // 16-byte pieces of a part: 16 KB

__global__ void __launch_bounds__(kCopyThreads) kv8_copy_kernel(const CopyParams p) {
  const int tid = threadIdx.x, lane = tid & 31;
  let_next_start();
  wait_for_last();
  const int row_log2 = p.bs_log2 + 4;                      // 16-byte pieces of a head's rows
  const long long items = p.n * p.parts, step = gridDim.x;
  // 32 of this CTA's items at a time: a lane looks one up, so that long lists with few copies cost little
  for (long long i0 = blockIdx.x; i0 < items; i0 += 32 * step) {
    const long long mine = i0 + lane * step;
    int from = -1, to = -1, rows = 0, part = 0;
    if (mine < items) {
      const long long c = mine / p.parts;
      part = int(mine - c * p.parts);
      from = __ldg(p.copies + 3 * c);
      to = __ldg(p.copies + 3 * c + 1);
      rows = __ldg(p.copies + 3 * c + 2);
    }
    const bool any = from >= 0 && to >= 0 && rows > 0;
    const bool ok = any && from < p.num_blocks && to < p.num_blocks && rows <= (1 << p.bs_log2) && from != to;
    if (any && !ok && from != to && tid < 32) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    for (uint32_t todo = __ballot_sync(0xffffffffu, ok); todo != 0u; todo &= todo - 1u) {
      const int l = __ffs(todo) - 1;
      const int f = __shfl_sync(0xffffffffu, from, l), t = __shfl_sync(0xffffffffu, to, l);
      const int n_rows = __shfl_sync(0xffffffffu, rows, l), pt = __shfl_sync(0xffffffffu, part, l);
      uint4 u[kUnroll];
      uint4* d[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int piece = pt * kChunk + k * kCopyThreads + tid, head = piece >> row_log2;   // K's heads, then V's
        const int in_head = piece & ((1 << row_log2) - 1);
        d[k] = nullptr;
        if (head < 2 * p.Hkv && (in_head >> 4) < n_rows) {
          uint4* const pool = head < p.Hkv ? p.k_pool : p.v_pool;
          const int h = head < p.Hkv ? head : head - p.Hkv;
          u[k] = pool[((size_t(f) * p.Hkv + h) << row_log2) + in_head];
          d[k] = pool + ((size_t(t) * p.Hkv + h) << row_log2) + in_head;
        }
      }
      if (pt == 0)
        for (int h = tid; h < 2 * p.Hkv; h += kCopyThreads) {
          float* const sc = h < p.Hkv ? p.k_scale + h : p.v_scale + (h - p.Hkv);
          sc[size_t(t) * p.Hkv] = sc[size_t(f) * p.Hkv];
        }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (d[k] != nullptr) *d[k] = u[k];
    }
  }
}

// Checks that the three planning calls share.
int check_tables(int B, int max_blocks, int num_blocks, int block_size) {
  if (B < 1 || max_blocks < 1) return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, 1, block_size);
  if (st != GQA_OK) return st;
  if (B > kMaxSeqs || (long long)B * max_blocks >= kWon || (long long)max_blocks * block_size >= (1LL << 31))
    return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

bool ints(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (q == nullptr || !aligned_to(q, 4)) return false;
  return true;
}

template <typename P>
int launch_cluster(void (*kernel)(P), const char* name, int ctas, size_t smem, size_t most, gqa_stream_t stream,
                   std::atomic<unsigned long long>& allowed, const P& p) {
  if (most > 0 && allow_smem_once(allowed, reinterpret_cast<const void*>(kernel), most) != cudaSuccess)
    return GQA_ERR_CUDA;
  if (launch_dependent(kernel, dim3(unsigned(ctas)), kThreads, smem, static_cast<cudaStream_t>(stream), ctas, p) !=
      cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch(name, ctas, kThreads, smem);
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_block_fork(const int* src, const int* dst, const int* lens, int* kv_lens, int* block_tables, int* n_blocks,
                   int* free_list, int* free_count, int* shares, int* copies, int F, int B, int max_blocks,
                   int num_blocks, int block_size, gqa_stream_t stream) {
  if (F < 0) return GQA_ERR_INVALID_ARG;
  const int st = check_tables(B, max_blocks, num_blocks, block_size);
  if (st != GQA_OK) return st;
  if (F > kMaxSeqs || (long long)F * max_blocks >= kWon) return GQA_ERR_UNSUPPORTED;
  if (F == 0) return GQA_OK;
  if (!ints({src, dst, kv_lens, block_tables, n_blocks, free_list, free_count, shares, copies}) || !aligned_to(lens, 4))
    return GQA_ERR_INVALID_ARG;
  PagesParams p{src, dst, lens, kv_lens, block_tables, n_blocks, free_list, free_count, shares, copies,
                F, B, max_blocks, num_blocks, 0, {}};
  while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  static std::atomic<unsigned long long> allowed{0};
  const size_t smem = (size_t(B) + size_t(3) * F) * sizeof(int), most = size_t(4) * kMaxSeqs * sizeof(int);
  static std::atomic<unsigned long long> allowed_few{0};
  return (long long)F * max_blocks > kFew * kThreads
             ? launch_cluster(block_fork_kernel<kMany>, "block_fork_kernel", kMaxCtas, smem, most, stream, allowed, p)
             : launch_cluster(block_fork_kernel<kFew>, "block_fork_kernel", 1, smem, most, stream, allowed_few, p);
}

int gqa_block_free(const int* kv_lens, int* block_tables, int* n_blocks, int* free_list, int* free_count, int* shares,
                   int B, int max_blocks, int num_blocks, int block_size, gqa_stream_t stream) {
  const int st = check_tables(B, max_blocks, num_blocks, block_size);
  if (st != GQA_OK) return st;
  if (!ints({kv_lens, block_tables, n_blocks, free_list, free_count, shares})) return GQA_ERR_INVALID_ARG;
  PagesParams p{nullptr, nullptr, kv_lens, nullptr, block_tables, n_blocks, free_list, free_count, shares, nullptr,
                0, B, max_blocks, num_blocks, 0, {}};
  while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  static std::atomic<unsigned long long> allowed{0};
  const size_t smem = size_t(3) * B * sizeof(int), most = size_t(3) * kMaxSeqs * sizeof(int);
  static std::atomic<unsigned long long> allowed_few{0};
  return (long long)B * max_blocks > kFew * kThreads
             ? launch_cluster(block_free_kernel<kMany>, "block_free_kernel", kMaxCtas, smem, most, stream, allowed, p)
             : launch_cluster(block_free_kernel<kFew>, "block_free_kernel", 1, smem, most, stream, allowed_few, p);
}

int gqa_block_compact(const int* block_tables, const int* n_blocks, const int* free_list, const int* free_count,
                      const int* shares, int* tables_out, int* free_list_out, int* shares_out, int* new_index,
                      int* copies, int B, int max_blocks, int num_blocks, int block_size, gqa_stream_t stream) {
  const int st = check_tables(B, max_blocks, num_blocks, block_size);
  if (st != GQA_OK) return st;
  if (!ints({block_tables, n_blocks, free_list, free_count, shares, tables_out, free_list_out, shares_out, new_index}) ||
      (num_blocks > 1 && !ints({copies})))
    return GQA_ERR_INVALID_ARG;
  if (tables_out == block_tables || free_list_out == free_list || shares_out == shares) return GQA_ERR_INVALID_ARG;
  CompactParams p{block_tables, n_blocks, free_list, free_count, shares, tables_out, free_list_out, shares_out,
                  new_index, copies, B, max_blocks, num_blocks, block_size, {}};
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  static std::atomic<unsigned long long> allowed{0};
  const int code =
      num_blocks > kFew * kThreads
          ? launch_cluster(compact_index_kernel<kMany>, "compact_index_kernel", kMaxCtas, 0, 0, stream, allowed, p)
          : launch_cluster(compact_index_kernel<kFew>, "compact_index_kernel", 1, 0, 0, stream, allowed, p);
  if (code != GQA_OK) return code;
  const long long work = (long long)B * max_blocks + num_blocks, ctas2 = (work + 511) / 512;
  const unsigned grid = unsigned(ctas2 < 4 * device_sm_count() ? ctas2 : 4 * device_sm_count());
  if (launch_dependent(compact_tables_kernel, dim3(grid), 256, 0, static_cast<cudaStream_t>(stream), 1, p) !=
      cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch("compact_tables_kernel", grid, 256, 0);
  return GQA_OK;
}

int gqa_kv8_copy(const int* copies, void* k_pool, void* v_pool, float* k_scale, float* v_scale, int n, int Hkv,
                 int num_blocks, int block_size, gqa_stream_t stream) {
  if (n < 0) return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, Hkv, block_size);
  if (st != GQA_OK) return st;
  if (n == 0) return GQA_OK;
  if (!ints({copies, k_scale, v_scale}) || k_pool == nullptr || v_pool == nullptr || !aligned_to(k_pool, 16) ||
      !aligned_to(v_pool, 16))
    return GQA_ERR_INVALID_ARG;
  if (Hkv >= (1 << 14)) return GQA_ERR_UNSUPPORTED;
  CopyParams p{copies, static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), k_scale, v_scale, n, num_blocks, Hkv,
               0, 0, {}};
  while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
  p.parts = (2 * Hkv * block_size * 16 + kChunk - 1) / kChunk;
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  const long long items = p.n * p.parts, most = 8LL * device_sm_count();
  const unsigned grid = unsigned(items < most ? items : most);
  if (launch_dependent(kv8_copy_kernel, dim3(grid), kCopyThreads, 0, static_cast<cudaStream_t>(stream), 1, p) !=
      cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch("kv8_copy_kernel", grid, kCopyThreads, 0);
  return GQA_OK;
}

}  // extern "C"
