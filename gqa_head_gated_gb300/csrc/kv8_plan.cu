// Block tables and slot maps of a paged KV cache, built on the GPU from request lengths.
//
//   need_b = ceil((len_b + r_b) / bs), have_b = n_blocks[b]
//   release: entries need_b .. have_b-1 go back on the free stack (the k-th of R such
//            entries, in (b, i) order, to free_list[fc + R - 1 - k]) and become -1;
//   grow:    b's j-th new block is free_list[avail - 1 - (G_b + j)], avail = fc + R, G_b
//            the blocks that sequences before b need; b is served when its blocks fit.
//   slots[t] = block * bs + row of new row t, -1 for a row that has no place.
// Releasing in that order makes a step that grows and a step that gives the same blocks
// back exact inverses.
//
// A few kB of integers: bound by latency.  One cluster; every CTA of it reads all
// lengths and scans both counts for itself in shared memory, so that only the stack's
// two orderings (all reads before any release, all releases before any grow, all grows
// before the slots) need a barrier across CTAs, which the cluster has in hardware.
// Measured on the GPU: a step of 16 sequences 3.7 us with one CTA, 65,536 new rows in 8
// sequences 12 us with eight (18 with the owner of every token found by itself in global
// memory).
#include <cuda_runtime.h>

#include "kv8_common.cuh"
#include "kv8_scan.cuh"
#include "ptx_sm100.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSeqs = 8192;    // sequences a launch plans: 5 words of shared memory each
constexpr int kMaxCtas = 8;       // the portable cluster size
constexpr int kUnroll = 4;

struct PlanParams {
  const int* kv_lens;
  const int* cu_rows;
  int* tables;
  int* n_blocks;
  int* free_list;
  int* free_count;
  int* slots;
  int* lens_out;
  int B, T, max_blocks, num_blocks, bs_log2;
  LaunchCtl ctl;
};

// Where row offsets fall, rows of one sequence may be rows of another: of those that keep the
// bounds, one that starts before the end of any before it is refused.  Warp 0, 32 sequences at a
// time, with the largest end so far.
__device__ __noinline__ void drop_overlaps(const int* s_cu, int* s_have, int* s_rel, int* s_grow,
                                           int B, int* status) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int end = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      const bool in = b < B && s_have[b] >= 0;
      int most = in ? s_cu[b + 1] : 0;   // largest end up to and with b
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, most, o);
        if (lane >= o) most = max(most, x);
      }
      const int before = __shfl_up_sync(0xffffffffu, most, 1);
      if (in && s_cu[b] < max(end, lane > 0 ? before : 0)) {
        s_have[b] = -1;
        s_rel[b] = s_grow[b] = 0;
        if (status != nullptr) record_status(status, GQA_ERR_DEVICE_RANGE);
      }
      end = max(end, __shfl_sync(0xffffffffu, most, 31));
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
block_plan_kernel(const PlanParams p) {
  extern __shared__ int smem[];
  __shared__ int2 part[kWarps];
  const int B = p.B, bs_log2 = p.bs_log2, bs = 1 << bs_log2;
  int* const s_cu = smem;              // B + 1
  int* const s_len = s_cu + B + 1;     // keys held
  int* const s_have = s_len + B;       // blocks held, -1 for a sequence that breaks the bounds
  int* const s_rel = s_have + B;       // blocks to release, then their exclusive sums
  int* const s_grow = s_rel + B;       // blocks to take, then their exclusive sums
  const int tid = threadIdx.x;
  const int cta = blockIdx.x, ctas = gridDim.x;   // the grid is one cluster
  const long long cap = (long long)p.max_blocks << bs_log2;

  let_next_start();
  wait_for_last();
  for (int b = tid; b <= B; b += kThreads) s_cu[b] = p.cu_rows[b];
  const int fc_read = *p.free_count;
  const int fc = min(max(fc_read, 0), p.num_blocks);
  __syncthreads();
  bool down = false;   // row offsets that fall
  for (int b = tid; b < B; b += kThreads) {
    const int len = p.kv_lens[b], have = p.n_blocks[b];
    down = down || s_cu[b + 1] < s_cu[b];
    const long long end = (long long)len + s_cu[b + 1] - s_cu[b];
    const bool ok = len >= 0 && s_cu[b] >= 0 && s_cu[b + 1] >= s_cu[b] && s_cu[b + 1] <= p.T &&
                    end <= cap && have >= 0 && have <= p.max_blocks;
    const int need = ok ? int((end + bs - 1) >> bs_log2) : 0;
    s_len[b] = len;
    s_have[b] = ok ? have : -1;
    s_rel[b] = ok ? max(have - need, 0) : 0;
    s_grow[b] = ok ? max(need - have, 0) : 0;
    if (!ok && cta == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
  const bool falls = __syncthreads_or(down);   // the same in every CTA
  if (falls) drop_overlaps(s_cu, s_have, s_rel, s_grow, B, cta == 0 ? p.ctl.status : nullptr);
  const int2 total = scan2<kThreads>(s_rel, s_grow, B, part);
  const int avail = min(fc + total.x, p.num_blocks);
  if (cta == 0 && tid == 0 && (fc != fc_read || fc + (long long)total.x > p.num_blocks))
    record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);   // more blocks than there are

  const auto need_of = [&](int b) {
    return int(((long long)s_len[b] + s_cu[b + 1] - s_cu[b] + bs - 1) >> bs_log2);
  };
  // Every CTA has read the lengths, counts and the stack's height.
  ptx::cluster_sync();
  // The last sequence whose first rank (exclusive sum) is at most k: the one with rank k.
  const auto owner = [&](const int* sums, int k) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sums[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int per = ctas * kThreads, first = cta * kThreads + tid;
  if (total.x > 0) {
    for (int k0 = first; k0 < total.x; k0 += kUnroll * per) {
      int blk[kUnroll];
      int* at[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = k0 + u * per;
        if (k >= total.x) continue;
        const int b = owner(s_rel, k);
        at[u] = p.tables + (long long)b * p.max_blocks + need_of(b) + (k - s_rel[b]);
        blk[u] = *at[u];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = k0 + u * per;
        if (k >= total.x) continue;
        const int to = fc + total.x - 1 - k;
        if (to < p.num_blocks) p.free_list[to] = blk[u];
        *at[u] = -1;
      }
    }
    ptx::cluster_sync();
  }
  // (sequences that are not served come last, so that ranks below `avail` tell them apart but
  // for the first of them, whose blocks would fit in part)
  for (int k0 = first; k0 < min(total.y, avail); k0 += kUnroll * per) {
    int blk[kUnroll], own[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * per;
      if (k >= min(total.y, avail)) continue;
      own[u] = owner(s_grow, k);
      blk[u] = __ldcg(p.free_list + avail - 1 - k);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * per;
      if (k >= min(total.y, avail)) continue;
      const int b = own[u], have = s_have[b], n = need_of(b) - have;
      if ((long long)s_grow[b] + n <= avail)
        p.tables[(long long)b * p.max_blocks + have + (k - s_grow[b])] = blk[u];
    }
  }
  for (int b = first; b < B; b += per) {
    const int have = s_have[b];
    const int need = have < 0 ? 0 : need_of(b), n = need - have;
    const bool served = have >= 0 && (n <= 0 || (long long)s_grow[b] + n <= avail);
    if (served && n != 0) p.n_blocks[b] = need;
    if (have >= 0 && !served) record_status(p.ctl.status, GQA_ERR_NO_BLOCKS);
    p.lens_out[b] = s_len[b] + (served ? s_cu[b + 1] - s_cu[b] : 0);
  }
  if (cta == 0 && tid == 0) {
    // The served sequences are those before the first that does not fit (and those that
    // need no block): the stack falls by the blocks that they take.
    int lo = 0, hi = B;   // first b whose blocks and those before it pass `avail`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      const long long after = mid + 1 < B ? s_grow[mid + 1] : total.y;
      if (after > avail) hi = mid; else lo = mid + 1;
    }
    *p.free_count = avail - (lo < B ? s_grow[lo] : total.y);
  }
  if (p.T == 0) return;
  if (falls) {   // no order to search in: a warp goes through a sequence's rows
    for (int t = first; t < p.T; t += per) p.slots[t] = -1;
    ptx::cluster_sync();
    for (int b = first >> 5; b < B; b += per >> 5) {
      const int have = s_have[b], n = have < 0 ? 0 : need_of(b) - have;
      if (have < 0 || (n > 0 && (long long)s_grow[b] + n > avail)) continue;
      for (int t = s_cu[b] + (tid & 31); t < s_cu[b + 1]; t += 32) {
        const int pos = s_len[b] + t - s_cu[b];
        const int blk = __ldcg(p.tables + (long long)b * p.max_blocks + (pos >> bs_log2));
        p.slots[t] = (blk << bs_log2) + (pos & (bs - 1));
      }
    }
    return;
  }
  ptx::cluster_sync();
  // Slots, kUnroll tokens a thread at a time: their table reads are in flight together.
  for (int t0 = first; t0 < p.T; t0 += kUnroll * per) {
    int row[kUnroll], blk[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = t0 + u * per;
      row[u] = -1;
      if (t >= p.T) continue;
      const int lo = owner(s_cu, t);
      const int have = s_have[lo];
      if (have < 0 || t < s_cu[lo] || t >= s_cu[lo + 1]) continue;
      const int n = need_of(lo) - have, pos = s_len[lo] + t - s_cu[lo];
      if (n > 0 && (long long)s_grow[lo] + n > avail) continue;
      row[u] = pos & (bs - 1);
      blk[u] = __ldcg(p.tables + (long long)lo * p.max_blocks + (pos >> bs_log2));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int t = t0 + u * per;
      if (t < p.T) p.slots[t] = row[u] < 0 ? -1 : (blk[u] << bs_log2) + row[u];
    }
  }
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_block_plan(const int* kv_lens, const int* cu_rows, int* block_tables,
                              int* n_blocks, int* free_list, int* free_count, int* slots,
                              int* kv_lens_out, int B, int T, int max_blocks, int num_blocks,
                              int block_size, gqa_stream_t stream) {
  if (B < 1 || T < 0 || max_blocks < 1) return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, 1, block_size);
  if (st != GQA_OK) return st;
  if (kv_lens == nullptr || cu_rows == nullptr || block_tables == nullptr || n_blocks == nullptr ||
      free_list == nullptr || free_count == nullptr || kv_lens_out == nullptr ||
      (slots == nullptr && T > 0))
    return GQA_ERR_INVALID_ARG;
  for (const void* q : {(const void*)kv_lens, (const void*)cu_rows, (const void*)block_tables,
                        (const void*)n_blocks, (const void*)free_list, (const void*)free_count,
                        (const void*)slots, (const void*)kv_lens_out})
    if (!aligned_to(q, 4)) return GQA_ERR_INVALID_ARG;
  // (T and the entries stay far enough below 2^31 for sums with strides and the pool's blocks)
  if (B > kMaxSeqs || T >= (1 << 30) || (long long)B * max_blocks >= (1LL << 30) ||
      (long long)max_blocks * block_size >= (1LL << 31))
    return GQA_ERR_UNSUPPORTED;
  PlanParams p{kv_lens, cu_rows, block_tables, n_blocks, free_list, free_count, slots, kv_lens_out,
               B, T, max_blocks, num_blocks, 0, {}};
  while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  const size_t smem = (size_t(5) * B + 1) * sizeof(int);
  static std::atomic<unsigned long long> allowed{0};
  if (allow_smem_once(allowed, reinterpret_cast<const void*>(block_plan_kernel),
                      (size_t(5) * kMaxSeqs + 1) * sizeof(int)) != cudaSuccess)
    return GQA_ERR_CUDA;
  // One CTA for a decode step (a barrier of a cluster of one costs little), a full cluster
  // where there is work to share.
  const int ctas = B > 2 * kThreads || T > 4 * kThreads ? kMaxCtas : 1;
  if (launch_dependent(block_plan_kernel, dim3(unsigned(ctas)), kThreads, smem,
                       static_cast<cudaStream_t>(stream), ctas, p) != cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch("block_plan_kernel", ctas, kThreads, smem);
  return GQA_OK;
}
