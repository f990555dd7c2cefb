// Gated attention of decode / verify rows over the paged 8-bit cache: the entry points, the
// plan, and the merge of the split kernel's parts (kv8_attn.cu holds the mathematics):
//
//   out = (sum_i w_i O_i) / (sum_i w_i) * sigmoid(G),  w_i = exp(lse_i - max_i lse_i)
//
// over the parts i of the row's segment.  The merge reads only the parts that were written
// (a count per segment), so that a plan with room for many parts costs a short batch
// nothing.  It is launched as a programmatic dependent: finding its row, which takes a
// chain of reads, and the gate overlap the split kernel's last CTAs.
#include <cuda_runtime.h>

#include "kv8_attn.h"
#include "kv8_common.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;     // of 64 threads, 4 columns a thread
constexpr int kBatch = 8;      // parts whose loads a thread issues together
constexpr int kMaxParts = kThreads;

struct MergeParams {
  const float* o_parts;
  const float* lse_parts;
  const int* n_parts;
  const int* kv_lens;
  const int* cu_rows;
  const uint16_t* gate;
  uint16_t* out;
  float* lse_out;
  int B, T, Hq, Hkv, gqa, max_rows, max_kv_len, max_rb, rows_per_block, parts;
};

// Merges a row's parts, gates and rounds them: one CTA a row.  Rows of no sequence, or of one
// that was skipped, are left as they are.  A chain of reads bounds it (the row's sequence,
// its count of parts, then lse and O side by side), so that a row's parts are spread over
// four groups of threads with eight loads each in flight: with one warp a row, 39 parts took
// 13 us, as long as a third of the split kernel at 2 x 131071 keys.
//
// With more rows than the SMs hold CTAs for, and so few parts a row, a group takes a row of its
// own (kOwn) and the chains of four rows run side by side.  A whole call, 250 sequences of 120
// keys x 8 rows x 16 heads: 95 us so, 194 with a CTA a row; 64 of 1500 keys 61 and 86; 200 of 300
// keys x 1 row 39 and 50.
template <bool kF16, bool kOwn>
__global__ void __launch_bounds__(kThreads) kv8_merge_kernel(const MergeParams p) {
  __shared__ float s_w[kMaxParts];
  __shared__ float s_red[2][kThreads / 32];
  __shared__ float4 s_acc[kGroups - 1][64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kSplit = kOwn ? 1 : kGroups;   // groups of a row
  const int grp = tid >> 6, c4 = (tid & 63) * 4, pg = kOwn ? 0 : grp;
  const int rows_all = p.T * p.Hq, n = kOwn ? min(blockIdx.x * kGroups + grp, rows_all - 1) : blockIdx.x;
  bool live = !kOwn || blockIdx.x * kGroups + grp < rows_all;
  let_next_start();
  const int t = n / p.Hq, h = n - t * p.Hq;
  int b = t, i = 0, rows = 1;
  if (p.cu_rows != nullptr) {
    int lo = 0, hi = p.B - 1;   // last sequence that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu_rows + mid) <= t) lo = mid; else hi = mid - 1;
    }
    const int t0 = __ldg(p.cu_rows + lo), t1 = __ldg(p.cu_rows + lo + 1);
    b = lo;
    i = t - t0;
    rows = t1 - t0;
    if (t0 < 0 || i < 0 || t >= t1 || t1 > p.T || rows > p.max_rows) b = -1;
  }
  const int kv_len = b < 0 ? -1 : __ldg(p.kv_lens + b);
  if (kv_len < rows || kv_len > p.max_kv_len) b = -1;
  if (b < 0) {   // (rows >= 1 where there is a row)
    if (!kOwn) {
      wait_for_last();
      return;
    }
    live = false;
  }
  uint2 gate = make_uint2(0u, 0u);
  if (p.gate != nullptr && pg == 0)
    gate = __ldg(reinterpret_cast<const uint2*>(p.gate + size_t(n) * 256 + c4));
  const int g = h / p.gqa, rb = (i * p.gqa + h - g * p.gqa) / p.rows_per_block;
  wait_for_last();
  const int cnt =
      live ? min(__ldcg(p.n_parts + (size_t(b) * p.Hkv + g) * p.max_rb + rb), p.parts) : 0;
  const size_t stride = size_t(p.T) * p.Hq;
  // the group's first parts are on their way while the weights are worked out
  float4 v[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int s = pg + kSplit * u;
    if (s < cnt)
      v[u] = __ldcg(reinterpret_cast<const float4*>(p.o_parts + (s * stride + n) * 256 + c4));
  }
  const int mine = kOwn ? tid & 63 : tid;   // the part whose weight this thread works out
  const float ls = mine < cnt ? __ldcg(p.lse_parts + mine * stride + n) : -INFINITY;
  float M = ls;   // fmaxf drops a NaN; a NaN part still gets weight NaN below
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) s_red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2 * kSplit; ++k) M = fmaxf(M, s_red[0][kOwn ? 2 * grp + k : k]);
  const float msub = M == -INFINITY ? 0.f : M;
  const float wl = ls == -INFINITY ? 0.f : __expf(ls - msub);
  s_w[tid] = ls == -INFINITY ? -1.f : wl;   // -1: the part saw no key, and its O was not written
  float sum = wl;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_red[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int k = 0; k < 2 * kSplit; ++k) sum += s_red[1][kOwn ? 2 * grp + k : k];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = pg; s0 < cnt; s0 += kSplit * kBatch) {
    if (s0 != pg) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int s = s0 + kSplit * u;
        if (s < cnt)
          v[u] = __ldcg(reinterpret_cast<const float4*>(p.o_parts + (s * stride + n) * 256 + c4));
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int s = s0 + kSplit * u;
      const float w = s < cnt ? s_w[kOwn ? grp * 64 + s : s] : -1.f;
      if (!(w < 0.f)) {   // a weight of 0 counts: its O may hold a NaN that the row sees
        acc.x += w * v[u].x;
        acc.y += w * v[u].y;
        acc.z += w * v[u].z;
        acc.w += w * v[u].w;
      }
    }
  }
  if (kOwn) {
    if (!live) return;
  } else {
    if (grp > 0) s_acc[grp - 1][tid & 63] = acc;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 x = s_acc[k][tid];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float gs[4] = {1.f, 1.f, 1.f, 1.f};
  if (p.gate != nullptr) {
    const float2 a = unpack_elem2<kF16>(gate.x), c = unpack_elem2<kF16>(gate.y);
    gs[0] = gate_sigmoid(a.x);
    gs[1] = gate_sigmoid(a.y);
    gs[2] = gate_sigmoid(c.x);
    gs[3] = gate_sigmoid(c.y);
  }
  uint2 o;
  o.x = pack_elem2<kF16>(acc.x * inv * gs[0], acc.y * inv * gs[1]);
  o.y = pack_elem2<kF16>(acc.z * inv * gs[2], acc.w * inv * gs[3]);
  *reinterpret_cast<uint2*>(p.out + size_t(n) * 256 + c4) = o;
  if (p.lse_out != nullptr && c4 == 0)
    p.lse_out[n] = sum == 0.f ? -INFINITY : msub + __logf(sum);
}

template <bool kF16>
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream) {
  const unsigned rows = unsigned(p.T) * unsigned(p.Hq);
  const bool own = p.parts <= 64 && rows > 2048u / kThreads * unsigned(device_sm_count());
  const unsigned grid = own ? (rows + kGroups - 1) / kGroups : rows;
  const cudaError_t e =
      launch_dependent(own ? kv8_merge_kernel<kF16, true> : kv8_merge_kernel<kF16, false>, dim3(grid),
                       kThreads, 0, stream, 1, p);
  if (e == cudaSuccess)
    note_launch(kF16 ? "kv8_merge_kernel<fp16>" : "kv8_merge_kernel<bf16>", grid, kThreads, 0);
  return e;
}

struct Plan {
  int rows_per_block, max_rb, parts;
  size_t o_bytes, lse_bytes, bytes;   // workspace: O parts, lse parts, parts per segment
};

// Part slots per row: so many that the longest sequence alone can spread over every SM, or
// (large batches, where no sequence need) four times the even share; never more than it
// has tiles of 128 keys.  The shares are cut on the device so that no segment needs more.
Plan plan_decode8(int B, int T, int Hq, int Hkv, int max_rows, int max_kv_len) {
  Plan q;
  const long long packed = (long long)max_rows * (Hq / Hkv), sms = device_sm_count();
  q.rows_per_block = kv8_rows_per_block(packed);
  q.max_rb = int((packed + q.rows_per_block - 1) / q.rows_per_block);
  const long long units = (long long)Hkv * q.max_rb, tiles = (max_kv_len + 127LL) / 128;
  long long parts = (sms + units - 1) / units + 2;
  const long long even = 4 * sms / (B * units) + 2;
  if (parts > (even > 16 ? even : 16)) parts = even > 16 ? even : 16;
  if (parts > tiles) parts = tiles;
  if (parts > kMaxParts) parts = kMaxParts;
  if (parts < 3) parts = 3;
  q.parts = int(parts);
  const size_t rows = size_t(parts) * T * Hq;
  q.o_bytes = rows * 256 * sizeof(float);
  q.lse_bytes = rows * sizeof(float);
  q.bytes = q.o_bytes + q.lse_bytes + size_t(B) * units * sizeof(int);
  return q;
}

int check_sizes(int B, int T, int Hq, int Hkv, int max_rows, int max_kv_len) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_rows < 1 || max_kv_len < 1 ||
      max_rows > max_kv_len)
    return GQA_ERR_INVALID_ARG;
  if ((long long)T * Hq >= (1LL << 31) ||
      (long long)max_rows * Hq >= (1LL << 31) || (long long)B * Hkv >= (1LL << 31) ||
      max_kv_len >= (1 << 30))
    return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

int decode_impl(bool f16, const void* Q, const void* k_pool, const void* v_pool,
                const float* k_scale, const float* v_scale, const void* G,
                const int* block_tables, const int* kv_lens, const int* cu_rows,
                const unsigned long long* tree_mask, void* out, float* lse_out, int B, int T,
                int Hq, int Hkv, int num_blocks, int block_size, int max_blocks, int max_rows,
                int max_kv_len, void* workspace, size_t workspace_bytes, gqa_stream_t stream) {
  int st = check_sizes(B, T, Hq, Hkv, max_rows, max_kv_len);
  if (st == GQA_OK) st = check_kv8_pool(num_blocks, Hkv, block_size);
  if (st != GQA_OK) return st;
  if (max_blocks < 1 || max_kv_len > (long long)max_blocks * block_size) return GQA_ERR_INVALID_ARG;
  if (cu_rows == nullptr && (T != B || max_rows != 1)) return GQA_ERR_INVALID_ARG;
  if (tree_mask != nullptr && cu_rows == nullptr) return GQA_ERR_INVALID_ARG;
  if (tree_mask != nullptr && max_rows > 64) return GQA_ERR_UNSUPPORTED;
  if (T == 0) return GQA_OK;
  if (Q == nullptr || k_pool == nullptr || v_pool == nullptr || k_scale == nullptr ||
      v_scale == nullptr || block_tables == nullptr || kv_lens == nullptr || out == nullptr)
    return GQA_ERR_INVALID_ARG;
  for (const void* q : {Q, k_pool, v_pool, G, (const void*)out})
    if (!aligned_to(q, 16)) return GQA_ERR_INVALID_ARG;
  for (const void* q : {(const void*)k_scale, (const void*)v_scale, (const void*)block_tables,
                        (const void*)kv_lens, (const void*)cu_rows, (const void*)lse_out})
    if (!aligned_to(q, 4)) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(tree_mask, 8)) return GQA_ERR_INVALID_ARG;
  const Plan plan = plan_decode8(B, T, Hq, Hkv, max_rows, max_kv_len);
  // the kernel counts a launch's positions (a segment's tiles and a few more) in 31 bits
  const long long per_seq = (long long)Hkv * plan.max_rb * ((max_kv_len + 127LL) / 128 + 16);
  if (per_seq >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < plan.bytes) return GQA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return GQA_ERR_INVALID_ARG;
  Kv8AttnArgs a{};
  a.q = static_cast<const uint4*>(Q);
  a.k_pool = static_cast<const uint8_t*>(k_pool);
  a.v_pool = static_cast<const uint8_t*>(v_pool);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.tree_mask = tree_mask;
  a.o_parts = static_cast<float*>(workspace);
  a.lse_parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.o_bytes);
  a.n_parts = reinterpret_cast<int*>(static_cast<char*>(workspace) + plan.o_bytes + plan.lse_bytes);
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.gqa = Hq / Hkv;
  a.num_blocks = num_blocks;
  while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
  a.max_blocks = max_blocks;
  a.max_rows = max_rows;
  a.max_kv_len = max_kv_len;
  a.max_rb = plan.max_rb;
  a.parts = plan.parts;
  if (!make_launch_ctl(&a.ctl)) return GQA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long fit = ((1LL << 31) - 1) / per_seq;
  const int step = fit < kKv8Seqs ? int(fit) : kKv8Seqs;
  for (int b0 = 0; b0 < B; b0 += step) {
    a.b0 = b0;
    a.B = B - b0 < step ? B - b0 : step;
    a.tables = block_tables + (long long)b0 * max_blocks;
    a.kv_lens = kv_lens + b0;
    a.cu_rows = cu_rows == nullptr ? nullptr : cu_rows + b0;
    bool encode_failed = false;
    const cudaError_t e = launch_kv8_attn(a, f16, device_sm_count(), s, &encode_failed);
    if (encode_failed) return GQA_ERR_UNSUPPORTED;
    if (e != cudaSuccess) return GQA_ERR_CUDA;
  }
  const MergeParams m{a.o_parts, a.lse_parts, a.n_parts, kv_lens, cu_rows,
                      static_cast<const uint16_t*>(G), static_cast<uint16_t*>(out), lse_out,
                      B, T, Hq, Hkv, a.gqa, max_rows, max_kv_len, plan.max_rb,
                      plan.rows_per_block, plan.parts};
  return (f16 ? launch_merge<true>(m, s) : launch_merge<false>(m, s)) == cudaSuccess ? GQA_OK
                                                                                     : GQA_ERR_CUDA;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_kv8_workspace_size(int B, int T, int Hq, int Hkv, int max_rows, int max_kv_len) {
  if (check_sizes(B, T, Hq, Hkv, max_rows, max_kv_len) != GQA_OK) return 0;
  return plan_decode8(B, T, Hq, Hkv, max_rows, max_kv_len).bytes;
}

int gqa_kv8_decode(const void* Q, const void* k_pool, const void* v_pool, const float* k_scale,
                   const float* v_scale, const void* G, const int* block_tables,
                   const int* kv_lens, const int* cu_rows, const unsigned long long* tree_mask,
                   void* out, float* lse_out, int B, int T, int Hq, int Hkv, int num_blocks,
                   int block_size, int max_blocks, int max_rows, int max_kv_len, void* workspace,
                   size_t workspace_bytes, gqa_stream_t stream) {
  return decode_impl(false, Q, k_pool, v_pool, k_scale, v_scale, G, block_tables, kv_lens, cu_rows,
                     tree_mask, out, lse_out, B, T, Hq, Hkv, num_blocks, block_size, max_blocks,
                     max_rows, max_kv_len, workspace, workspace_bytes, stream);
}
int gqa_kv8_decode_f16(const void* Q, const void* k_pool, const void* v_pool,
                       const float* k_scale, const float* v_scale, const void* G,
                       const int* block_tables, const int* kv_lens, const int* cu_rows,
                       const unsigned long long* tree_mask, void* out, float* lse_out, int B,
                       int T, int Hq, int Hkv, int num_blocks, int block_size, int max_blocks,
                       int max_rows, int max_kv_len, void* workspace, size_t workspace_bytes,
                       gqa_stream_t stream) {
  return decode_impl(true, Q, k_pool, v_pool, k_scale, v_scale, G, block_tables, kv_lens, cu_rows,
                     tree_mask, out, lse_out, B, T, Hq, Hkv, num_blocks, block_size, max_blocks,
                     max_rows, max_kv_len, workspace, workspace_bytes, stream);
}

}  // extern "C"
