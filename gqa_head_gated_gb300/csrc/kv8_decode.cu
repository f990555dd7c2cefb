// Gated attention of decode / verify rows over the paged 8-bit cache:
//
//   s_j = (Q . k_j) * k_scale[block(j), g] / 16      p_j = exp(s_j - m), l = sum_j p_j
//   out = (sum_j p_j v_j * v_scale[block(j), g]) / l * sigmoid(G)
//
// over the keys a row sees (chain: j < kv_len - rows + i + 1; tree: the keys before the
// new rows, and new key k where bit k of the row's mask is set).
//
// One warp per (row, query head, key split): a lane holds 8 of the 256 dims of q and of
// the running sum, and the keys go by one after another (online softmax, fp32).
#include <cuda_runtime.h>

#include "kv8_common.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;

struct DecodeParams {
  const uint4* q;
  const uint2* k_pool;
  const uint2* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int* tables;
  const int* kv_lens;
  const int* cu_rows;
  const unsigned long long* tree_mask;
  const uint16_t* gate;
  uint16_t* out;
  float* lse_out;
  float* o_parts;
  float* lse_parts;
  int B, T, Hq, Hkv, num_blocks, bs_log2, max_blocks, max_rows, max_kv_len, splits, split_keys;
  LaunchCtl ctl;
};

// The sequence of token t and its row there; false for a token of no (valid) sequence.
__device__ __forceinline__ bool find_row(const DecodeParams& p, int t, int& b, int& i, int& rows,
                                         int& kv_len, bool& bad) {
  bad = false;
  if (p.cu_rows == nullptr) {
    b = t;
    i = 0;
    rows = 1;
  } else {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu_rows + mid) <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    const int t0 = __ldg(p.cu_rows + lo), t1 = __ldg(p.cu_rows + lo + 1);
    i = t - t0;
    rows = t1 - t0;
    if (i < 0 || t >= t1) return false;
    bad = t0 < 0 || t1 > p.T || rows > p.max_rows;
  }
  kv_len = __ldg(p.kv_lens + b);
  bad = bad || kv_len < rows || kv_len > p.max_kv_len;
  return !bad;
}

template <bool kF16>
__global__ void __launch_bounds__(kWarps * 32) kv8_rows_kernel(const DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long n = w / p.splits;
  const int split = int(w - n * p.splits);
  if (n >= (long long)p.T * p.Hq) return;
  const int t = int(n / p.Hq), h = int(n - (long long)t * p.Hq), g = h / (p.Hq / p.Hkv);
  int b, i, rows, kv_len;
  bool bad;
  if (!find_row(p, t, b, i, rows, kv_len, bad)) {
    if (bad && lane == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    return;
  }
  float q[8], acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  {
    const uint4 u = __ldg(p.q + size_t(n) * 32 + lane);
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
    for (int c = 0; c < 4; ++c) {
      const float2 f = unpack_elem2<kF16>(x[c]);
      q[2 * c] = f.x;
      q[2 * c + 1] = f.y;
    }
  }
  const int base = kv_len - rows, bs = 1 << p.bs_log2;
  const bool tree = p.tree_mask != nullptr;
  const unsigned long long mask = tree ? p.tree_mask[t] : 0ull;
  const int lo = split * p.split_keys;
  const int hi = min(lo + p.split_keys, tree ? kv_len : base + i + 1);
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    if (tree && j >= base && !((mask >> (j - base)) & 1ull)) continue;
    const int blk = __ldg(p.tables + (long long)b * p.max_blocks + (j >> p.bs_log2));
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
      break;
    }
    const size_t bg = size_t(blk) * p.Hkv + g;
    const size_t row = (bg * bs + (j & (bs - 1))) * 32 + lane;
    float k[8], v[8], s = 0.f;
    from_e4m3x8(__ldg(p.k_pool + row), k);
    from_e4m3x8(__ldg(p.v_pool + row), v);
    for (int c = 0; c < 8; ++c) s = fmaf(q[c], k[c], s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= __ldg(p.k_scale + bg) * (1.f / 16.f);
    const float m_new = fmaxf(m, s);
    const float msub = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = __expf(m - msub), e = __expf(s - msub), sv = __ldg(p.v_scale + bg);
    m = m_new;
    l = l * alpha + e;
    for (int c = 0; c < 8; ++c) acc[c] = acc[c] * alpha + e * (v[c] * sv);
  }
  const size_t part = size_t(split) * size_t(p.T) * p.Hq + size_t(n);
  if (lane == 0) p.lse_parts[part] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + __logf(l);
  if (l == 0.f) return;
  float4* const o = reinterpret_cast<float4*>(p.o_parts + part * 256 + lane * 8);
  o[0] = make_float4(acc[0] / l, acc[1] / l, acc[2] / l, acc[3] / l);
  o[1] = make_float4(acc[4] / l, acc[5] / l, acc[6] / l, acc[7] / l);
}

// Merges a row's parts, gates and rounds them: one warp a row.  Rows of no sequence, or of
// one that was skipped, are left as they are.
template <bool kF16>
__global__ void __launch_bounds__(kWarps * 32) kv8_merge_kernel(const DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n >= p.T * p.Hq) return;
  int b, i, rows, kv_len;
  bool bad;
  if (!find_row(p, n / p.Hq, b, i, rows, kv_len, bad)) return;
  const size_t stride = size_t(p.T) * p.Hq;
  float M = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) M = fmaxf(M, __ldcg(p.lse_parts + s * stride + n));
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float msub = M == -INFINITY ? 0.f : M;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float ls = __ldcg(p.lse_parts + s * stride + n);
    if (ls == -INFINITY) continue;
    const float w = __expf(ls - msub);
    sum += w;
    const float4* const src =
        reinterpret_cast<const float4*>(p.o_parts + (s * stride + n) * 256 + lane * 8);
    const float4 a = __ldcg(src), c = __ldcg(src + 1);
    const float x[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
    for (int k = 0; k < 8; ++k) acc[k] += w * x[k];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  float gs[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  if (p.gate != nullptr) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p.gate + size_t(n) * 256 + lane * 8));
    const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_elem2<kF16>(w4[e]);
      gs[2 * e] = gate_sigmoid(f.x);
      gs[2 * e + 1] = gate_sigmoid(f.y);
    }
  }
  uint4 o;
  o.x = pack_elem2<kF16>(acc[0] * inv * gs[0], acc[1] * inv * gs[1]);
  o.y = pack_elem2<kF16>(acc[2] * inv * gs[2], acc[3] * inv * gs[3]);
  o.z = pack_elem2<kF16>(acc[4] * inv * gs[4], acc[5] * inv * gs[5]);
  o.w = pack_elem2<kF16>(acc[6] * inv * gs[6], acc[7] * inv * gs[7]);
  *reinterpret_cast<uint4*>(p.out + size_t(n) * 256 + lane * 8) = o;
  if (p.lse_out != nullptr && lane == 0)
    p.lse_out[n] = sum == 0.f ? -INFINITY : msub + __logf(sum);
}

constexpr int kMaxSplits = 16;
int plan_splits(int max_kv_len, int* split_keys) {
  int s = (max_kv_len + 511) / 512;
  if (s > kMaxSplits) s = kMaxSplits;
  *split_keys = (max_kv_len + s - 1) / s;
  return s;
}

int check_sizes(int B, int T, int Hq, int Hkv, int max_rows, int max_kv_len) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_rows < 1 || max_kv_len < 1 ||
      max_rows > max_kv_len)
    return GQA_ERR_INVALID_ARG;
  if ((long long)T * Hq >= (1LL << 31) || (long long)max_rows * (Hq / Hkv) >= (1LL << 30))
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
  DecodeParams p{};
  p.splits = plan_splits(max_kv_len, &p.split_keys);
  const size_t rows = size_t(T) * Hq;
  if (workspace == nullptr || workspace_bytes < p.splits * rows * 257 * sizeof(float))
    return GQA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return GQA_ERR_INVALID_ARG;
  p.q = static_cast<const uint4*>(Q);
  p.k_pool = static_cast<const uint2*>(k_pool);
  p.v_pool = static_cast<const uint2*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.tables = block_tables;
  p.kv_lens = kv_lens;
  p.cu_rows = cu_rows;
  p.tree_mask = tree_mask;
  p.gate = static_cast<const uint16_t*>(G);
  p.out = static_cast<uint16_t*>(out);
  p.lse_out = lse_out;
  p.o_parts = static_cast<float*>(workspace);
  p.lse_parts = p.o_parts + p.splits * rows * 256;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.num_blocks = num_blocks;
  while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
  p.max_blocks = max_blocks;
  p.max_rows = max_rows;
  p.max_kv_len = max_kv_len;
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  const long long grid = ((long long)rows * p.splits + kWarps - 1) / kWarps;
  const long long mgrid = ((long long)rows + kWarps - 1) / kWarps;
  if (grid >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (f16) {
    kv8_rows_kernel<true><<<unsigned(grid), kWarps * 32, 0, s>>>(p);
    kv8_merge_kernel<true><<<unsigned(mgrid), kWarps * 32, 0, s>>>(p);
  } else {
    kv8_rows_kernel<false><<<unsigned(grid), kWarps * 32, 0, s>>>(p);
    kv8_merge_kernel<false><<<unsigned(mgrid), kWarps * 32, 0, s>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return GQA_ERR_CUDA;
  note_launch(f16 ? "kv8_rows_kernel<fp16>" : "kv8_rows_kernel<bf16>", grid, kWarps * 32, 0);
  note_launch(f16 ? "kv8_merge_kernel<fp16>" : "kv8_merge_kernel<bf16>", mgrid, kWarps * 32, 0);
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_kv8_workspace_size(int B, int T, int Hq, int Hkv, int max_rows, int max_kv_len) {
  if (check_sizes(B, T, Hq, Hkv, max_rows, max_kv_len) != GQA_OK) return 0;
  int c = 0;
  return size_t(plan_splits(max_kv_len, &c)) * T * Hq * 257 * sizeof(float);
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
