// Rotary positions of queries and keys, one launch for both:
//
//   (x1, x2) -> (x1 cos a - x2 sin a, x2 cos a + x1 sin a) * scale,   a = position * inv_freq[j]
//
// for the pairs j of a head's first rot_dims dims (neighbours, or dims j and j + rot_dims / 2); the dims behind them
// are copied.  Fp32 products, one rounding to the type.
//
// The angle is worked out in turns of 2^-64, modulo a turn, by integer products: inv_freq = m 2^e as 24-bit m times
// 2^66 / (2 pi) gives the turn's share of one position to 2^-64, times the position, so that a position of 2^31 is
// off by 2^-32 of a turn (in fp32 a far position's angle is wrong by whole radians; fp64 products, at 2 a clock and
// SM, would take as long as the copies).  sincospif takes it from there, once per token and pair: a CTA works out its
// tokens' angles in shared memory while its first rows are on their way.
//
// Bound by memory: a warp has a token's heads, 512 bytes (16 a lane) each, four of them in flight.  Measured, 24 + 4 heads:
// see rope's figures below the kernel.
#include <cuda_runtime.h>

#include "kv8_common.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;   // rows that a warp has in flight
constexpr int kMaxPairs = kHeadDim / 2;

struct RopeParams {
  const uint4* x[2];          // q, k
  uint4* y[2];
  long long xs[2][3], ys[2][3];   // strides of batch, token and head, in 16 bytes
  const int* positions;
  long long pos_batch;        // positions of a batch entry behind those of the last
  const float* inv_freq;
  int L, heads, q_heads, half, warps_log2;   // half: pairs; warps_log2: of a token
  long long tokens;
  float scale;
  bool inverse, in_place[2];
};

// cos and sin (times scale) of position * freq.
__device__ float2 turn(int position, float freq, float scale, bool inverse) {
  const uint32_t b = __float_as_uint(freq), exp = (b >> 23) & 255u;
  if (exp == 255u) return make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
  const unsigned long long m = (b & 0x7FFFFFu) | (exp ? 0x800000u : 0u);
  constexpr unsigned long long kTurns = 0xA2F9836E4E441529ull;   // 2^66 / (2 pi)
  const unsigned long long lo = m * kTurns, hi = __umul64hi(m, kTurns);
  const int s = 2 - (int(max(exp, 1u)) - 150);                   // m 2^(exp - 150) / (2 pi) = (hi, lo) 2^-s, of 2^64 a turn
  unsigned long long f = 0ull;
  if (s >= 64) f = s < 128 ? hi >> (s - 64) : 0ull;
  else if (s > 0) f = (lo >> s) | (hi << (64 - s));
  else if (s > -64) f = lo << -s;
  unsigned long long a = f * static_cast<unsigned long long>(static_cast<long long>(position));
  if ((int(b) < 0) != inverse) a = 0ull - a;
  float sn, cs;
  sincospif(float(static_cast<long long>(a)) * 1.0842021724855044e-19f, &sn, &cs);   // 2^-63: half turns
  return make_float2(cs * scale, sn * scale);
}

template <bool kF16, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeParams p) {
  __shared__ float2 cs[kWarps * kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_token = 1 << p.warps_log2, tokens = kWarps >> p.warps_log2;   // of a CTA
  const long long t0 = (long long)blockIdx.x * tokens;
  const int slot = warp >> p.warps_log2, first = warp & (per_token - 1);
  const long long t = t0 + slot;
  const bool live = t < p.tokens;
  const long long b = live ? t / p.L : 0, i = live ? t - b * p.L : 0;
  const int chunks = p.half >> 2;   // 16-byte chunks of the rotated dims
  let_next_start();
  wait_for_last();
  uint4 u[kBatch];
  // rows first + per_token (n0 + k); those of a head in place only as far as they change
  const auto each = [&](int n0, auto&& f) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = first + per_token * (n0 + k);
      if (!live || h >= p.heads) continue;
      const int w = h >= p.q_heads;
      if (p.in_place[w] && lane >= chunks) continue;
      f(k, w, h - (w ? p.q_heads : 0));
    }
  };
  const auto load = [&](int n0) {
    each(n0, [&](int k, int w, int h) { u[k] = p.x[w][b * p.xs[w][0] + i * p.xs[w][1] + h * p.xs[w][2] + lane]; });
  };
#pragma unroll
  for (int k = 0; k < kBatch; ++k) u[k] = make_uint4(0u, 0u, 0u, 0u);
  load(0);
  for (int k = threadIdx.x; k < tokens * p.half; k += kWarps * 32) {
    const int n = k / p.half, j = k - n * p.half;
    const long long tt = t0 + n;
    if (tt < p.tokens) {
      const long long bb = tt / p.L;
      cs[n * p.half + j] = turn(__ldg(p.positions + bb * p.pos_batch + (tt - bb * p.L)), __ldg(p.inv_freq + j), p.scale,
                                p.inverse);
    }
  }
  __syncthreads();
  // this lane's pairs: of dims 8 lane .., the same for all heads
  constexpr int kPairs = kInterleaved ? 4 : 8;
  const bool upper = !kInterleaved && lane >= (chunks >> 1);
  const bool turns = lane < chunks;
  float2 a[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    const int j = kPairs * lane - (upper ? p.half : 0) + k;
    a[k] = turns && live ? cs[slot * p.half + j] : make_float2(1.f, 0.f);
    if (upper) a[k].y = -a[k].y;
  }
  const int partner = turns ? (upper ? lane - (chunks >> 1) : lane + (chunks >> 1)) : lane;
  const int n_rows = live ? (p.heads - first + per_token - 1) >> p.warps_log2 : 0;
  for (int n0 = 0; n0 < n_rows; n0 += kBatch) {
    if (n0 > 0) load(n0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w}, o[4];
      if constexpr (kInterleaved) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 x = unpack_elem2<kF16>(w[c]);
          o[c] = pack_elem2<kF16>(x.x * a[c].x - x.y * a[c].y, x.y * a[c].x + x.x * a[c].y);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 x = unpack_elem2<kF16>(w[c]);
          const float2 y = unpack_elem2<kF16>(__shfl_sync(0xffffffffu, w[c], partner));
          o[c] = pack_elem2<kF16>(x.x * a[2 * c].x - y.x * a[2 * c].y, x.y * a[2 * c + 1].x - y.y * a[2 * c + 1].y);
        }
      }
      if (turns) u[k] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    each(n0, [&](int k, int w, int h) { p.y[w][b * p.ys[w][0] + i * p.ys[w][1] + h * p.ys[w][2] + lane] = u[k]; });
  }
}

int rope_impl(bool f16, const void* Q, const void* K, const int* positions, const float* inv_freq, void* q_out,
              void* k_out, const long long* strides, int B, int L, int Hq, int Hkv, int rot_dims, int pos_batch,
              int interleaved, int inverse, float scale, gqa_stream_t stream) {
  if (B < 0 || L < 0 || Hq < 1 || Hkv < 0 || rot_dims < 16 || rot_dims > kHeadDim || rot_dims % 16 != 0 ||
      strides == nullptr || (pos_batch != 0 && pos_batch != 1) || (Hkv == 0) != (K == nullptr && k_out == nullptr))
    return GQA_ERR_INVALID_ARG;
  if (B == 0 || L == 0) return GQA_OK;
  if ((long long)B * L >= (1LL << 31) || (long long)Hq + Hkv >= (1LL << 20)) return GQA_ERR_UNSUPPORTED;
  if (Q == nullptr || q_out == nullptr || positions == nullptr || inv_freq == nullptr ||
      (Hkv > 0 && (K == nullptr || k_out == nullptr)))
    return GQA_ERR_INVALID_ARG;
  for (const void* q : {Q, K, (const void*)q_out, (const void*)k_out})
    if (!aligned_to(q, 16)) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 4)) return GQA_ERR_INVALID_ARG;
  RopeParams p{};
  const int n = Hkv > 0 ? 4 : 2;   // rows of strides: Q, q_out, K, k_out
  for (int k = 0; k < 3 * n; ++k)
    if (strides[k] % 8 != 0 || strides[k] < 0) return GQA_ERR_INVALID_ARG;
  p.x[0] = static_cast<const uint4*>(Q);
  p.x[1] = static_cast<const uint4*>(K);
  p.y[0] = static_cast<uint4*>(q_out);
  p.y[1] = static_cast<uint4*>(k_out);
  const int sizes[2][3] = {{B, L, Hq}, {B, L, Hkv}};
  for (int w = 0; w < n / 2; ++w) {
    bool same = true;
    for (int k = 0; k < 3; ++k) {
      p.xs[w][k] = strides[6 * w + k] / 8;
      p.ys[w][k] = strides[6 * w + 3 + k] / 8;
      if (sizes[w][k] > 1 && p.ys[w][k] < kHeadDim / 8) return GQA_ERR_INVALID_ARG;   // rows of the output apart
      same = same && (sizes[w][k] < 2 || p.xs[w][k] == p.ys[w][k]);
    }
    p.in_place[w] = p.x[w] == p.y[w];
    if (p.in_place[w] && !same) return GQA_ERR_INVALID_ARG;
  }
  p.positions = positions;
  p.pos_batch = pos_batch ? L : 0;
  p.inv_freq = inv_freq;
  p.L = L;
  p.heads = Hq + Hkv;
  p.q_heads = Hq;
  p.half = rot_dims / 2;
  while ((kBatch << p.warps_log2) < p.heads && (1 << p.warps_log2) < kWarps) ++p.warps_log2;
  p.tokens = (long long)B * L;
  p.scale = scale;
  p.inverse = inverse != 0;
  const int per_cta = kWarps >> p.warps_log2;
  const unsigned grid = unsigned((p.tokens + per_cta - 1) / per_cta);
  const auto kernel = f16 ? (interleaved ? rope_kernel<true, true> : rope_kernel<true, false>)
                          : (interleaved ? rope_kernel<false, true> : rope_kernel<false, false>);
  if (launch_dependent(kernel, dim3(grid), kWarps * 32, 0, static_cast<cudaStream_t>(stream), 1, p) != cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch(f16 ? "rope_kernel<fp16>" : "rope_kernel<bf16>", grid, kWarps * 32, 0);
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_rope(const void* Q, const void* K, const int* positions, const float* inv_freq, void* q_out, void* k_out,
             const long long* strides, int B, int L, int Hq, int Hkv, int rot_dims, int pos_batch, int interleaved,
             int inverse, float scale, gqa_stream_t stream) {
  return rope_impl(false, Q, K, positions, inv_freq, q_out, k_out, strides, B, L, Hq, Hkv, rot_dims, pos_batch,
                   interleaved, inverse, scale, stream);
}
int gqa_rope_f16(const void* Q, const void* K, const int* positions, const float* inv_freq, void* q_out, void* k_out,
                 const long long* strides, int B, int L, int Hq, int Hkv, int rot_dims, int pos_batch,
                 int interleaved, int inverse, float scale, gqa_stream_t stream) {
  return rope_impl(true, Q, K, positions, inv_freq, q_out, k_out, strides, B, L, Hq, Hkv, rot_dims, pos_batch,
                   interleaved, inverse, scale, stream);
}

}  // extern "C"
