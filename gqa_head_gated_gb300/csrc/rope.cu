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
// SM, would take as long as the copies).  What is left of it, half a turn at most, is rounded to fp32 (2^-23 of a radian)
// for sincospif, once per pair of an item, a lane a pair.
//
// Bound by memory: a warp takes items of 8 heads of a token, 512 bytes (16 a lane) each, the next item's loads under way
// while it turns one.  8192 tokens of 24 + 4 heads, 64 dims turned: 42 us (83 % of the copy rate); 32749 of 16 + 2, whole
// heads: 100 us (89 %).  With a CTA a token they took 56 and 172.  [B, H, L, 256] takes 7 % longer than token-major rows
// (single calls of the first case, L2 full of other data: 62 us for 58; in place 51 for 49).
#include <cuda_runtime.h>

#include "kv8_common.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 8;    // heads of an item
constexpr int kMaxPairs = kHeadDim / 2;

struct RopeParams {
  const uint4* x[2];          // q, k
  uint4* y[2];
  long long xs[2][3], ys[2][3];   // strides of batch, token and head, in 16 bytes
  const int* positions;
  long long pos_batch;        // positions of a batch entry behind those of the last
  const float* inv_freq;
  int L, heads[2], half, groups, q_groups;   // half: pairs; groups: items of a token, of q
  uint32_t items;
  bool one;                   // one batch entry
  float scale;
  bool inverse, in_place[2];
};

// freq / (2 pi), the turns that a position adds, in 2^-64 of a turn, modulo a turn.
__device__ __forceinline__ unsigned long long turns_of(float freq) {
  const uint32_t b = __float_as_uint(freq), exp = (b >> 23) & 255u;
  const unsigned long long m = (b & 0x7FFFFFu) | (exp ? 0x800000u : 0u);
  constexpr unsigned long long kTurns = 0xA2F9836E4E441529ull;   // 2^66 / (2 pi)
  const unsigned long long lo = m * kTurns, hi = __umul64hi(m, kTurns);
  const int s = 2 - (int(max(exp, 1u)) - 150);   // m 2^(exp - 150) / (2 pi) = (hi, lo) 2^-s, of 2^64 a turn
  unsigned long long f = 0ull;
  if (s >= 64) f = s < 128 ? hi >> (s - 64) : 0ull;
  else if (s > 0) f = (lo >> s) | (hi << (64 - s));
  else if (s > -64) f = lo << -s;
  return int(b) < 0 ? 0ull - f : f;
}

// cos and sin of a position's turns, whose upper 32 bits do: 2^-32 of a turn, and then fp32's 24 bits of up to half a turn.
__device__ __forceinline__ float2 turn(int position, unsigned long long turns) {
  const unsigned long long a = turns * static_cast<unsigned long long>(static_cast<long long>(position));
  float sn, cs;
  sincospif(float(int(a >> 32)) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31: in half turns
  return make_float2(cs, sn);
}

template <bool kF16, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, 2) rope_kernel(const RopeParams p) {
  __shared__ float2 s_cs[kWarps][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* const cs = s_cs[warp];
  const int chunks = p.half >> 2;   // 16-byte chunks of the rotated dims
  constexpr int kPairs = kInterleaved ? 4 : 8;   // of a lane's dims 8 lane ..
  const bool turns = lane < chunks, upper = !kInterleaved && lane >= (chunks >> 1);
  const int pair0 = kPairs * lane - (upper ? p.half : 0);
  const int partner = turns ? (upper ? lane - (chunks >> 1) : lane + (chunks >> 1)) : lane;
  const uint32_t step = gridDim.x * kWarps;
  // An item: up to kRows heads of a token, of q or of k.
  struct Item {
    const uint4* x;
    uint4* y;
    long long xs, ys;   // from head to head
    int n;              // heads; 0 for lanes that have nothing to do (of rows that are turned in place, the dims
                        // that are not turned stay where they are)
  };
  const auto place = [&](uint32_t item, int& position) {
    const uint32_t t = item / uint32_t(p.groups), b = p.one ? 0u : t / uint32_t(p.L), i = t - b * uint32_t(p.L);
    position = __ldg(p.positions + size_t(b) * p.pos_batch + i);
    const int g = int(item - t * uint32_t(p.groups));
    const bool k = g >= p.q_groups;
    const int h0 = (k ? g - p.q_groups : g) * kRows, heads = k ? p.heads[1] : p.heads[0];
    Item r;
    r.xs = k ? p.xs[1][2] : p.xs[0][2];
    r.ys = k ? p.ys[1][2] : p.ys[0][2];
    r.x = (k ? p.x[1] : p.x[0]) + (b * (k ? p.xs[1][0] : p.xs[0][0]) + i * (k ? p.xs[1][1] : p.xs[0][1]) + h0 * r.xs + lane);
    r.y = (k ? p.y[1] : p.y[0]) + (b * (k ? p.ys[1][0] : p.ys[0][0]) + i * (k ? p.ys[1][1] : p.ys[0][1]) + h0 * r.ys + lane);
    r.n = (k ? p.in_place[1] : p.in_place[0]) && !turns ? 0 : min(kRows, heads - h0);
    return r;
  };
  const auto load = [&](const Item& r, uint4 (&u)[kRows]) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (k < r.n) u[k] = __ldcs(r.x + k * r.xs);
  };
  let_next_start();
  wait_for_last();
  unsigned long long freq[kMaxPairs / 32];   // of this lane's pairs
  float size[kMaxPairs / 32];                // scale; NaN for a frequency that is none
#pragma unroll
  for (int m = 0; m < kMaxPairs / 32; ++m) {
    const int j = lane + 32 * m;
    const float f = j < p.half ? __ldg(p.inv_freq + j) : 0.f;
    freq[m] = turns_of(p.inverse ? -f : f);
    size[m] = fabsf(f) < INFINITY ? p.scale : __int_as_float(0x7FC00000);
  }
  uint4 u[kRows], next[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) u[k] = next[k] = make_uint4(0u, 0u, 0u, 0u);
  uint32_t item = blockIdx.x * kWarps + warp;
  if (item >= p.items) return;
  int at, at_next = 0;
  Item r = place(item, at), r_next = r;
  load(r, u);
  for (;;) {
    const bool more = p.items - item > step;
    if (more) {
      r_next = place(item + step, at_next);
      load(r_next, next);
    }
    __syncwarp();
#pragma unroll
    for (int m = 0; m < kMaxPairs / 32; ++m)
      if (32 * m < p.half) {
        const float2 c = turn(at, freq[m]);
        if (lane + 32 * m < p.half) cs[lane + 32 * m] = make_float2(c.x * size[m], c.y * size[m]);
      }
    __syncwarp();
    float2 a[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      a[k] = turns ? cs[pair0 + k] : make_float2(1.f, 0.f);
      if (upper) a[k].y = -a[k].y;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      uint32_t o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 x = unpack_elem2<kF16>(w[c]);
        if constexpr (kInterleaved) {
          o[c] = pack_elem2<kF16>(x.x * a[c].x - x.y * a[c].y, x.y * a[c].x + x.x * a[c].y);
        } else {
          const float2 y = unpack_elem2<kF16>(__shfl_sync(0xffffffffu, w[c], partner));
          o[c] = pack_elem2<kF16>(x.x * a[2 * c].x - y.x * a[2 * c].y, x.y * a[2 * c + 1].x - y.y * a[2 * c + 1].y);
        }
      }
      if (turns) u[k] = make_uint4(o[0], o[1], o[2], o[3]);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (k < r.n) __stcs(r.y + k * r.ys, u[k]);
    if (!more) break;
    item += step;
#pragma unroll
    for (int k = 0; k < kRows; ++k) u[k] = next[k];
    r = r_next;
    at = at_next;
  }
}

// Whether two of the rows (512 bytes each) that na x nb steps of sa and sb reach share bytes; steps of a row or more,
// in 16 bytes.  Nested dims end at the first test; else the multiples of the longer step are compared with the
// nearest of the shorter, over one period of what is left.
bool rows_meet(long long sa, int na, long long sb, int nb) {
  if (sa > sb) return rows_meet(sb, nb, sa, na);
  constexpr int kRow = kHeadDim / 8;
  const __int128 reach = __int128(na - 1) * sa + kRow;   // of the shorter one
  for (int j = 1; j < nb && j <= sa && __int128(j) * sb < reach; ++j) {
    const __int128 at = __int128(j) * sb, i = at / sa, rest = at - i * sa;
    if (rest < kRow || (sa - rest < kRow && i + 1 < na)) return true;
  }
  return false;
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
  const int sizes[2][3] = {{B, L, Hq}, {B, L, Hkv}};
  for (int k = 0; k < 3 * n; ++k)   // (the stride of a dim of one is nobody's)
    if (sizes[k / 6][k % 3] > 1 && (strides[k] % 8 != 0 || strides[k] < 0)) return GQA_ERR_INVALID_ARG;
  p.x[0] = static_cast<const uint4*>(Q);
  p.x[1] = static_cast<const uint4*>(K);
  p.y[0] = static_cast<uint4*>(q_out);
  p.y[1] = static_cast<uint4*>(k_out);
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
  p.heads[0] = Hq;
  p.heads[1] = Hkv;
  p.half = rot_dims / 2;
  p.q_groups = (Hq + kRows - 1) / kRows;
  p.groups = p.q_groups + (Hkv + kRows - 1) / kRows;
  const long long items = (long long)B * L * p.groups;
  if (items >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  for (int w = 0; w < n / 2; ++w)
    for (int k = 0; k < 3; ++k) {
      const int m = (k + 1) % 3;
      if (sizes[w][k] > 1 && sizes[w][m] > 1 && rows_meet(p.ys[w][k], sizes[w][k], p.ys[w][m], sizes[w][m]))
        return GQA_ERR_INVALID_ARG;
    }
  p.items = uint32_t(items);
  p.one = B == 1;
  p.scale = scale;
  p.inverse = inverse != 0;
  // as many CTAs as the SMs hold, of a warp's worth of items each where there are few
  const long long ctas = (items + kWarps - 1) / kWarps, most = 2LL * device_sm_count();
  const unsigned grid = unsigned(ctas < most ? ctas : most);
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
