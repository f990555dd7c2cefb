// The attention of decode / verify rows over the paged 8-bit cache, written as partial
// results (O / l, m + ln l) for the merge in kv8_decode.cu.
//
//   s_rj = (q_r . k_j) * ks_j / 16     p_rj = exp(s_rj - m_r)     l_r = sum_j p_rj
//   O_r  = sum_j p_rj * vs_j * v_j     (ks_j, vs_j: the scales of key j's block and head)
//
// What bounds it: HBM.  A key costs 512 bytes per KV head; the rows of a decode or draft
// step that share it are few.  So the cache's bytes go from TMA straight into the tensor
// core, never through registers: both products run as tcgen05 kind::f8f6f4 with the
// cache as operand A and the rows, few, along N:
//   S^T [128 keys, rows]   = K [128 keys, 256] . Q^T      A K-major as it lies in the block
//   O^T [2 x 128 dims, rows] += V^T [dims, 128 keys] . P^T    A MN-major, the same bytes
// With N this small a product costs reading A (32 KB at 128 bytes a clock per operand),
// whatever N is, and that pays for exactness: Q and P, which have more bits than e4m3,
// enter as sums of e4m3 terms in columns of their own:
//   q = 2^e (t0 + t1 / 16 (+ t2 / 256)): 2 terms hold a bf16's 8 bits, 3 an fp16's 11
//     (each step of 16 is the 4 bits that e4m3 rounds to; elements below 2^-18 of the
//     row's largest lose bits, an absolute error of 2^-23 of that, 2^-27 in fp16);
//   p = t0 + t1 / 32 + t2 / 1024, p <= 256: relative error 2^-13, and what is dropped is
//     below 2^-20, 2^-25 of the row's largest p when its reference has just moved.
//
// The softmax thread of key j holds S^T's lane j: its block's scales are two scalars of
// the thread, the visible-key test is one comparison per row, and block sizes cost
// nothing.  Two references per row, the same in all threads: p uses ref_r, for s + log2 vs
// (the probabilities as the product sees them, so a block of tiny values next to one of
// large ones loses no bits), l uses ml_r, for s.  They move only when a key passes them
// by more than 2^8 (2^64), which one barrier per tile detects; then the warps exchange
// maxima and O is rescaled in tensor memory.
// What a key loses below 2^-25 of the largest p adds up over the keys that a piece has: to 2^-12
// over 64 tiles.  In a longer piece ref_r goes down again where the keys stay far below it, so that
// 131071 keys of which each weighs e^-18 of one other come out as they should (they were lost or
// doubled: 2^-26).  40 sequences of 65536 keys whose scores have a deviation of 8 nats in one key
// of a hundred: 769 us with it, 781 without, for one row; 974 and 818 for four, whose references
// such keys keep moving both ways; shares of 64 tiles and less are as they were but for a
// register (8 x 4 draft rows 75.1 us, 74.2 before).
//
// Roles (64 + 128 threads for 8 rows: 320, 448 or 576): warp 0 copies (TMA, a block per box; scales by
// cp.async), warp 1 issues the products, the others are the softmax and epilogue, a group of
// 128 threads (key by thread) for every 8 rows.  A group agrees at its own barrier whether a
// reference moves; between groups there are only bounded waits, so that one that gives up
// leaves none at a barrier.  One CTA per SM; shares of tiles as kv8_attn.cuh cuts them.
//
// Measured (HBM copies run at 6.78 TB/s): 16 sequences of 32768 keys, 4 rows of a group, 89 us
// for 555 MB (92 %); 2 of 131071 keys in fp16, 53 us for 268 MB (75 %: a launch, a start and a
// merge are 13 us of it); 8 x 4 draft rows, 24 packed, 75 us for 303 MB (60 %), where tiles
// whose references move (1,500 clocks more, by a barrier and the rescale) hold the copies up.
// kTop 5, 3 and 1 are as fast; 5 keeps more of the small probabilities.
//
// A key that a row does not see has p = 0 by selection.  V rows past the last visible key
// of a tile are zeroed in shared memory, and NaN codes of keys that only some rows see are
// taken out before the product and put back for the rows that see them.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv8_attn.cuh"

namespace gqa {
namespace {

constexpr int kGroupRows = 8;                    // rows of one softmax thread
constexpr int kGroupThreads = 128;               // one thread per key of a tile
constexpr int kPTerms = 3;
constexpr float kSlack = 8.f;      // p <= 2^8
constexpr float kTop = 5.f;        // a moved reference leaves the row's largest p at 2^5
// One that has come to stand too high goes down again, to where a tile's largest p is 1: when that
// was below 2^kFall, and above 2^-kDrop of the highest reference: of keys below, 2^-31 of the row's
// largest p, a million weigh 2^-11 of it.  (It keeps O finite, too.)  Looked at in a piece's second
// tile and every 32nd from there, and in the one behind a rise of 2^kJump past all before.
constexpr float kFall = -8.f, kDrop = 26.f, kJump = 8.f;
constexpr int kLook = 32;
template <int MB, bool kF16>
struct Cfg {
  static constexpr int kQTerms = kF16 ? 3 : 2;
  static constexpr int kGroups = MB / kGroupRows;          // softmax thread groups
  static constexpr int kSoftmax = kGroups * kGroupThreads;
  static constexpr int kThreads = 64 + kSoftmax;
  // columns of S^T and of each half of O^T, whole 16s (a column more than there are terms holds
  // nothing that is read)
  static constexpr int kNS = (MB * kQTerms + 15) / 16 * 16;
  static constexpr int kNO = (MB * kPTerms + 15) / 16 * 16;
  // K and V slots of a tile each.  A K slot is free once S has read it, a V slot a softmax
  // and a product later; with two and three the copies' order (K, V, K, V, ...) is the order
  // in which slots come free.
  static constexpr int kKS = MB == 16 ? 3 : 2;
  static constexpr int kVS = 3;
  static constexpr uint32_t kStep = MB == 16 ? 64 : 128;   // tensor-memory columns of each of
  static constexpr uint32_t kTmS = 0;            // the two S buffers
  static constexpr uint32_t kTmO = 2 * kStep;    // and the two halves of O
  static constexpr uint32_t kCols = 4 * kStep;
  static_assert(kNS <= int(kStep) && kNO <= int(kStep), "S and O fit their columns");
  static constexpr uint32_t kIdescS = ptx::idesc_f32acc(128, kNS, 0, 0, 0);
  static constexpr uint32_t kIdescO = ptx::idesc_f32acc(128, kNO, 1, 1, 0);
};

template <int MB, bool kF16>
struct __align__(1024) AttnSmem : RingSmem<Cfg<MB, kF16>::kKS, Cfg<MB, kF16>::kVS> {
  using C = Cfg<MB, kF16>;
  alignas(1024) uint8_t q[2][C::kNS * 128];   // [half of D][column][128 bytes, swizzled]
  uint8_t p[2][C::kNO * kTile];            // [buffer][16 columns][key][16 bytes]
  alignas(16) float red[C::kGroups][2 * kGroupRows][4];   // [group][value][warp], read as float4
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, o_full, drain;
  // by piece, kRowSets in turn
  unsigned long long hit[kRowSets];        // NaN V rows taken out: bit of key pr_lo + i
  unsigned long long mask[kRowSets][MB];   // tree mask of each row
  int lim[kRowSets][MB];                   // keys before this one are seen
  int row[kRowSets][MB];                   // output row (token * Hq + head)
  float fac[kRowSets][MB];                     // scale of the row's Q terms, with log2(e) / 16
  int failed[C::kGroups];
};

// The three terms (columns t0, t0 + MB, t0 + 2 MB) of 8 rows of one half of O^T times f, in
// tensor memory (whole warp).
template <int MB>
__device__ __forceinline__ void rescale_cols(uint32_t t0, const float (&f)[8]) {
  uint32_t a[8], b[8], c[8];
  ptx::tmem_ld8x3_wait(t0, t0 + MB, t0 + 2 * MB, a, b, c);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = __float_as_uint(__uint_as_float(a[i]) * f[i]);
    b[i] = __float_as_uint(__uint_as_float(b[i]) * f[i]);
    c[i] = __float_as_uint(__uint_as_float(c[i]) * f[i]);
  }
  ptx::tmem_st8x3_wait(t0, t0 + MB, t0 + 2 * MB, a, b, c);
}

// Maxima over the warp of 16 values a thread (NaN left out): lane 2 i gets the i-th.  Each
// step halves the values that a lane still carries: 16 shuffles (measured: redux.sync.max.f32
// took 230 cycles a value, 3,700 in all; this about 150).
__device__ __forceinline__ float warp_max16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8; n > 0; n >>= 1) {
    const bool up = (lane & (2 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 2 * n));
    }
  }
  return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// Two probabilities (at most 2^8) as three e4m3 terms each, steps of 32: the first remainder
// is exact in fp32 and goes on as fp16, whose 11 bits hold the two terms to come.
__device__ __forceinline__ void p_terms(float lo, float hi, uint32_t (&t)[kPTerms]) {
  t[0] = take_term(lo, hi, 32.f);
  __half2 r = __floats2half2_rn(lo, hi);
  t[1] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
  const __half2 f(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(t[1]), __NV_E4M3));
  r = __hmul2(__hsub2(r, f), __float2half2_rn(32.f));
  t[2] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
}

template <int MB, bool kF16>
__global__ void __launch_bounds__(Cfg<MB, kF16>::kThreads, 1)
kv8_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const Kv8AttnArgs p) {
  using C = Cfg<MB, kF16>;
  extern __shared__ uint8_t smem_raw[];
  AttnSmem<MB, kF16>& sm = *reinterpret_cast<AttnSmem<MB, kF16>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t tmo = p.ctl.timeout_ns;

  if (tid == 0) {
    init_ring(sm);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.s_full[i], 1);
      ptx::mbar_init(&sm.p_full[i], C::kSoftmax / 32);
      ptx::mbar_init(&sm.pv_done[i], 1);
    }
    ptx::mbar_init(&sm.q_full, C::kSoftmax / 32);
    ptx::mbar_init(&sm.o_full, 1);
    ptx::mbar_init(&sm.drain, 1);
    for (int i = 0; i < C::kGroups; ++i) sm.failed[i] = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem_base, C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Share share = cut_shares<MB>(sm, p);

  if (warp == 0) {
    copy_role<MB, false>(sm, p, tmK, tmV, share);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      const uint64_t qd = ptx::sdesc_sw128(ptx::smem_addr(sm.q), 16, 1024);
      const uint64_t pd = ptx::sdesc_plain(ptx::smem_addr(sm.p), 128, 2048);
      uint32_t J = 0;
      bool ok = true;
      const auto issue_s = [&](uint32_t n) -> bool {
        const uint32_t ks = n % C::kKS;
        if (!wait(&sm.k_full[ks], (n / C::kKS) & 1u, tmo, &sm.abort)) return false;
        ptx::tc_fence_after();
        const uint64_t kd = ptx::sdesc_sw128(ptx::smem_addr(sm.k[ks]), 16, 1024);
        const uint32_t d = tmem + C::kTmS + (n & 1u) * C::kStep;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_ss_f8(d, ptx::sdesc_at(kd, (kk >> 2) * kHalfBytes + (kk & 3) * 32),
                         ptx::sdesc_at(qd, (kk >> 2) * (C::kNS * 128) + (kk & 3) * 32), C::kIdescS,
                         kk > 0);
        ptx::tc_commit(&sm.s_full[n & 1]);
        ptx::tc_commit(&sm.k_empty[ks]);
        return true;
      };
      const auto issue_pv = [&](uint32_t n, bool first) -> bool {
        const uint32_t vs = n % C::kVS, buf = n & 1u;
        if (!wait(&sm.p_full[buf], (n >> 1) & 1u, tmo, &sm.abort)) return false;
        if (!wait(&sm.v_full[vs], (n / C::kVS) & 1u, tmo, &sm.abort)) return false;
        ptx::tc_fence_after();
        const uint64_t vd = ptx::sdesc_sw128(ptx::smem_addr(sm.v[vs]), kHalfBytes, 1024);
        const uint64_t pb = ptx::sdesc_at(pd, buf * (C::kNO * kTile));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_ss_f8(tmem + C::kTmO + h * C::kStep,
                           ptx::sdesc_at(vd, h * kHalfBytes + kk * 4096), ptx::sdesc_at(pb, kk * 512),
                           C::kIdescO, !first || kk > 0);
        ptx::tc_commit(&sm.pv_done[buf]);
        ptx::tc_commit(&sm.v_empty[vs]);
        return true;
      };
      uint32_t pc = 0;   // pieces with tiles so far
      while (ok) {
        ok = wait(&sm.piece_full[pc % kPieceRing], (pc / kPieceRing) & 1u, tmo, &sm.abort);
        if (!ok) break;
        const int n_tiles = sm.piece[pc % kPieceRing].n_tiles;
        if (n_tiles == 0) break;
        ok = wait(&sm.q_full, pc & 1u, tmo, &sm.abort);
        if (!ok) break;
        ptx::tc_fence_after();
        ok = issue_s(J);
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (j + 1 < n_tiles) ok = issue_s(J + j + 1);
          if (ok) ok = issue_pv(J + j, j == 0);
        }
        if (ok) ptx::tc_commit(&sm.o_full);
        J += n_tiles;
        ++pc;
      }
      if (!ok) {
        sm.abort = 1;
        record_status(p.ctl.status, GQA_ERR_TIMEOUT);
      }
      // every product issued has to end before tensor memory is given back
      ptx::tc_commit(&sm.drain);
      wait(&sm.drain, 0, tmo, &sm.zero);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    // Group rg of 128 threads has rows 8 rg .. 8 rg + 7 of the block, thread by key.
    constexpr int kR = kGroupRows;
    const int qd = warp & 3;                   // tensor-memory lanes 32 qd .. 32 qd + 31
    const int rg = (warp - 2) >> 2;
    const int key_in = qd * 32 + lane;         // this thread's key of a tile
    const int st = tid - 64;                   // 0 .. kSoftmax - 1
    const uint32_t trow = tmem + (uint32_t(qd * 32) << 16) + uint32_t(rg * kR);
    const bool tree = p.tree_mask != nullptr;
    const uint32_t bar_id = 1 + rg;            // this group's barrier
    uint32_t J = 0, pc = 0;
    // This thread's waits.  A group agrees at its barriers before it leaves; across groups
    // there are only bounded waits, so that none is left behind at a barrier.
    bool ok = true;
    bool stop = false;   // the same in all threads of a group
    Piece x;
    // The share's next piece into x; false at the share's end, or when the wait ran out.
    uint32_t n_fetched = 0;
    const auto fetch = [&]() -> bool {
      ok = warp_all(ok && wait(&sm.piece_full[n_fetched % kPieceRing], (n_fetched / kPieceRing) & 1u,
                               tmo, &sm.abort));
      x = sm.piece[n_fetched % kPieceRing];
      ++n_fetched;
      return ok && x.n_tiles > 0;
    };
    // Q's terms, the rows' limits and places of piece x, into set `par` of the piece arrays;
    // then the products of the piece may start.  The last piece's S products are done.
    const auto prepare = [&](uint32_t par) {
      constexpr int kWarpsQ = C::kSoftmax / 32, kPer = MB / kWarpsQ;   // rows of each warp
      static_assert(kPer == 2, "two rows a warp");
      const int p0 = x.rb * MB, n_rows = min(MB, x.rows * p.gqa - p0);
      uint4 u[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int r = warp - 2 + k * kWarpsQ;
        const int i = (p0 + r) / p.gqa;
        const int row = (x.t0 + i) * p.Hq + x.g * p.gqa + (p0 + r - i * p.gqa);
        u[k] = r < n_rows ? __ldg(p.q + size_t(row) * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
        if (lane == 0) {
          sm.row[par][r] = row;
          sm.lim[par][r] = r >= n_rows ? 0 : tree ? x.kv_len : x.kv_len - x.rows + i + 1;
          sm.mask[par][r] = tree && r < n_rows ? p.tree_mask[x.t0 + i] : 0ull;
        }
      }
      if (st == 0) sm.hit[par] = 0ull;
#pragma unroll 1
      for (int k = 0; k < kPer; ++k) {
        const int r = warp - 2 + k * kWarpsQ;
        float f[8];
        const uint4 v = k == 0 ? u[0] : u[kPer - 1];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 a = unpack_elem2<kF16>(w[c]);
          f[2 * c] = a.x;
          f[2 * c + 1] = a.y;
        }
        const int e = scale_exp(__reduce_max_sync(0xffffffffu, finite_amax_bits(f)));
        if (lane == 0) sm.fac[par][r] = pow2f(e) * kScaleLog2;
        const float inv = pow2f(-e);
        // an infinite element makes its row's scores NaN, as in the formula
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = isinf(f[c]) ? __int_as_float(0x7FC00000) : f[c] * inv;
#pragma unroll 1
        for (int t = 0; t < C::kQTerms; ++t) {
          const int n = t * MB + r;
          uint2 o;
          o.x = take_term(f[0], f[1], 16.f);
          o.x |= take_term(f[2], f[3], 16.f) << 16;
          o.y = take_term(f[4], f[5], 16.f);
          o.y |= take_term(f[6], f[7], 16.f) << 16;
          *reinterpret_cast<uint2*>(sm.q[lane >> 4] + n * 128 +
                                    ((((lane & 15) >> 1) ^ (n & 7)) << 4) + (lane & 1) * 8) = o;
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.q_full);
    };

    // The piece whose tiles are done and whose parts are due
    int seq = 0, head = 0, s_idx = 0, n_mine = 0, base = 0, pr_lo = 0;
    float ref[kR], ml[kR], l[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) ref[r] = ml[r] = l[r] = 0.f;
    for (bool first = true;; first = false) {
      // ---- the next piece may start while the last one ends (its S products are done)
      const bool more = fetch();
      if (more) prepare(pc % kRowSets);
      if (!first) {
        // ---- the last piece's sums
        ok = warp_all(ok && wait(&sm.o_full, (pc - 1u) & 1u, tmo, &sm.abort));
#pragma unroll
        for (int r = 0; r < kR; ++r) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
          if (lane == r) sm.red[rg][r][qd] = l[r];
        }
      }
      stop = ptx::named_bar_or(bar_id, kGroupThreads, !ok);
      if (stop) break;
      if (!first) {
        // ---- and parts
        const uint32_t par = (pc - 1u) % kRowSets;
        ptx::tc_fence_after();
        const size_t part0 = size_t(s_idx) * size_t(p.T) * p.Hq;
        const unsigned long long hits = sm.hit[par];
        if (n_mine > 0) {
          float inv[kR], ex[kR];
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(sm.red[rg][r]);
            const float L = (a.x + a.y) + (a.z + a.w);
            inv[r] = L == 0.f ? 0.f : 1.f / L;
            ex[r] = ex2(0.5f * (ref[r] - ml[r]));
            if (s_idx >= 0 && key_in == r && r < n_mine)
              p.lse_parts[part0 + sm.row[par][rg * kR + r]] =
                  L == 0.f ? -INFINITY : (ml[r] + __log2f(L)) * kLn2;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            __syncwarp();
            uint32_t a[8], b[8], c[8];
            const uint32_t ta = trow + C::kTmO + h * C::kStep;
            ptx::tmem_ld8x3_wait(ta, ta + MB, ta + 2 * MB, a, b, c);
            const int dim = h * 128 + key_in;
#pragma unroll
            for (int i = 0; i < kR; ++i) {
              if (i >= n_mine || s_idx < 0) continue;
              const int r = rg * kR + i;
              float o = fmaf(__uint_as_float(c[i]), 1.f / 1024.f,
                             fmaf(__uint_as_float(b[i]), 1.f / 32.f, __uint_as_float(a[i])));
              o = o * inv[i] * ex[i] * ex[i];
              if (hits != 0ull)
                o = put_back_nan(p, seq, head, hits, pr_lo, sm.lim[par][r], tree, base,
                                 sm.mask[par][r], dim, o);
              p.o_parts[(part0 + sm.row[par][r]) * 256 + dim] = o;
            }
          }
        }
        ptx::tc_fence_before();
      }
      if (!more) break;
      const uint32_t par = pc % kRowSets;
      ok = ok && wait(&sm.q_full, pc & 1u, tmo, &sm.abort);   // rows, limits, factors are written
      const int n_tiles = x.n_tiles, k_lo = x.k_lo, k_hi = x.k_hi;
      seq = x.b;
      head = x.g;
      s_idx = x.s;
      n_mine = min(max(x.rows * p.gqa - x.rb * MB - rg * kR, 0), kR);   // this group's rows
      base = x.kv_len - x.rows;
      // keys from pr_lo on are seen by some rows of the block only
      pr_lo = max(k_lo, tree ? base : base + x.rb * MB / p.gqa + 1);
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        ref[r] = kNone;
        ml[r] = kNone;
        l[r] = 0.f;
      }
      float peak = kNone;   // lanes 2 r, 2 r + 1: the highest that ref[r] was
      bool look = false;    // the next tile's maxima are wanted (the same in all threads)
      for (int j = 0; j < n_tiles; ++j, ++J) {
        const uint32_t buf = J & 1u;
        const int key = k_lo + j * kTile + key_in;
        const int tile_end = k_lo + (j + 1) * kTile;
        // This group's rows only; a group without rows keeps step with the others.
        ok = ok && wait(&sm.s_full[buf], (J >> 1) & 1u, tmo, &sm.abort);
        uint2 w[kPTerms];
#pragma unroll
        for (int t = 0; t < kPTerms; ++t) w[t] = make_uint2(0u, 0u);
        if (n_mine > 0) {
          float s[kR], d[kR];   // log2 scores; with vs, minus p's reference
          float lv = 0.f;
          bool need = false;
          ok = ok && wait(&sm.sc_full[J % kScaleRing], (J / kScaleRing) & 1u, tmo, &sm.abort);
          ok = warp_all(ok);
          __syncwarp();
          if (ok) {
            ptx::tc_fence_after();
            float sk = sm.scale[J % kScaleRing][0][key_in >> p.bs_log2];
            const float sv = sm.scale[J % kScaleRing][1][key_in >> p.bs_log2];
            if (key >= k_hi) {
              sk = 0.f;
            } else {
              lv = log2_scale(sv);
            }
            const uint32_t sa = trow + C::kTmS + buf * C::kStep;
            uint32_t a[8], b[8];
            if constexpr (kF16) {
              uint32_t c[8];
              ptx::tmem_ld8x3_wait(sa, sa + MB, sa + 2 * MB, a, b, c);
#pragma unroll
              for (int r = 0; r < kR; ++r)
                s[r] = fmaf(__uint_as_float(c[r]), 0.00390625f,
                            fmaf(__uint_as_float(b[r]), 0.0625f, __uint_as_float(a[r])));
            } else {
              ptx::tmem_ld8x2_wait(sa, sa + MB, a, b);
#pragma unroll
              for (int r = 0; r < kR; ++r)
                s[r] = fmaf(__uint_as_float(b[r]), 0.0625f, __uint_as_float(a[r]));
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) s[r] = s[r] * sm.fac[par][rg * kR + r] * sk;
            if (tile_end > pr_lo || tile_end > k_hi) {
#pragma unroll
              for (int r = 0; r < kR; ++r) {
                const bool vis =
                    key < min(sm.lim[par][rg * kR + r], k_hi) &&
                    (!tree || key < base || ((sm.mask[par][rg * kR + r] >> (key - base)) & 1ull));
                if (!vis) s[r] = -INFINITY;
              }
            }
            float md = -INFINITY, me = -INFINITY;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              d[r] = (s[r] - ref[r]) + lv;
              md = fmaxf(md, d[r]);
              me = fmaxf(me, s[r] - ml[r]);
            }
            need = md > kSlack || me > kLSlack ||
                   (n_tiles > kLongPiece && (look || (j & (kLook - 1)) == 1));
          }
          // ---- does a reference have to move (or has a wait run out)?
          bool moved = false;
          float alpha[kR];
          if (!ok) sm.failed[rg] = 1;
          if (ptx::named_bar_or(bar_id, kGroupThreads, need || !ok)) {
            if (sm.failed[rg]) {   // written before the barrier, by this group alone
              stop = true;
              break;
            }
            {
              float v[2 * kR];
#pragma unroll
              for (int r = 0; r < kR; ++r) {
                v[r] = s[r] + lv;
                v[kR + r] = s[r];
              }
              const float m = warp_max16(v);
              if ((lane & 1) == 0) sm.red[rg][lane >> 1][qd] = m;
            }
            ptx::named_bar_sync_any(bar_id, kGroupThreads);
            // lane 2 i, 2 i + 1: the i-th maximum over the tile
            const float4 q4 = *reinterpret_cast<const float4*>(sm.red[rg][lane >> 1]);
            const float top = fmaxf(fmaxf(q4.x, q4.y), fmaxf(q4.z, q4.w));
            bool move = false;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
              const float ma = __shfl_sync(0xffffffffu, top, 2 * r);
              const float mc = __shfl_sync(0xffffffffu, top, 2 * (kR + r));
              const bool up = ma > ref[r] + kSlack, up_l = mc > ml[r] + kLSlack;
              alpha[r] = up ? ex2(ref[r] - (ma - kTop)) : 1.f;
              ref[r] = up ? ma - kTop : ref[r];
              move = move || up;
              l[r] *= up_l ? ex2(ml[r] - mc) : 1.f;
              ml[r] = up_l ? mc : ml[r];
              d[r] = (s[r] - ref[r]) + lv;
            }
            if (n_tiles > kLongPiece) {
              look = false;
#pragma unroll
              for (int r = 0; r < kR; ++r) {
                const float ma = __shfl_sync(0xffffffffu, top, 2 * r);
                const float pk = __shfl_sync(0xffffffffu, peak, 2 * r);
                look = look || ref[r] > pk + kJump;
                if (ma < ref[r] + kFall && ma > pk - kDrop) {
                  alpha[r] = ex2(ref[r] - ma);
                  ref[r] = ma;
                  d[r] = (s[r] - ref[r]) + lv;
                  move = true;
                }
                if ((lane >> 1) == r) peak = fmaxf(pk, ref[r]);
              }
            }
            moved = move && j > 0;   // the same in all threads: references and maxima are
          }
          // ---- P's terms
#pragma unroll
          for (int i = 0; i < kR / 4; ++i) {
            if (4 * i >= n_mine) break;
            float pr[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              l[4 * i + c] += ex2(s[4 * i + c] - ml[4 * i + c]);
              pr[c] = ex2(d[4 * i + c]);
            }
            uint32_t lo[kPTerms], hi[kPTerms];
            p_terms(pr[0], pr[1], lo);
            p_terms(pr[2], pr[3], hi);
#pragma unroll
            for (int t = 0; t < kPTerms; ++t) (i == 0 ? w[t].x : w[t].y) = lo[t] | (hi[t] << 16);
          }
          if (moved) {
            // O, with PV of tile J - 1 in it, moves to the new references only now: the terms
            // above were computed while that product ran
            ok = warp_all(ok && wait(&sm.pv_done[buf ^ 1u], ((J - 1) >> 1) & 1u, tmo, &sm.abort));
            __syncwarp();
            if (ok) {
              ptx::tc_fence_after();
#pragma unroll 1
              for (int h = 0; h < 2; ++h) rescale_cols<MB>(trow + C::kTmO + h * C::kStep, alpha);
            }
          }
        }
        if (rg == 0 && (tile_end > k_hi || tile_end > pr_lo)) {
          ok = ok && wait(&sm.v_full[J % C::kVS], (J / C::kVS) & 1u, tmo, &sm.abort);
          if (ok && (key >= k_hi || key >= pr_lo) &&
              clean_v_row(sm.v[J % C::kVS], key_in, key >= k_hi))
            atomicOr(&sm.hit[par], 1ull << (key - pr_lo));
        }
        // PV of tile J - 2 has read this buffer: it was issued before S of tile J, whose
        // completion (s_full) covers every product issued before it.
        ok = warp_all(ok);
        if (ok) {
#pragma unroll
          for (int t = 0; t < kPTerms; ++t) {
            const int c8 = t * C::kGroups + rg;   // which 8 columns
            *reinterpret_cast<uint2*>(sm.p[buf] + (c8 >> 1) * (kTile * 16) + key_in * 16 +
                                      (c8 & 1) * 8) = w[t];
          }
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sm.p_full[buf]);
        }
      }
      ++pc;
      if (stop) break;
    }
    if (stop && key_in == 0) {
      sm.abort = 1;
      record_status(p.ctl.status, GQA_ERR_TIMEOUT);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, C::kCols);
}

template <int MB, bool kF16>
cudaError_t launch_t(const Kv8AttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                     long long grid, cudaStream_t stream) {
  const size_t smem = sizeof(AttnSmem<MB, kF16>) + 1024;
  static_assert(sizeof(AttnSmem<MB, kF16>) + 1024 <= 227 * 1024, "one CTA per SM");
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e =
      allow_smem_once(allowed, reinterpret_cast<const void*>(kv8_attn_kernel<MB, kF16>), smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv8_attn_kernel<MB, kF16>, dim3(unsigned(grid)), Cfg<MB, kF16>::kThreads, smem,
                       stream, 1, tmK, tmV, a);
  if (e == cudaSuccess) {
    static const char* const kNames[3][2] = {
        {"kv8_attn_kernel<16,bf16>", "kv8_attn_kernel<16,fp16>"},
        {"kv8_attn_kernel<24,bf16>", "kv8_attn_kernel<24,fp16>"},
        {"kv8_attn_kernel<32,bf16>", "kv8_attn_kernel<32,fp16>"}};
    note_launch(kNames[MB / 8 - 2][kF16], grid, Cfg<MB, kF16>::kThreads, smem);
  }
  return e;
}

}  // namespace

// 16, 24, 32 or 128 packed rows share a tile.  Up to 32 rows fewer columns cost less (8 x 4 draft
// rows x 6 heads, 24 packed: 74 us in tiles of 24, 80 of 32, 93 of 128); past 32 a
// second row block would read the cache again, which the wide kernel's 128 rows do not (its
// own comment has both sides measured).
int kv8_rows_per_block(long long packed_rows) {
  return packed_rows <= 16 ? 16 : packed_rows <= 24 ? 24 : packed_rows <= 32 ? 32 : 128;
}

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, bool f16, int sms, cudaStream_t stream,
                            bool* encode_failed) {
  CUtensorMap tmK, tmV;
  const int mb = kv8_rows_per_block((long long)a.max_rows * a.gqa);
  if (mb == 128) return launch_kv8_wide(a, f16, sms, stream, encode_failed);
  *encode_failed = !encode_pools(&tmK, &tmV, a);
  if (*encode_failed) return cudaSuccess;
  const long long tiles = (a.max_kv_len + kTile - 1) / kTile;
  const long long most = (long long)a.B * a.Hkv * a.max_rb * tiles;   // < 2^31: the caller's check
  const long long grid = most < sms ? most : sms;
  if (mb == 16)
    return f16 ? launch_t<16, true>(a, tmK, tmV, grid, stream)
               : launch_t<16, false>(a, tmK, tmV, grid, stream);
  if (mb == 24)
    return f16 ? launch_t<24, true>(a, tmK, tmV, grid, stream)
               : launch_t<24, false>(a, tmK, tmV, grid, stream);
  return f16 ? launch_t<32, true>(a, tmK, tmV, grid, stream)
             : launch_t<32, false>(a, tmK, tmV, grid, stream);
}

}  // namespace gqa
