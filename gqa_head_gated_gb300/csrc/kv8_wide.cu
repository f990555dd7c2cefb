// The attention of many rows (wide draft trees, prompt chunks) over the paged 8-bit cache: 128
// packed rows (query heads of a KV group x new rows) share each tile.  The mathematics, parts
// and schedule are kv8_attn.cu's; what differs is the side of the product that the rows take,
// and the terms:
//
//   S [rows, 128 keys] = Q . K^T       A = Q's terms, B = the tile's K, as it lies
//   O [rows, 256]     += P . V         A = P's terms (tensor memory), B = V, the same bytes
//
// Q is e4m3 terms (two for a bf16's 8 bits, three for an fp16's 11) that add up in one
// accumulator, with no scale between them: what a row's elements lose is below 2^-19 of its
// largest.  P is e5m2 terms, again in one accumulator: e5m2 has 3 bits a term but the range of
// fp16, so that p <= 2^15 splits into three (four) terms with a relative error of 2^-8.8 (2^-11)
// at most, a bf16 (fp16) P's own, and an absolute one of 2^-17: 2^-26 of the row's largest when its
// reference has just moved (to 2^9; 2^7 and 2^8 are as fast) and less after.  In pieces of more than
// 64 tiles the reference goes down again where the keys stay far below it, as in kv8_attn.cu (40
// trees of 16 rows x 6 heads over 65536 keys, one in a hundred with 8 times the score: 1,205 us,
// 1,128 without).  One accumulator for all terms is what leaves
// room for 128 rows: with e4m3 terms a column or lane each, as the kernel for few rows
// has them, O alone would take three times 256 columns.
//
// What bounds it: the softmax's latency beside the tensor pipe.  A tile has 2 x 8 products of 64
// clocks for S and 3 x 4 of 128 for P.V, 2,560 clocks (shared memory: 2,250 for their operands
// and the copies; HBM: 2,800 for 64 KB), and takes about 3,800.  The rows of a draft tree
// that pass 128 packed rows read the cache once more, through L2 or HBM.
//
// Two teams of 8 warps take the tiles in turn, so that one's softmax runs beside the other's and
// beside the products.  That takes two buffers of scores, for which tensor memory has room
// only because a tile's P goes where its scores were: each warp loads 32 keys' scores and
// stores their terms over them.  S of tile J + 2 is issued behind P.V of tile J, whose P it
// overwrites.  The references pass from tile to tile through shared memory (ref_full), and a
// row's l is kept apart in the four warps that share it.  Measured, 8 trees of 1 to 32 rows x 8
// heads, keys 4 K to 64 K: 150 us (548 MB, 3.7 TB/s at 128-row blocks); all 16 warps on one
// tile at a time, 32 keys each, 163 us; terms by conversion instructions, not by masks, took
// a tile 5,300 cycles for 4,200.  With a limit of 96 registers a thread, code that makes
// values live across a call (a rescale out of line) costs 30 us in spills.
//
// The kernel for few rows reads the cache once for 32 rows; 36 packed rows and more are faster
// here (the same trees: 314 us there in row blocks of 32), 24 are not (8 x 4 draft rows x 6
// heads: 74 us there, 93 here).
//
// Roles (576 threads): warp 0 copies (K a tile ahead of V: S runs two tiles ahead of P.V), warp 1
// issues the products, warps 2..17 are the softmax and epilogue: tensor-memory lane = row, two
// warps of a team share a quadrant's rows, 64 keys each.
// TMEM: O 256 columns, two buffers of 128 for S and, 8 columns a term and 32 keys, P.
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv8_attn.cuh"

namespace gqa {
namespace {

constexpr int kRows = 128;
constexpr int kTeams = 2;              // a team of 8 warps takes every other tile
constexpr int kHalves = 2;             // softmax threads of a row in a team
constexpr int kMine = kTile / kHalves; // keys of each
constexpr int kWarpsS = 4 * kTeams * kHalves;   // softmax warps
constexpr int kWarpsTeam = kWarpsS / kTeams;
constexpr int kShare = kTeams * kHalves;        // warps of a quadrant, which share the epilogue
constexpr int kCols = 256 / kShare;    // columns of O of each there
constexpr int kWideThreads = 64 + 32 * kWarpsS;
template <bool kF16>
struct WideCfg {
  static constexpr int kQTerms = kF16 ? 3 : 2, kPTerms = kF16 ? 4 : 3;
  // K and V slots.  One K slot does: the next K lands while the teams' softmax goes on; fp16's
  // third Q term takes the other's place.
  static constexpr int kKS = kF16 ? 1 : 2, kVS = 2;
};
constexpr uint32_t kTmWideO = 0, kTmWideS = 256;   // two buffers of 128 columns for S and P
constexpr float kWideCap = 15.f;       // p <= 2^15
constexpr float kWideTop = 9.f;        // a moved reference leaves the row's largest p at 2^9
// One that has come to stand too high goes down again, to where a tile's largest p is 2^kWideLow: when
// that was below 2^kWideFall and above 2^-kWideDrop of the highest reference (2^-31 of the row's
// largest p, as in kv8_attn.cu), in a piece's second tile and every 16th from there.
constexpr float kWideFall = -6.f, kWideDrop = 22.f, kWideLow = 5.f;
constexpr int kWideLook = 16;
constexpr uint32_t kIdescS = ptx::idesc_f32acc(128, 128, 0, 0, 0);
// A e5m2 (format 1), B e4m3 (format 0), B MN-major
constexpr uint32_t kIdescO = ptx::idesc_f32acc(128, 256, 0, 1, 0) | (1u << 7);

template <bool kF16>
struct __align__(1024) WideSmem : RingSmem<WideCfg<kF16>::kKS, WideCfg<kF16>::kVS> {
  alignas(1024) uint8_t q[WideCfg<kF16>::kQTerms][2][kRows * 128];   // [term][half of D][row][128 bytes, swizzled]
  float2 red[kTeams][kHalves][kRows];      // by row: maxima with vs, without
  float2 refs[2][kRows];                   // [tile parity][row]: the references after the tile
  float peak[kRows];                       // and the highest that p's was
  float sum[kShare][kRows];                // [share][row]
  // by tile parity: scores done; terms stored; by quadrant, references published and read
  uint64_t s_full[2], p_full[2], ref_full[2][4], pv_done, q_full, o_full, o_free, drain;
  // by piece, kRowSets in turn
  unsigned long long hit[kRowSets][2];     // NaN V rows taken out: bits of keys pr_lo + 64 w + i
  unsigned long long mask[kRowSets][kRows];
  int lim[kRowSets][kRows], row[kRowSets][kRows];
  float fac[kRowSets][kRows];
};

// D[tmem] (+)= A[tmem] * B[smem desc], 8-bit inputs.
__device__ __forceinline__ void mma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four probabilities as e5m2 terms, a word of four bytes per term.  They go as
// fp16 (a rounding of 2^-11 at most), whose remainders are exact.  An e5m2 number is the upper
// byte of the fp16 of the same value, so rounding to it is an integer add and a mask, for two
// values at once (the sums stay below 2^16): the conversion instructions made the terms of a
// tile take 1,700 cycles.  The last of a bf16's three terms has two bits to round, so that one
// value in four lies half way: even keys go down there and odd ones up, which leaves a mean of
// 4e-7 (all up: 1.6e-4 too much of V, beside an exact sum of the weights).  Four terms for bf16
// too took the draft trees 167 us for 148.  (A NaN loses its bits
// here; the row's sum, in fp32, keeps it.)
template <int kPTerms>
__device__ __forceinline__ void p_terms5(float2 lo, float2 hi, uint32_t (&w)[kPTerms]) {
  __half2 a = __floats2half2_rn(lo.x, lo.y), b = __floats2half2_rn(hi.x, hi.y);
#pragma unroll
  for (int i = 0; i < kPTerms; ++i) {
    const uint32_t up = i + 1 < kPTerms ? 0u : 0x0080007Fu;
    const uint32_t ta = (*reinterpret_cast<const uint32_t*>(&a) + up) & 0xFF00FF00u;
    const uint32_t tb = (*reinterpret_cast<const uint32_t*>(&b) + up) & 0xFF00FF00u;
    w[i] = __byte_perm(ta, tb, 0x7531);
    if (i + 1 < kPTerms) {
      a = __hsub2(a, *reinterpret_cast<const __half2*>(&ta));
      b = __hsub2(b, *reinterpret_cast<const __half2*>(&tb));
    }
  }
}

// Half of a row of O times f, in tensor memory (whole warp).
__device__ __forceinline__ void rescale_o(uint32_t ta, float f) {
#pragma unroll 1
  for (int c = 0; c < 256 / kHalves / 32; ++c) {
    uint32_t o[32];
    ptx::tmem_ld32_wait(ta + 32 * c, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
    ptx::tmem_st32_wait(ta + 32 * c, o);
  }
}

template <bool kF16>
__global__ void __launch_bounds__(kWideThreads, 1)
kv8_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const Kv8AttnArgs p) {
  using C = WideCfg<kF16>;
  constexpr int kPTerms = C::kPTerms, kQTerms = C::kQTerms;
  extern __shared__ uint8_t smem_raw[];
  WideSmem<kF16>& sm = *reinterpret_cast<WideSmem<kF16>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t tmo = p.ctl.timeout_ns;
  if (tid == 0) {
    init_ring(sm);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.s_full[i], 1);
      ptx::mbar_init(&sm.p_full[i], kWarpsTeam);
      for (int k = 0; k < 4; ++k) ptx::mbar_init(&sm.ref_full[i][k], kHalves);
    }
    ptx::mbar_init(&sm.pv_done, 1);
    ptx::mbar_init(&sm.o_free, kWarpsS);
    ptx::mbar_init(&sm.q_full, kWarpsS);
    ptx::mbar_init(&sm.o_full, 1);
    ptx::mbar_init(&sm.drain, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&sm.tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Share share = cut_shares<kRows>(sm, p);

  if (warp == 0) {
    copy_role<kRows, true>(sm, p, tmK, tmV, share);
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      const uint64_t qd = ptx::sdesc_sw128(ptx::smem_addr(sm.q), 16, 1024);
      uint32_t J = 0, pc = 0;
      bool ok = true;
      const auto issue_s = [&](uint32_t n) -> bool {
        const uint32_t ks = n % C::kKS;
        if (!wait(&sm.k_full[ks], (n / C::kKS) & 1u, tmo, &sm.abort)) return false;
        ptx::tc_fence_after();
        const uint64_t kd = ptx::sdesc_sw128(ptx::smem_addr(sm.k[ks]), 16, 1024);
#pragma unroll
        for (int t = 0; t < kQTerms; ++t)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ss_f8(tmem + kTmWideS + (n & 1u) * 128,
                           ptx::sdesc_at(qd, t * (2 * kRows * 128) + (kk >> 2) * (kRows * 128) + (kk & 3) * 32),
                           ptx::sdesc_at(kd, (kk >> 2) * kHalfBytes + (kk & 3) * 32), kIdescS,
                           t > 0 || kk > 0);
        ptx::tc_commit(&sm.s_full[n & 1u]);
        ptx::tc_commit(&sm.k_empty[ks]);
        return true;
      };
      const auto issue_pv = [&](uint32_t n, bool first) -> bool {
        const uint32_t vs = n % C::kVS;
        if (!wait(&sm.p_full[n & 1u], (n >> 1) & 1u, tmo, &sm.abort)) return false;
        if (!wait(&sm.v_full[vs], (n / C::kVS) & 1u, tmo, &sm.abort)) return false;
        ptx::tc_fence_after();
        const uint64_t vd = ptx::sdesc_sw128(ptx::smem_addr(sm.v[vs]), kHalfBytes, 1024);
#pragma unroll
        for (int t = 0; t < kPTerms; ++t)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts_f8(tmem + kTmWideO, tmem + kTmWideS + (n & 1u) * 128 + kk * 32 + t * 8,
                      ptx::sdesc_at(vd, kk * 4096), kIdescO, !first || t > 0 || kk > 0);
        ptx::tc_commit(&sm.pv_done);
        ptx::tc_commit(&sm.v_empty[vs]);
        return true;
      };
      while (ok) {
        ok = wait(&sm.piece_full[pc % kPieceRing], (pc / kPieceRing) & 1u, tmo, &sm.abort);
        if (!ok) break;
        const int n_tiles = sm.piece[pc % kPieceRing].n_tiles;
        if (n_tiles == 0) break;
        ok = wait(&sm.q_full, pc & 1u, tmo, &sm.abort);
        if (!ok) break;
        ptx::tc_fence_after();
        ok = issue_s(J);
        if (ok && n_tiles > 1) ok = issue_s(J + 1);
        // O of the last piece has been read by every warp
        if (ok && pc > 0) ok = wait(&sm.o_free, (pc - 1u) & 1u, tmo, &sm.abort);
        for (int j = 0; ok && j < n_tiles; ++j) {
          ok = issue_pv(J + j, j == 0);
          // S of tile j + 2 goes where P of tile j lies: products run in the order of issue
          if (ok && j + 2 < n_tiles) ok = issue_s(J + j + 2);
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
    const int sw = warp - 2;
    const int qt = sw >> 2;                    // this warp among its quadrant's
    const uint32_t team = qt & 1;              // tiles of this parity
    const int half = qt >> 1;                  // keys kMine half .. of a tile
    const int qd = warp & 3;                   // tensor-memory lanes 32 qd .. 32 qd + 31
    const int r = qd * 32 + lane;              // this thread's row of the block
    const uint32_t trow = tmem + (uint32_t(qd * 32) << 16);
    const bool tree = p.tree_mask != nullptr;
    const uint32_t bar_id = 1 + qd;            // the four warps of a quadrant
    const uint32_t pair_id = 5 + 2 * qd + team;   // those of a team
    constexpr int kBar = 32 * kShare, kPairBar = 32 * kHalves;
    uint32_t J = 0, pc = 0;
    // This warp's waits.  A pair agrees at its barrier in each tile; a pair that leaves there
    // takes the quadrant's next barrier on its way, so that the other one leaves at that.
    bool ok = true;
    bool stop = false;
    // Piece n's description stays in its ring until this warp is far past it.
    const auto piece = [&](uint32_t n) -> const Piece& { return sm.piece[n % kPieceRing]; };
    // Q's terms, the rows' limits and places of piece n; then its products may start.  The
    // last piece's S products are done.
    const auto prepare = [&](uint32_t n) {
      const uint32_t par = n % kRowSets;
      const Piece x = piece(n);
      const int p0 = x.rb * kRows, n_rows = min(kRows, x.rows * p.gqa - p0);
      if (sw < kRows / 32) {   // thread by row
        const int rr = sw * 32 + lane, i = (p0 + rr) / p.gqa;
        sm.row[par][rr] = (x.t0 + i) * p.Hq + x.g * p.gqa + (p0 + rr - i * p.gqa);
        sm.lim[par][rr] = rr >= n_rows ? 0 : tree ? x.kv_len : x.kv_len - x.rows + i + 1;
        sm.mask[par][rr] = tree && rr < n_rows ? p.tree_mask[x.t0 + i] : 0ull;
      }
#pragma unroll 1
      for (int r0 = sw; r0 < kRows; r0 += 4 * kWarpsS) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = r0 + k * kWarpsS, i = (p0 + rr) / p.gqa;
          const int row = (x.t0 + i) * p.Hq + x.g * p.gqa + (p0 + rr - i * p.gqa);
          u[k] = rr < n_rows ? __ldg(p.q + size_t(row) * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = r0 + k * kWarpsS;
          float f[8];
          const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 a = unpack_elem2<kF16>(w[c]);
            f[2 * c] = a.x;
            f[2 * c + 1] = a.y;
          }
          const int e = scale_exp(__reduce_max_sync(0xffffffffu, finite_amax_bits(f)));
          if (lane == 0) sm.fac[par][rr] = pow2f(e) * kScaleLog2;
          const float inv = pow2f(-e);
          // an infinite element makes its row's scores NaN, as in the formula
#pragma unroll
          for (int c = 0; c < 8; ++c) f[c] = isinf(f[c]) ? __int_as_float(0x7FC00000) : f[c] * inv;
#pragma unroll 1
          for (int t = 0; t < kQTerms; ++t) {
            uint2 o;
            o.x = take_term(f[0], f[1], 1.f);
            o.x |= take_term(f[2], f[3], 1.f) << 16;
            o.y = take_term(f[4], f[5], 1.f);
            o.y |= take_term(f[6], f[7], 1.f) << 16;
            *reinterpret_cast<uint2*>(sm.q[t][lane >> 4] + rr * 128 +
                                      ((((lane & 15) >> 1) ^ (rr & 7)) << 4) + (lane & 1) * 8) = o;
          }
        }
      }
      if (sw == 0 && lane < 2) sm.hit[par][lane] = 0ull;
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sm.q_full);
    };

    // First key of a piece that some rows of its block do not see (fewer than 128 are like it).
    const auto part_seen_from = [&](const Piece& x) {
      const int base = x.kv_len - x.rows;
      return max(x.k_lo, tree ? base : base + x.rb * kRows / p.gqa + 1);
    };
    float ref = kNone, ml = kNone, l = 0.f;
    for (bool first = true;; first = false) {
      // ---- the next piece may start while the last one ends (its S products are done)
      ok = warp_all(ok && wait(&sm.piece_full[pc % kPieceRing], (pc / kPieceRing) & 1u, tmo, &sm.abort));
      const bool more = ok && piece(pc).n_tiles > 0;
      if (more) prepare(pc);
      if (!first) {
        const uint32_t last = (J - 1u) & 1u, phase = ((J - 1u) >> 1) & 1u;
        ok = warp_all(ok && wait(&sm.ref_full[last][qd], phase, tmo, &sm.abort) &&
                      wait(&sm.o_full, (pc - 1u) & 1u, tmo, &sm.abort));
        const float2 fin = sm.refs[last][r];
        ref = fin.x;
        l *= ex2(ml - fin.y);
        ml = fin.y;
        sm.sum[qt][r] = l;
      }
      stop = ptx::named_bar_or(bar_id, kBar, !ok);
      if (stop) break;
      if (!first) {
        // ---- the last piece's parts: this thread's row, kCols of its columns
        ptx::tc_fence_after();
        const Piece& x = piece(pc - 1u);
        const uint32_t par = (pc - 1u) % kRowSets;
        float L = 0.f;
#pragma unroll
        for (int i = 0; i < kShare; ++i) L += sm.sum[i][r];
        const float inv = L == 0.f ? 0.f : 1.f / L, ex = ex2(0.5f * (ref - ml));
        const bool mine = x.s >= 0 && x.rb * kRows + r < x.rows * p.gqa;
        const size_t part = size_t(x.s) * size_t(p.T) * p.Hq + sm.row[par][r];
        if (mine && qt == 0) p.lse_parts[part] = L == 0.f ? -INFINITY : (ml + __log2f(L)) * kLn2;
        // Four lanes have 8 columns of a row (two rows) of each load; they exchange two, so that
        // a lane stores 16 bytes and the four 64 bytes in a row.
        const int ok_row = mine && L != 0.f;
#pragma unroll 1
        for (int n = 0; n < 2 * kCols / 32; ++n) {
          const int r16 = (n & 1) * 16, col = qt * kCols + (n >> 1) * 32;
          __syncwarp();
          uint32_t o[16];
          ptx::tmem_ld16x256_x4_wait(trow + (uint32_t(r16) << 16) + kTmWideO + col, o);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int of = r16 + h * 8 + (lane >> 2);      // the row, as a lane of the warp
            const float iv = __shfl_sync(0xffffffffu, inv, of), ev = __shfl_sync(0xffffffffu, ex, of);
            const bool in = __shfl_sync(0xffffffffu, ok_row, of) != 0;
            const size_t at = size_t(x.s) * size_t(p.T) * p.Hq + sm.row[par][qd * 32 + of];
#pragma unroll
            for (int k = 0; k < 2; ++k) {                  // columns 16 k .. 16 k + 15
              float a[4];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t lo = o[8 * k + 2 * h + c], hi = o[8 * k + 4 + 2 * h + c];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? lo : hi, 1);
                a[c] = __uint_as_float((lane & 1) ? got : lo);
                a[2 + c] = __uint_as_float((lane & 1) ? hi : got);
              }
              if (in)
                *reinterpret_cast<float4*>(p.o_parts + at * 256 + col + 16 * k + (lane & 1) * 8 +
                                           (lane & 2) * 2) =
                    make_float4(a[0] * iv * ev * ev, a[1] * iv * ev * ev, a[2] * iv * ev * ev,
                                a[3] * iv * ev * ev);
            }
          }
        }
        __syncwarp();
        const unsigned long long h0 = sm.hit[par][0], h1 = sm.hit[par][1];
        if ((h0 | h1) != 0ull && mine && L != 0.f) {
          // NaN values that were taken out, put back into what this thread wrote
          const int base = x.kv_len - x.rows, first_key = part_seen_from(x);
#pragma unroll 1
          for (int c = qt * kCols; c < (qt + 1) * kCols; ++c) {
            float v = p.o_parts[part * 256 + c];
            v = put_back_nan(p, x.b, x.g, h0, first_key, sm.lim[par][r], tree, base, sm.mask[par][r], c, v);
            v = put_back_nan(p, x.b, x.g, h1, first_key + 64, sm.lim[par][r], tree, base,
                             sm.mask[par][r], c, v);
            p.o_parts[part * 256 + c] = v;
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.o_free);
      }
      if (!more) break;
      const uint32_t par = pc % kRowSets;
      ok = ok && wait(&sm.q_full, pc & 1u, tmo, &sm.abort);   // rows, limits, factors are written
      const int n_tiles = piece(pc).n_tiles;
      // tiles from this one on have keys that some rows do not see
      const int part_from = (min(piece(pc).k_hi, part_seen_from(piece(pc))) - piece(pc).k_lo) / kTile;
      const float fac = sm.fac[par][r];
      ref = ml = kNone;
      l = 0.f;
      // Bit c: this thread's row sees key `key0` + c of the piece.
      const auto seen = [&](int key0) -> uint32_t {
        const Piece& x = piece(pc);
        const int n = min(sm.lim[par][r], x.k_hi) - key0;
        uint32_t bits = n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u;
        if (tree) {
          const int o = key0 - (x.kv_len - x.rows);
          const unsigned long long m = sm.mask[par][r];
          bits &= o >= 0 ? (o < 64 ? uint32_t(m >> o) : 0u)
                         : o > -32 ? (uint32_t(m) << -o) | ((1u << -o) - 1u) : 0xffffffffu;
        }
        return bits;
      };
      const auto hide = [&](uint32_t (&s)[32], int key0) {
        const uint32_t bits = seen(key0);
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((bits >> c) & 1u)) s[c] = 0xFF800000u;   // -inf
      };
      for (int j = 0; j < n_tiles; ++j, ++J) {
        const uint32_t buf = J & 1u;
        if (buf != team) continue;
        const bool part = j >= part_from;
        const uint32_t ts = trow + kTmWideS + buf * 128 + half * kMine;
        ok = ok && wait(&sm.sc_full[J % kScaleRing], (J / kScaleRing) & 1u, tmo, &sm.abort);
        float f[kMine / 16], lv[kMine / 16];   // by run of 16 keys: score factor, log2 of the V scale
#pragma unroll
        for (int i = 0; i < kMine / 16; ++i) {
          const int blk = (half * kMine + i * 16) >> p.bs_log2;
          // (of blocks behind the last key no scale was copied)
          const bool in = !part || piece(pc).k_lo + j * kTile + half * kMine + i * 16 < piece(pc).k_hi;
          // finite and not 0, so that a hidden key's -inf stays one and 0 stays 0
          f[i] = fminf(fmaxf(fac * (in ? sm.scale[J % kScaleRing][0][blk] : 1.f), 1e-37f), 3e38f);
          lv[i] = in ? log2_scale(sm.scale[J % kScaleRing][1][blk]) : 0.f;
        }
        ok = ok && wait(&sm.s_full[buf], (J >> 1) & 1u, tmo, &sm.abort);
        ok = warp_all(ok);
        __syncwarp();
        float mp = -INFINITY, ms = -INFINITY;
        if (ok) {
          ptx::tc_fence_after();
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) {
            uint32_t s[32];
            ptx::tmem_ld32_wait(ts + 32 * h, s);
            if (part) hide(s, piece(pc).k_lo + j * kTile + half * kMine + 32 * h);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float m0 = __uint_as_float(s[16 * i]), m1 = __uint_as_float(s[16 * i + 1]);
#pragma unroll
              for (int c = 2; c < 16; c += 2) {
                m0 = fmaxf(m0, __uint_as_float(s[16 * i + c]));
                m1 = fmaxf(m1, __uint_as_float(s[16 * i + c + 1]));
              }
              const float m = fmaxf(m0, m1) * f[2 * h + i];
              ms = fmaxf(ms, m);
              mp = fmaxf(mp, m + lv[2 * h + i]);
            }
          }
          sm.red[team][half][r] = make_float2(mp, ms);
        }
        if (ptx::named_bar_or(pair_id, kPairBar, !ok)) {
          stop = true;
          break;
        }
        {
          const float2 o = sm.red[team][half ^ 1][r];
          mp = fmaxf(mp, o.x);
          ms = fmaxf(ms, o.y);
        }
        // ---- references: those after the last tile, moved on (both threads of a row do the same)
        float2 at = make_float2(kNone, kNone);
        if (j > 0) {
          ok = warp_all(ok && wait(&sm.ref_full[buf ^ 1u][qd], ((J - 1u) >> 1) & 1u, tmo, &sm.abort));
          at = sm.refs[buf ^ 1u][r];
        }
        const bool up = mp > at.x + kWideCap, up_l = ms > at.y + kLSlack;
        ref = up ? mp - kWideTop : at.x;
        if (n_tiles > kLongPiece) {
          if ((j & (kWideLook - 1)) == 1 && mp < at.x + kWideFall &&
              mp > sm.peak[r] - kWideDrop)
            ref = mp - kWideLow;
          // (a row that falls here does not rise: its peak is not read in this tile)
          if (half == 0 && (j == 0 || up)) sm.peak[r] = j == 0 ? ref : fmaxf(sm.peak[r], ref);
        }
        if (up_l) at.y = ms;
        if (half == 0) sm.refs[buf][r] = make_float2(ref, at.y);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.ref_full[buf][qd]);
        l *= ex2(ml - at.y);
        ml = at.y;
        const bool moved = j > 0 && __any_sync(0xffffffffu, ref != at.x);
        const float alpha = ex2(at.x - ref);
        // ---- V rows that some row does not see
        if (part) {
          ok = ok && wait(&sm.v_full[J % C::kVS], (J / C::kVS) & 1u, tmo, &sm.abort);
          const int k_hi = piece(pc).k_hi, pr_lo = part_seen_from(piece(pc));
          const int key = piece(pc).k_lo + j * kTile + r;   // thread by key here, its half of the row
          if (ok && (key >= k_hi || key >= pr_lo) &&
              clean_v_row(sm.v[J % C::kVS], r, key >= k_hi, 16 / kHalves * half, 16 / kHalves * (half + 1)))
            atomicOr(&sm.hit[par][(key - pr_lo) >> 6], 1ull << ((key - pr_lo) & 63));
          ptx::fence_proxy_async_smem();
          ok = warp_all(ok);
          __syncwarp();
        }
        // ---- P's terms, a run of 16 keys at a time: those of 32 keys go where their scores were
        if (ok) {
#pragma unroll
          for (int h = 0; h < kMine / 32; ++h) {
            uint32_t s[32];
            ptx::tmem_ld32_wait(ts + 32 * h, s);
            if (part) hide(s, piece(pc).k_lo + j * kTile + half * kMine + 32 * h);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float fi = f[2 * h + i], a = lv[2 * h + i] - ref;
              const float2 f2 = make_float2(fi, fi), a2 = make_float2(a, a);
              // l's terms from p's: p * 2^(ref - log2 vs - ml), unless p may have lost them (a
              // block of tiny values that p hardly sees)
              const float d = -a - ml;
              const bool far = __any_sync(0xffffffffu, d > 60.f);
              if (far) {
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 16; ++c) sum += ex2(fmaf(__uint_as_float(s[16 * i + c]), fi, -ml));
                l += sum;
              }
              float2 sum2 = make_float2(0.f, 0.f);
              uint32_t w[kPTerms][4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int k = 16 * i + 4 * c;
                const float2 x0 = fma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), f2, a2);
                const float2 x1 = fma2(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), f2, a2);
                const float2 e0 = make_float2(ex2(x0.x), ex2(x0.y)), e1 = make_float2(ex2(x1.x), ex2(x1.y));
                sum2 = add2(sum2, add2(e0, e1));
                uint32_t t4[kPTerms];
                p_terms5(e0, e1, t4);
#pragma unroll
                for (int t = 0; t < kPTerms; ++t) w[t][c] = t4[t];
              }
              if (!far) l += (sum2.x + sum2.y) * ex2(d);
#pragma unroll
              for (int t = 0; t < kPTerms; ++t) ptx::tmem_st4(ts + 32 * h + 8 * t + 4 * i, w[t]);
            }
          }
          ptx::tmem_wait_st();
        }
        if (moved) {
          // O, with PV of tile J - 1 in it, moves to the new references only now: the terms
          // were computed while that product ran
          ok = warp_all(ok && wait(&sm.pv_done, (J - 1u) & 1u, tmo, &sm.abort));
          __syncwarp();
          if (ok) {
            ptx::tc_fence_after();
            rescale_o(trow + kTmWideO + half * (256 / kHalves), alpha);
          }
        }
        if (ok) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sm.p_full[buf]);
        }
      }
      // S of the last tile, be it the other team's, has read Q before the next piece's is written
      if (!stop)
        ok = warp_all(ok && wait(&sm.s_full[(J - 1u) & 1u], ((J - 1u) >> 1) & 1u, tmo, &sm.abort));
      ++pc;
      if (stop) {
        ptx::named_bar_or(bar_id, kBar, true);
        break;
      }
    }
    if (stop && lane == 0) {
      sm.abort = 1;
      record_status(p.ctl.status, GQA_ERR_TIMEOUT);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

template <bool kF16>
cudaError_t launch_wide_t(const Kv8AttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          long long grid, cudaStream_t stream) {
  const size_t smem = sizeof(WideSmem<kF16>) + 1024;
  static_assert(sizeof(WideSmem<kF16>) + 1024 <= 227 * 1024, "one CTA per SM");
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem_once(allowed, reinterpret_cast<const void*>(kv8_wide_kernel<kF16>), smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv8_wide_kernel<kF16>, dim3(unsigned(grid)), kWideThreads, smem, stream, 1, tmK,
                       tmV, a);
  if (e == cudaSuccess)
    note_launch(kF16 ? "kv8_wide_kernel<fp16>" : "kv8_wide_kernel<bf16>", grid, kWideThreads, smem);
  return e;
}

}  // namespace

cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, bool f16, int sms, cudaStream_t stream,
                            bool* encode_failed) {
  CUtensorMap tmK, tmV;
  *encode_failed = !encode_pools(&tmK, &tmV, a);
  if (*encode_failed) return cudaSuccess;
  const long long tiles = (a.max_kv_len + kTile - 1) / kTile;
  const long long most = (long long)a.B * a.Hkv * a.max_rb * tiles;
  const long long grid = most < sms ? most : sms;
  return f16 ? launch_wide_t<true>(a, tmK, tmV, grid, stream)
             : launch_wide_t<false>(a, tmK, tmV, grid, stream);
}

}  // namespace gqa
