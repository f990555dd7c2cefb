// Attention of prompt chunks over the paged 8-bit cache, on CTA pairs (tcgen05 .cta_group::2):
//
//   out[t] = softmax_j(q[t] . K[j] / 16, j <= base + i) V * sigmoid(g[t]),   K[j] = k_pool row * scale
//
// for every new row i of every sequence (base = kv_len - rows).  A segment is 256 packed rows (query
// heads of a KV group x new rows, heads innermost) of one sequence; each CTA of a pair has 128 of
// them, and the two share each tile of 128 keys: CTA r brings keys 64 r .. of K and dims 128 r .. of V.
//
// Scores are 8-bit products of the keys as they lie and of Q as e4m3 terms (two for a bf16's 8 bits, three for
// an fp16's 11; what a row's elements lose is below 2^-19 of its largest), K's scale goes in after, per
// run of 16 keys.  P.V is a 16-bit product: an e4m3 number is an fp16 number, so V enters as it is stored and its
// scale goes into the exponent of the probability, p = 2^(score + log2 vs - ref).  p goes as fp16: off by
// 2^-11 of itself, and by 2^-25 at least.  A reference moves when p would pass 2^15, and then leaves the largest at
// 2^top, which the row's largest does not fall below.  In a piece of 64 tiles or fewer top is 0: its 8192 keys lose
// 2^-12 of that one's weight at most, together.  In a longer one it is 8, so that very many keys far below one keep
// theirs: 131071 keys 18 nats below come out within 2^-7 (with 0 they were lost, and 1.76 times themselves at 17.2).
// It costs moves of O: 2048 rows at 30720 keys 646 us for 637 (with 10 for 8: 650), ragged fp16 chunks 1640 for 1613; in
// every piece it would cost 8192 rows 606 for 592, and 4 x 37 behind 65000 111 for 108.  The row's sum l is taken from the
// fp32 probabilities against a reference of its own, without the V scales.
//
// What bounds it: 2 x 1024 tensor clocks a tile of 128 rows x 128 keys (three 8-bit terms of p, as the kernels for
// few rows have them, would take 2560 in all; fp16 takes 2560), beside 1024 clocks of ex2.  Measured, bf16, new inputs at
// each call: 2048 rows behind 30720 keys 645 us (1,650 TFLOP/s of 1,919), a prompt of 8192 rows 592 us (1,390: 768
// segments' starts and ends show); fp16 costs its third term.
//
// The hot loops are small on purpose, but for the issuing warp's: five roles share an SM's instruction caches (the
// softmax unrolled over all of a row's keys: 1077 us), while operands made in a loop make a product's issue longer than its
// 64 clocks (856 us for 718).
//
// The segments' tiles (only those that some row sees) are laid end to end and cut into equal shares,
// one a pair.  A piece that is a whole segment goes straight to `out`; the pieces of a segment that is
// cut leave fp32 parts, two a pair at most, that kv8_join_kernel puts together.
//
// Roles (512 threads): warp 0 schedules (pieces, block numbers and scales of the tiles), warp 1 of the even
// CTA issues the products, warp 2 copies K, warps 4..7 convert V into shared memory, warps 8..15 are softmax and
// epilogue: a thread has a row (its tensor-memory lane) and 64 keys of each tile.
// TMEM: O 256 columns, two buffers of 128 for S and P.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "kv8_attn.cuh"

namespace gqa {
namespace {

constexpr int kPairRows = 256;                  // packed rows of a segment
constexpr int kThreadsC = 512;                  // four warpgroups: schedule and products, conversion, softmax
constexpr int kConvWarp = 4, kSoftWarp = 8;     // first warps
// Registers a thread, by warpgroup, out of the launch's 128 (inc waits until they are there).
constexpr int kRegsRest = 80, kRegsConv = 112, kRegsSoft = 160;
static_assert(kRegsRest + kRegsConv + 2 * kRegsSoft <= 4 * 128, "the launch's registers");
constexpr int kSlotK = 16384, kKs = 2;          // half a tile of K as it lies; slots
constexpr int kSlotV = 32768, kVs = 2;          // half a tile of V in fp16
constexpr int kGroup = 4;                       // tiles that the scheduler looks up together
constexpr int kGroups = 4;                      // groups held
constexpr int kTiles = kGroup * kGroups;
constexpr int kPieces = 32;                     // more than tiles held, and every piece has one
constexpr int kHitSets = 4;                     // pieces whose NaN keys are held
constexpr int kHitWords = kPairRows / 32;       // keys that only some rows of a segment see: < 256
// What a segment costs beside its tiles, in tiles (Q's terms, the first tiles, whose references still move, the
// end).  8192 rows with 4, 6, 7, 8, 10 and 12: 711, 649, 607, 582, 597, 597 us.
constexpr uint32_t kLead = 8;
constexpr int kSnap = 2;                        // a cut this close to a segment's end is made there
// No segment is cut where there is a pair for each and the longest is at most this many tiles above an equal share:
// parts and their joining cost as much (24/4 heads, with 0, 6, 10 and 14: 16 sequences of 40 rows behind 2000 keys 60, 50,
// 50, 50 us; of 42 behind 4000 84, 75, 75, 78; 4 of 64 behind 1000 39, 35, 33, 33; 512 rows behind 2000 55, 55, 50, 49;
// 64 behind 1000 29, 29, 32, 32).
constexpr uint32_t kWhole = 10;
constexpr float kCap = 15.f;                    // p <= 2^15
constexpr float kLongTop = 8.f;                 // what a moved reference leaves in a piece of more than kLongPiece tiles
constexpr uint32_t kTmOc = 0, kTmSc = 256;
constexpr uint32_t kIdescSc = ptx::idesc_f32acc(256, 128, 0, 0, 0);   // e4m3 (format 0)
constexpr uint32_t kIdescOc = ptx::idesc_f32acc(256, 256, 0, 1, 0);   // fp16 (format 0)

struct ChunkArgs {
  const uint4* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const uint16_t* gate;
  const int* tables;
  const int* kv_lens;
  const int* cu_rows;
  uint16_t* out;
  float* lse;
  float* o_parts;      // [2 * pairs][256][256]
  float* lse_parts;    // [2 * pairs][256]
  int* cuts;           // [pairs][8]: see the scheduler
  int B, T, Hkv, Hq, gqa, num_blocks, bs_log2, max_blocks, max_rows, max_kv_len, pairs;
  LaunchCtl ctl;
};

// A place in the row of all segments: sequence, KV head, row block, tile.
struct Cut {
  int b, g, rb, t;
};

struct ChunkPiece {
  int b, g, rb, rows, t0, base;   // base: keys before the new rows
  int part;                    // -1: a whole segment
};

struct TileRec {
  int key0, k_hi, pr_lo;       // first key; keys from k_hi on are not there; from pr_lo on not all rows see
  int g, n_tiles, piece;       // n_tiles of the piece that starts here; 0: the end of the share
  int last;                    // of its piece
  float lv_min;
  int blk[8];                  // by run of 16 keys: block, scale of K, log2 of V's
  float ks[8], lv[8];
};

template <bool kF16>
struct __align__(1024) ChunkSmem {
  static constexpr int kQTerms = kF16 ? 3 : 2;
  uint8_t q[kQTerms][2][128 * 128];       // [term][half of D][row][128 bytes, swizzled]
  uint8_t k[kKs][kSlotK], v[kVs][kSlotV];
  TileRec rec[kTiles];
  ChunkPiece piece[kPieces];
  float2 red[2][2][128];                  // [tile parity][half][row]: maxima with vs, without
  float sum[2][128];                      // [half][row]
  float fac[2][128];                      // by piece parity
  uint32_t hit[kHitSets][kHitWords];
  uint64_t rec_full[kGroups], rec_empty[kGroups];
  // By tile parity: K has landed; S is done, and its K slot free; V and P are there; PV is done, its V slot free.  None
  // can come round again before all of its users have waited: each of them arrives on what leads to the next phase, the
  // odd CTA's copying warp too where it has no key of a tile to bring.
  uint64_t k_full[2], s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, o_free, drain;
  uint64_t hit_full[kHitSets];
  int4 seq[kKv8Seqs];                     // first token, rows, keys, row blocks
  uint32_t cost[kKv8Seqs], at[kKv8Seqs + 1];   // of one KV head; of all, before each sequence
  uint32_t segments, longest, whole;      // of the launch; tiles; none is cut, and each costs 1
  uint32_t tmem_base;
  int abort, zero;
};
static_assert(sizeof(ChunkSmem<true>) + 1024 <= 227 * 1024, "one CTA per SM");

template <int N>
__device__ __forceinline__ void take_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void leave_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Arrives on a barrier of the even CTA: each CTA's own, or through the cluster's window.
__device__ __forceinline__ void arrive_lead(uint64_t* bar, bool lead) {
  if (lead) ptx::mbar_arrive(bar); else ptx::mbar_arrive_remote(ptx::mapa_shared(ptx::smem_addr(bar), 0));
}

// Tiles that some row of row block rb sees.
__device__ __forceinline__ int tiles_of(const int4& s, int rb, int gqa) {
  const int rows = min(s.y, ((rb + 1) * kPairRows - 1) / gqa + 1);
  return (s.z - s.y + rows + kTile - 1) / kTile;
}

// The cut at position pos of the launch's segments (whole warp): at a segment's end where one is near.
template <typename Sm>
__device__ Cut cut_at(const Sm& sm, const ChunkArgs& p, uint32_t pos) {
  const int lane = threadIdx.x & 31;
  if (pos >= sm.at[p.B]) return Cut{p.B, 0, 0, 0};
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.at[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  const int4 s = sm.seq[lo];
  uint32_t rest = pos - sm.at[lo];
  Cut c{lo, int(rest / sm.cost[lo]), 0, 0};
  rest -= uint32_t(c.g) * sm.cost[lo];
  int n = 0;
  for (int rb0 = 0;; rb0 += 32) {   // (the last row block's sum is the cost, which rest is below)
    const uint32_t own = rb0 + lane >= s.w ? 0u
                         : sm.whole != 0u  ? 1u
                                           : uint32_t(tiles_of(s, rb0 + lane, p.gqa)) + kLead;
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += u;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, sum > rest);
    if (over != 0u || rb0 + 32 >= s.w) {
      const int w = over != 0u ? __ffs(over) - 1 : 31;
      c.rb = rb0 + w;
      const uint32_t before = __shfl_sync(0xffffffffu, sum - own, w);
      n = int(__shfl_sync(0xffffffffu, own, w)) - int(kLead);
      c.t = int(rest - before) - int(kLead);
      break;
    }
    rest -= __shfl_sync(0xffffffffu, sum, 31);
  }
  if (c.t <= kSnap) {
    c.t = 0;
  } else if (n - c.t <= kSnap) {
    c.t = 0;
    if (++c.rb == s.w) {
      c.rb = 0;
      if (++c.g == p.Hkv) {
        c.g = 0;
        do ++c.b; while (c.b < p.B && sm.at[c.b + 1] == sm.at[c.b]);   // (sequences without rows)
      }
    }
  }
  return c;
}

__device__ __forceinline__ bool before(const Cut& a, const Cut& b) {
  return a.b != b.b ? a.b < b.b : a.g != b.g ? a.g < b.g : a.rb != b.rb ? a.rb < b.rb : a.t < b.t;
}

// Two values to e4m3, and what they leave: h becomes h - e4m3(h), exactly.
__device__ __forceinline__ uint32_t take_half_term(__half2& h) {
  const uint32_t t = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&h), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw d = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(t), __NV_E4M3);
  h = __hsub2(h, __half2(d));
  return t;
}

// Eight e4m3 values to fp16.
__device__ __forceinline__ uint4 to_f16x8(uint2 u) {
  const uint32_t w[2] = {u.x, u.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n"
        "  .reg .b16 l, h;\n"
        "  mov.b32 {l, h}, %2;\n"
        "  cvt.rn.f16x2.e4m3x2 %0, l;\n"
        "  cvt.rn.f16x2.e4m3x2 %1, h;\n"
        "}\n"
        : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
        : "r"(w[i]));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// (in line: the warps that gave registers away hold fewer than a called function of this launch may use)
__device__ __forceinline__ bool hold(uint64_t* bar, uint32_t parity, uint64_t tmo, int* abort) {
  return ptx::mbar_wait(bar, parity, tmo, abort);
}

template <typename Sm>
__device__ __forceinline__ bool wait_rec(Sm& sm, uint32_t J, uint64_t tmo) {
  const uint32_t G = J / kGroup;
  return hold(&sm.rec_full[G % kGroups], (G / kGroups) & 1u, tmo, &sm.abort);
}

// The dims of 128 from `dim` on in which a hit key that this row sees has a NaN: NaN in the row's output
// (rare; called by the softmax warps, which hold more registers than a function of this launch may use).  part: its
// fp32 part, else out: its 16-bit output.
__device__ __noinline__ void put_back(const ChunkArgs& p, const uint32_t* hit, int b, int g, int pr_lo,
                                      int lim, int dim, float* part, uint16_t* out, uint16_t nan16) {
  for (int w = 0; w < kHitWords; ++w)
    for (uint32_t bits = hit[w]; bits != 0u; bits &= bits - 1u) {
      const int key = pr_lo + 32 * w + __ffs(bits) - 1;
      if (key >= lim) continue;
      const int blk = __ldg(p.tables + (long long)b * p.max_blocks + (key >> p.bs_log2));
      if (blk < 0 || blk >= p.num_blocks) continue;
      const size_t row = ((size_t(blk) * p.Hkv + g) << p.bs_log2) + (key & ((1 << p.bs_log2) - 1));
#pragma unroll 1
      for (int c = dim; c < dim + 128; ++c)
        if ((p.v_pool[row * 256 + c] & 0x7Fu) == 0x7Fu) {
          if (part != nullptr) part[c] = __int_as_float(0x7FC00000); else out[c] = nan16;
        }
    }
}

template <bool kF16>
__global__ void __launch_bounds__(kThreadsC, 1) kv8_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ ChunkArgs p) {
  extern __shared__ uint8_t smem_raw[];
  using Sm = ChunkSmem<kF16>;
  // (an offset, not a rounded pointer: the compiler then knows that it is shared memory; with generic accesses 2048
  // rows at 30720 took 640 us for 603, 8192 rows 608 for 583, each repeated on two inputs)
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((0u - ptx::smem_addr(smem_raw)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint64_t tmo = p.ctl.timeout_ns;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool lead = rank == 0;
  const int pair = int(blockIdx.x) >> 1;
  if (tid == 0) {
    for (int i = 0; i < kGroups; ++i) {
      ptx::mbar_init(&sm.rec_full[i], 1);
      ptx::mbar_init(&sm.rec_empty[i], 13);   // K's copies, 4 converting warps, 8 of softmax
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sm.k_full[i], 2);       // both CTAs' copying warps
      ptx::mbar_init(&sm.s_full[i], 1);
      ptx::mbar_init(&sm.p_full[i], 16 + 8);   // softmax and converting warps of both CTAs
      ptx::mbar_init(&sm.pv_done[i], 1);
    }
    ptx::mbar_init(&sm.q_full, 16);
    ptx::mbar_init(&sm.o_free, 16);
    ptx::mbar_init(&sm.drain, 1);
    for (int i = 0; i < kHitSets; ++i) ptx::mbar_init(&sm.hit_full[i], 8);
    sm.abort = 0;
    sm.zero = 0;
    sm.at[0] = 0;
    sm.segments = sm.longest = sm.whole = 0u;
    ptx::fence_mbar_init();
  }
  if (tid < kHitSets * kHitWords) (&sm.hit[0][0])[tid] = 0u;
  if (warp == 1) {
    ptx::tmem_alloc_pair(&sm.tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  wait_for_last();
  let_next_start();
  // ---- what each sequence costs
  for (int b = tid; b < p.B; b += kThreadsC) {
    const int kv = p.kv_lens[b], t0 = p.cu_rows[b], rows = p.cu_rows[b + 1] - t0;
    const bool ok = rows >= 0 && rows <= p.max_rows && t0 >= 0 && rows <= p.T - t0 && kv >= rows &&
                    kv <= p.max_kv_len;
    const int n_rb = ok ? int(((long long)rows * p.gqa + kPairRows - 1) / kPairRows) : 0;
    sm.seq[b] = make_int4(t0, rows, kv, n_rb);
    if (!ok && blockIdx.x == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
  }
  __syncthreads();
  for (int b = warp; b < p.B; b += kThreadsC / 32) {
    const int4 s = sm.seq[b];
    uint32_t sum = 0;
    for (int rb = lane; rb < s.w; rb += 32) sum += uint32_t(tiles_of(s, rb, p.gqa)) + kLead;
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) {
      sm.cost[b] = sum;
      if (s.w > 0) {
        atomicAdd(&sm.segments, uint32_t(s.w) * uint32_t(p.Hkv));
        atomicMax(&sm.longest, uint32_t(tiles_of(s, s.w - 1, p.gqa)));
      }
    }
  }
  __syncthreads();
  if (warp == 0) {   // inclusive sums over the sequences, 32 at a time; once more where no segment is cut
#pragma unroll 1
    for (;;) {
      uint32_t run = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        uint32_t v = b0 + lane < p.B ? sm.cost[b0 + lane] * uint32_t(p.Hkv) : 0u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        if (b0 + lane < p.B) sm.at[b0 + lane + 1] = run + v;
        run += __shfl_sync(0xffffffffu, v, 31);
      }
      const uint32_t pairs = uint32_t(p.pairs);
      if (sm.whole != 0u || sm.segments > pairs || sm.longest > (run - sm.segments * kLead) / pairs + kWhole)
        break;
      for (int b = lane; b < p.B; b += 32) sm.cost[b] = uint32_t(sm.seq[b].w);
      __syncwarp();
      if (lane == 0) sm.whole = 1u;
      __syncwarp();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers exist before any arrive reaches them
  ptx::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp < kConvWarp) {
    leave_regs<kRegsRest>();
    if (warp == 0) {
      // ---------------------------------------------------------- schedule
      const unsigned long long W = sm.at[p.B];
      const uint32_t n = uint32_t(min((unsigned long long)p.pairs, W));
      Cut at{p.B, 0, 0, 0}, end = at;
      if (uint32_t(pair) < n) {
        at = cut_at(sm, p, uint32_t(W * pair / n));
        end = cut_at(sm, p, uint32_t(W * (pair + 1) / n));
      }
      // cuts[0..1]: whether this pair's first piece goes on with a segment (1) and ends it (2); the
      // rest: the segment that its last piece starts and does not end
      int first_state = 0, starts = 0;
      ChunkPiece open{0, 0, 0, 0, 0, 0, -1};
      uint32_t J = 0, n_pieces = 0;
      bool ok = true, done = false;
      int4 s = make_int4(0, 0, 0, 0);
      int t = 0, t_end = 0, pr_lo = 0, k_hi = 0;
      bool in_piece = false;
      while (!done) {
        // this group's tiles: every lane goes through them, and keeps its own
        TileRec r;
        r.n_tiles = 0;
        r.key0 = r.k_hi = r.pr_lo = r.g = r.piece = r.last = 0;
        int my_b = 0;
        const uint32_t G = J / kGroup;
        if (G >= kGroups) {
          ok = warp_all(hold(&sm.rec_empty[G % kGroups], (G / kGroups - 1) & 1u, tmo, &sm.abort));
          if (!ok) break;
        }
        for (int q = 0; q < kGroup && !done; ++q) {
          if (!in_piece) {
            if (!before(at, end)) {
              done = true;
              break;
            }
            s = sm.seq[at.b];
            const int all = tiles_of(s, at.rb, p.gqa);
            const bool ends = at.b != end.b || at.g != end.g || at.rb != end.rb;
            t = at.t;
            t_end = ends ? all : end.t;
            const int rows_to = min(s.y, ((at.rb + 1) * kPairRows - 1) / p.gqa + 1);
            k_hi = s.z - s.y + rows_to;
            pr_lo = s.z - s.y + at.rb * kPairRows / p.gqa + 1;
            ChunkPiece x{at.b, at.g, at.rb, s.y, s.x, s.z - s.y, -1};
            if (t != 0) {
              x.part = 2 * pair;
              first_state = ends ? 2 : 1;
            } else if (!ends) {
              x.part = 2 * pair + 1;
              starts = 1;
              open = x;
            }
            if (lane == 0) sm.piece[n_pieces % kPieces] = x;
            // this CTA's rows of Q and of the gate are on their way to L2
            const int r0 = at.rb * kPairRows + 128 * int(rank), r1 = min(r0 + 128, s.y * p.gqa);
            for (int i = r0 + (lane >> 2); i < r1; i += 8) {
              const size_t row = size_t(s.x + i / p.gqa) * p.Hq + at.g * p.gqa + i % p.gqa;
              asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + row * 32 + (lane & 3) * 8));
              if (p.gate != nullptr && x.part < 0)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.gate + row * 256 + (lane & 3) * 64));
            }
            in_piece = true;
          }
          if ((lane >> 3) == q) {
            r.key0 = t * kTile;
            r.k_hi = k_hi;
            r.pr_lo = pr_lo;
            r.g = at.g;
            r.n_tiles = t_end - t;
            r.piece = int(n_pieces);
            r.last = t + 1 == t_end;
            my_b = at.b;
          }
          if (++t == t_end) {
            in_piece = false;
            ++n_pieces;
            at.t = 0;
            if (++at.rb == s.w) {
              at.rb = 0;
              if (++at.g == p.Hkv) {
                at.g = 0;
                do ++at.b; while (at.b < p.B && sm.seq[at.b].w == 0);
              }
            }
          }
        }
        // block and scales of run lane & 7 of this lane's tile
        TileRec& o = sm.rec[(J + (lane >> 3)) % kTiles];
        const int u = lane & 7, key = r.key0 + 16 * u;
        int blk = -1;
        float ks = 1.f, lv = 0.f;
        if (r.n_tiles > 0 && key < r.k_hi) {
          blk = __ldg(p.tables + (long long)my_b * p.max_blocks + (key >> p.bs_log2));
          if (blk >= 0 && blk < p.num_blocks) {
            ks = __ldg(p.k_scale + size_t(blk) * p.Hkv + r.g);
            lv = log2_scale(__ldg(p.v_scale + size_t(blk) * p.Hkv + r.g));
          } else {
            blk = -1;   // reads as zeros
            record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
          }
        }
        o.blk[u] = blk;
        o.ks[u] = ks;
        o.lv[u] = lv;
        float least = lv;
#pragma unroll
        for (int k = 1; k < 8; k <<= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, k));
        if (u == 0) {
          o.key0 = r.key0;
          o.k_hi = r.k_hi;
          o.pr_lo = r.pr_lo;
          o.g = r.g;
          o.n_tiles = r.n_tiles;
          o.piece = r.piece;
          o.last = r.last;
          o.lv_min = least;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sm.rec_full[G % kGroups]);
        J += kGroup;
        if (done) break;
        // (a group that the share's end fills exactly is followed by one that says so)
      }
      if (lane == 0 && lead && pair < p.pairs) {
        int* const c = p.cuts + 8 * pair;
        c[0] = first_state;
        c[1] = starts;
        c[2] = open.g;
        c[3] = open.rb;
        c[4] = open.rows;
        c[5] = open.t0;
      }
      if (!ok && lane == 0) {
        sm.abort = 1;
        record_status(p.ctl.status, GQA_ERR_TIMEOUT);
      }
    } else if (warp == 1 && lead) {
      // ---------------------------------------------------------- products
      // The whole warp goes through the loop, with what the products take in uniform registers (hence the shuffles);
      // one lane issues.
      const uint32_t go = lane == 0;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t base = __shfl_sync(0xffffffffu, ptx::smem_addr(&sm), 0);
      const uint64_t qd = ptx::sdesc_sw128(base + offsetof(Sm, q), 16, 1024);
      uint32_t J = 0, pc = 0;
      bool ok = true;
      const auto issue_s = [&](uint32_t n) -> bool {
        const uint32_t ks = n & 1u;
        if (!warp_all(hold(&sm.k_full[ks], (n >> 1) & 1u, tmo, &sm.abort))) return false;
        ptx::tc_fence_after();
        const uint64_t kd = ptx::sdesc_sw128(base + offsetof(Sm, k) + ks * kSlotK, 16, 1024);
        const uint32_t d = tm + kTmSc + ks * 128;
#pragma unroll
        for (int t = 0; t < Sm::kQTerms; ++t)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            ptx::mma_ss_pair_f8_if(go, d, ptx::sdesc_at(qd, t * 32768 + (kk >> 2) * 16384 + (kk & 3) * 32),
                                   ptx::sdesc_at(kd, (kk >> 2) * (kSlotK / 2) + (kk & 3) * 32), kIdescSc,
                                   t > 0 || kk > 0);
        if (go) ptx::tc_commit_pair(&sm.s_full[ks], 3);
        __syncwarp();
        return true;
      };
      const auto issue_pv = [&](uint32_t n, uint32_t accumulate) -> bool {
        const uint32_t vs = n & 1u;
        const uint64_t vd = ptx::sdesc_sw128(base + offsetof(Sm, v) + vs * kSlotV, kSlotV / 2, 1024);
        const uint32_t a = tm + kTmSc + vs * 128;
        if (!warp_all(hold(&sm.p_full[vs], (n >> 1) & 1u, tmo, &sm.abort))) return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_ts_pair_if(go, tm + kTmOc, a + (kk >> 2) * 64 + (kk & 3) * 8, ptx::sdesc_at(vd, kk * 2048), kIdescOc,
                              kk > 0 ? 1u : accumulate);
        if (go) ptx::tc_commit_pair(&sm.pv_done[vs], 3);
        __syncwarp();
        return true;
      };
      while (ok) {
        ok = warp_all(wait_rec(sm, J, tmo));
        if (!ok) break;
        const int n_tiles = __shfl_sync(0xffffffffu, sm.rec[J % kTiles].n_tiles, 0);
        if (n_tiles == 0) break;
        ok = warp_all(hold(&sm.q_full, pc & 1u, tmo, &sm.abort));
        if (!ok) break;
        ptx::tc_fence_after();
        ok = issue_s(J);
        if (ok && n_tiles > 1) ok = issue_s(J + 1);
        // O of the last piece has been read by every warp
        if (ok && pc > 0) ok = warp_all(hold(&sm.o_free, (pc - 1u) & 1u, tmo, &sm.abort));
        for (int j = 0; ok && j < n_tiles; ++j) {
          ok = issue_pv(J + j, j > 0);
          // S of tile j + 2 goes where P of tile j lies: products run in the order of issue
          if (ok && j + 2 < n_tiles) ok = issue_s(J + j + 2);
        }
        J += n_tiles;
        ++pc;
      }
      if (go) {
        if (!ok) {
          sm.abort = 1;
          record_status(p.ctl.status, GQA_ERR_TIMEOUT);
        }
        // every product issued has to end before tensor memory is given back
        ptx::tc_commit_pair(&sm.drain, 1);
        hold(&sm.drain, 0, tmo, &sm.zero);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- copies of K
      // This CTA's 64 keys of a tile, a box of up to 64 keys x 128 dims a lane; both CTAs' bytes count on the
      // even CTA's barrier.  Keys that are not there are not copied (their scores are not used).
      const int box_log2 = min(p.bs_log2, 6), boxes = 64 >> box_log2;
      uint32_t J = 0;
      bool ok = true;
      if (lane == 0) ptx::prefetch_tmap(&tmK);
      for (;; ++J) {
        ok = warp_all(wait_rec(sm, J, tmo));
        if (!ok) break;
        const TileRec& r = sm.rec[J % kTiles];
        if (r.n_tiles == 0) break;
        const uint32_t ks = J & 1u;
        if (J >= kKs) ok = warp_all(hold(&sm.s_full[ks], ((J >> 1) - 1u) & 1u, tmo, &sm.abort));
        if (!ok) break;
        const int left = r.k_hi - r.key0;
        if (!lead && lane == 0) ptx::mbar_arrive_remote(ptx::mapa_shared(ptx::smem_addr(&sm.k_full[ks]), 0));
        if (lead && lane == 0) {
          const int n0 = (min(max(left, 0), 64) + (1 << box_log2) - 1) >> box_log2;
          const int n1 = (min(max(left - 64, 0), 64) + (1 << box_log2) - 1) >> box_log2;
          ptx::mbar_arrive_expect_tx(&sm.k_full[ks], uint32_t(n0 + n1) << (box_log2 + 8));
        }
        __syncwarp();
        const int at = 64 * int(rank) + (lane << box_log2);   // first key of this lane's box
        if (lane < boxes && at < left) {
          const int blk = r.blk[at >> 4];
          // a block outside the pool: past the map's last row, which copies zeros
          const int row = blk >= 0 ? ((blk * p.Hkv + r.g) << p.bs_log2) + ((r.key0 + at) & ((1 << p.bs_log2) - 1))
                                   : (p.num_blocks * p.Hkv) << p.bs_log2;
          const uint32_t bar = ptx::mapa_shared(ptx::smem_addr(&sm.k_full[ks]), 0);
          uint8_t* const d = sm.k[ks] + (lane << (box_log2 + 7));
          ptx::tma_load_2d_pair(d, &tmK, bar, 0, row);
          ptx::tma_load_2d_pair(d + kSlotK / 2, &tmK, bar, 128, row);
        }
        __syncwarp();
        if (lane == 0 && J % kGroup == kGroup - 1) ptx::mbar_arrive(&sm.rec_empty[(J / kGroup) % kGroups]);
      }
      if (!ok && lane == 0) {
        sm.abort = 1;
        record_status(p.ctl.status, GQA_ERR_TIMEOUT);
      }
      // every copy of the pair has landed before it ends
      if (lead && lane == 0)
        for (uint32_t c = J - min(J, uint32_t(kKs)); c < J; ++c)
          hold(&sm.k_full[c % kKs], (c / kKs) & 1u, tmo, &sm.zero);
    }
    __syncwarp();
  } else if (warp < kSoftWarp) {
    // ------------------------------------------------------------ conversion
    leave_regs<kRegsConv>();
    const int w = warp - kConvWarp;
    const int bs_mask = (1 << p.bs_log2) - 1;
    const uint32_t peer_hit = ptx::mapa_shared(ptx::smem_addr(&sm.hit[0][0]), rank ^ 1u);
    bool ok = true;
    // The next tile's loads are on their way while the slot is waited for.  A warp has the 32 keys of two runs, four
    // keys a load; a thread has dims 8 c .. of both 64s (c = lane % 8), so that eight lanes' stores meet no bank
    // twice.
    const int sub = lane >> 3;          // key of a load
    const uint32_t off = (w * 32 + sub) * 128 + (((lane & 7) ^ sub) << 4);
    uint2 u[8][2];
    const auto load = [&](uint32_t J) -> bool {
      if (!warp_all(ok && wait_rec(sm, J, tmo))) {
        ok = false;
        return false;
      }
      const TileRec& r = sm.rec[J % kTiles];
      if (r.n_tiles == 0) return false;
      const int left = r.k_hi - r.key0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int run = 2 * w + h, blk = r.blk[run];
        const int n = blk >= 0 ? left - 16 * run : 0;          // its keys
        const uint8_t* const a =
            p.v_pool + 128 * rank + (lane & 7) * 8 + sub * 256 +
            (((size_t(max(blk, 0)) * p.Hkv + r.g) << p.bs_log2) + ((r.key0 + 16 * run) & bs_mask)) * 256;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u[4 * h + i][0] = u[4 * h + i][1] = make_uint2(0u, 0u);
          if (4 * i + sub < n) {
            u[4 * h + i][0] = __ldg(reinterpret_cast<const uint2*>(a + i * 1024));
            u[4 * h + i][1] = __ldg(reinterpret_cast<const uint2*>(a + i * 1024 + 64));
          }
        }
      }
      return true;
    };
    for (uint32_t J = 0; load(J); ++J) {
      const uint32_t vs = J & 1u;
      if (J >= kVs)
        ok = warp_all(ok && hold(&sm.pv_done[vs], ((J >> 1) - 1u) & 1u, tmo, &sm.abort));
      if (!ok) break;
      const TileRec& r = sm.rec[J % kTiles];
      if (r.key0 + kTile > r.pr_lo) {
        // rows that some rows of the segment do not see: their NaN are taken out, and noted in both CTAs
        const int key0 = r.key0 + 32 * w + sub, pr_lo = r.pr_lo, set = r.piece % kHitSets;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int key = key0 + 4 * s;
          uint4 x = make_uint4(u[s][0].x, u[s][0].y, u[s][1].x, u[s][1].y);
          if (key >= pr_lo && clear_nan8(x)) {
            const int h = key - pr_lo;
            atomicOr(&sm.hit[set][h >> 5], 1u << (h & 31));
            asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(
                             peer_hit + uint32_t(set * kHitWords + (h >> 5)) * 4u),
                         "r"(1u << (h & 31))
                         : "memory");
            u[s][0] = make_uint2(x.x, x.y);
            u[s][1] = make_uint2(x.z, x.w);
          }
        }
      }
      const uintptr_t slot = reinterpret_cast<uintptr_t>(sm.v[vs] + off);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        // row 4 s + sub of the warp's: its swizzle differs from row sub's in one bit
        const uintptr_t a = (slot ^ uintptr_t((s & 1) * 64)) + s * 512;
        *reinterpret_cast<uint4*>(a) = to_f16x8(u[s][0]);
        *reinterpret_cast<uint4*>(a + kSlotV / 2) = to_f16x8(u[s][1]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        arrive_lead(&sm.p_full[vs], lead);
        if (r.last) {
          uint64_t* const h = &sm.hit_full[r.piece % kHitSets];
          ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(h), 0));
          ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(h), 1));
        }
        if (J % kGroup == kGroup - 1) ptx::mbar_arrive(&sm.rec_empty[(J / kGroup) % kGroups]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      sm.abort = 1;
      record_status(p.ctl.status, GQA_ERR_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    take_regs<kRegsSoft>();
    const int sw = warp - kSoftWarp, half = sw >> 2, qd = warp & 3, row = qd * 32 + lane;
    const uint32_t trow = tmem + (uint32_t(qd * 32) << 16);
    const uint32_t bar_id = 1 + qd;   // the two warps of a quadrant
    uint32_t J = 0, pc = 0;
    bool ok = true;
    // Q's terms of piece n; then its products may start.  (The last piece's S products are done.)
    const auto prepare = [&](uint32_t n) {
      const ChunkPiece& x = sm.piece[n % kPieces];
      const int p0 = x.rb * kPairRows + int(rank) * 128, n_rows = min(128, x.rows * p.gqa - p0);
      // rows 16 sw .. of the CTA's 128: a lane finds the place of one, four rows' loads run ahead
      long long place = -1;
      {
        const int rr = sw * 16 + (lane & 15), i = (p0 + rr) / p.gqa;
        if (rr < n_rows) place = (long long)(x.t0 + i) * p.Hq + x.g * p.gqa + (p0 + rr - i * p.gqa);
      }
      const auto load4 = [&](int r, uint4 (&u)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const long long at = __shfl_sync(0xffffffffu, place, r + k);
          u[k] = at >= 0 ? __ldg(p.q + at * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      uint4 u[4], next[4];
      load4(0, u);
#pragma unroll 1
      for (int r = 0; r < 16; r += 4) {
        load4(min(r + 4, 12), next);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rr = sw * 16 + r + k;
          const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
          // the row's largest |x|: 16-bit patterns without the sign are in order
          uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
          m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
          const int e = scale_exp(__float_as_uint(elem_to_float<kF16>(m)));
          if (lane == 0) sm.fac[n & 1u][rr] = pow2f(e) * kScaleLog2;
          // a NaN or an infinity makes the row's scores NaN, as it does in the formula
          const float inv = m >= (kF16 ? 0x7C00u : 0x7F80u) ? __int_as_float(0x7FC00000) : inv_pow2f(e);
          __half2 h[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float2 x = mul2(unpack_elem2<kF16>(w[c]), make_float2(inv, inv));
            h[c] = __floats2half2_rn(x.x, x.y);
          }
          uint8_t* const to = sm.q[0][lane >> 4] + rr * 128 +
                              ((((lane & 15) >> 1) ^ (rr & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
          for (int t = 0; t < Sm::kQTerms; ++t) {
            uint32_t o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = take_half_term(h[c]);
            *reinterpret_cast<uint2*>(to + t * 2 * 128 * 128) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = next[k];
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(&sm.q_full, lead);
    };

    ok = warp_all(wait_rec(sm, 0, tmo));
    bool more = ok && sm.rec[0].n_tiles > 0;
    if (more) prepare(0);
    // All softmax warps meet here once before the first piece and once in each: one that gives up
    // comes once more on its way out, and the others leave with it.
    bool stop = ptx::named_bar_or(9, 256, !ok);
    while (more && !stop) {
      const int n_tiles = sm.rec[J % kTiles].n_tiles;
      int lim = 0;   // keys that this thread's row sees; 0: there is no such row
      {
        const ChunkPiece& x = sm.piece[pc % kPieces];
        const int pk = x.rb * kPairRows + int(rank) * 128 + row;
        if (pk < x.rows * p.gqa) lim = x.base + pk / p.gqa + 1;
      }
      const float fac = sm.fac[pc & 1u][row];
      const float top = n_tiles > kLongPiece ? kLongTop : 0.f;
      float ref = kNone, ml = kNone, l = 0.f;
      for (int j = 0; j < n_tiles; ++j, ++J) {
        const uint32_t buf = J & 1u;
        ok = ok && wait_rec(sm, J, tmo) && hold(&sm.s_full[buf], (J >> 1) & 1u, tmo, &sm.abort);
        ok = warp_all(ok);
        __syncwarp();
        ptx::tc_fence_after();
        const TileRec& r = sm.rec[J % kTiles];
        const uint32_t ts = trow + kTmSc + buf * 128 + half * 64;
        const int left = lim - r.key0 - half * 64;   // of this thread's keys, those that the row sees
        // Loops over 32 keys, not unrolled: the roles' code shares the schedulers' instruction caches.
        // A run's score factor is finite and not 0, so that a hidden key's -inf stays one and 0 stays 0.
        const auto factors = [&](int q) -> float2 {
          const float2 k2 = *reinterpret_cast<const float2*>(&r.ks[4 * half + 2 * q]);
          return make_float2(fminf(fmaxf(fac * k2.x, 1e-37f), 3e38f), fminf(fmaxf(fac * k2.y, 1e-37f), 3e38f));
        };
        if (ok && __any_sync(0xffffffffu, left < 64)) {   // keys that some row does not see: -inf
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t s[32];
            ptx::tmem_ld32_wait(ts + 32 * q, s);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * q + c >= left) s[c] = 0xFF800000u;
            ptx::tmem_st32_wait(ts + 32 * q, s);
          }
        }
        // f(q, scores) for each 32 keys
        const auto each = [&](auto&& f) {
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t s[32];
            ptx::tmem_ld32_wait(ts + 32 * q, s);
            f(q, s);
          }
        };
        float mp = -INFINITY, ms = -INFINITY;
        if (ok) each([&](int q, uint32_t (&s)[32]) {
          const float2 f2 = factors(q), lv2 = *reinterpret_cast<const float2*>(&r.lv[4 * half + 2 * q]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = fmaxf(__uint_as_float(s[16 * i]), __uint_as_float(s[16 * i + 1]));
            float n = fmaxf(__uint_as_float(s[16 * i + 2]), __uint_as_float(s[16 * i + 3]));
#pragma unroll
            for (int c = 4; c < 16; c += 4) {
              m = fmaxf(fmaxf(m, __uint_as_float(s[16 * i + c])), __uint_as_float(s[16 * i + c + 1]));
              n = fmaxf(fmaxf(n, __uint_as_float(s[16 * i + c + 2])), __uint_as_float(s[16 * i + c + 3]));
            }
            m = fmaxf(m, n) * (i ? f2.y : f2.x);
            ms = fmaxf(ms, m);
            mp = fmaxf(mp, m + (i ? lv2.y : lv2.x));
          }
        });
        // (a maximum is never NaN: that says that the warp gives up)
        sm.red[buf][half][row] = make_float2(ok ? mp : __int_as_float(0x7FC00000), ms);
        ptx::named_bar_sync(bar_id, 64);
        {
          const float2 o = sm.red[buf][half ^ 1][row];
          ok = ok && o.x == o.x;
          mp = fmaxf(mp, o.x);
          ms = fmaxf(ms, o.y);
        }
        if (!warp_all(ok)) {
          ok = false;
          break;
        }
        // ---- references (both threads of a row do the same).  Where one row's has to move, O is scaled anyway, and those
        // of the warp's others go along.
        const float at = ref;
        const bool moved = __any_sync(0xffffffffu, mp > at + kCap);
        if (moved) ref = fmaxf(at, mp - top);
        if (ms > ml + kLSlack) {
          l *= ex2(ml - ms);
          ml = ms;
        }
        // ---- P goes where the scores were
        // l's terms come from p's: p * 2^(ref - log2 vs - ml), unless p may have lost them
        const float back = ref - ml;
        const bool far = __any_sync(0xffffffffu, back - r.lv_min > 60.f);
        if (far) {
          each([&](int q, uint32_t (&s)[32]) {
            const float2 f2 = factors(q);
#pragma unroll
            for (int c = 0; c < 32; ++c) l += ex2(fmaf(__uint_as_float(s[c]), c < 16 ? f2.x : f2.y, -ml));
          });
        }
        each([&](int q, uint32_t (&s)[32]) {
          const float2 f2 = factors(q), lv2 = *reinterpret_cast<const float2*>(&r.lv[4 * half + 2 * q]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float fi = i ? f2.y : f2.x, lv = i ? lv2.y : lv2.x, a = lv - ref;
            const float2 ff = make_float2(fi, fi), aa = make_float2(a, a);
            uint32_t pk[8];
            float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float2 y = fma2(make_float2(__uint_as_float(s[16 * i + 2 * c]),
                                                __uint_as_float(s[16 * i + 2 * c + 1])), ff, aa);
              const float2 e = make_float2(ex2(y.x), ex2(y.y));
              sum2 = add2(sum2, e);
              pk[c] = pack_half2(e.x, e.y);
            }
            ptx::tmem_st8(ts + 16 * q + 8 * i, pk);
            if (!far) l += (sum2.x + sum2.y) * ex2(back - lv);
          }
        });
        ptx::tmem_wait_st();
        if (moved && j > 0) {
          // O, with PV of tile J - 1 in it, moves to the new references.  (A warp that gives up here says so at the
          // next tile's barrier, or at the piece's end.)
          ok = warp_all(hold(&sm.pv_done[buf ^ 1u], ((J - 1u) >> 1) & 1u, tmo, &sm.abort));
          if (ok) {
            ptx::tc_fence_after();
            const float alpha = ex2(at - ref);
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
              const uint32_t to = trow + kTmOc + half * 128 + 32 * cc;
              uint32_t o[32];
              ptx::tmem_ld32_wait(to, o);
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              ptx::tmem_st32_wait(to, o);
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) arrive_lead(&sm.p_full[buf], lead);
        if (lane == 0 && J % kGroup == kGroup - 1)
          ptx::mbar_arrive(&sm.rec_empty[(J / kGroup) % kGroups]);
      }
      if (!ok) {
        sm.abort = 1;
        ptx::named_bar_or(9, 256, true);
        stop = true;
        break;
      }
      // ---- the next piece may start while this one ends
      ok = warp_all(ok && wait_rec(sm, J, tmo));
      more = ok && sm.rec[J % kTiles].n_tiles > 0;
      if (more) prepare(pc + 1u);
      sm.sum[half][row] = l;
      const ChunkPiece& x = sm.piece[pc % kPieces];
      const bool mine = lim > 0;
      const int i_new = lim - 1 - x.base, pk = x.rb * kPairRows + int(rank) * 128 + row;
      const size_t at = size_t(x.t0 + i_new) * p.Hq + x.g * p.gqa + (pk - i_new * p.gqa);
      const bool gated = p.gate != nullptr && mine && x.part < 0;
      const auto gate32 = [&](int cc, uint4 (&g4)[4]) {   // 32 of this thread's 128 columns
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (gated) g4[c] = __ldg(reinterpret_cast<const uint4*>(p.gate + at * 256 + half * 128) + 4 * cc + c);
      };
      uint4 g4[4], g_next[4];
      gate32(0, g4);
      ok = warp_all(ok && hold(&sm.hit_full[pc % kHitSets], (pc / kHitSets) & 1u, tmo, &sm.abort) &&
                    hold(&sm.pv_done[(J - 1u) & 1u], ((J - 1u) >> 1) & 1u, tmo, &sm.abort));
      stop = ptx::named_bar_or(9, 256, !ok);
      if (stop) break;
      ptx::tc_fence_after();
      const float L = l + sm.sum[half ^ 1][row];
      const float ex = ex2(0.5f * (ref - ml)), inv = L == 0.f ? 0.f : ex / L;   // (O times both)
      const float lse = L == 0.f ? -INFINITY : (ml + __log2f(L)) * kLn2;
      const int set = pc % kHitSets;
      // every warp is past the last piece, whose hits may go
      if (half == 0 && row < kHitWords) sm.hit[(pc + kHitSets - 1) % kHitSets][row] = 0u;
      uint32_t any = 0u;
#pragma unroll
      for (int w = 0; w < kHitWords; ++w) any |= *reinterpret_cast<volatile uint32_t*>(&sm.hit[set][w]);
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int col = half * 128 + 32 * cc;
        __syncwarp();
        uint32_t o[32];
        ptx::tmem_ld32_wait(trow + kTmOc + col, o);
        if (!mine) continue;
        gate32(min(cc + 1, 3), g_next);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 y = mul2(mul2(make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1])),
                                     make_float2(inv, inv)), make_float2(ex, ex));
          o[c] = __float_as_uint(L == 0.f ? 0.f : y.x);
          o[c + 1] = __float_as_uint(L == 0.f ? 0.f : y.y);
        }
        if (x.part >= 0) {
          float4* const d = reinterpret_cast<float4*>(
              p.o_parts + (size_t(x.part) * kPairRows + int(rank) * 128 + row) * 256 + col);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            d[c] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                               __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
        } else {
          uint4* const d = reinterpret_cast<uint4*>(p.out + at * 256 + col);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
            const uint32_t gw[4] = {g4[c].x, g4[c].y, g4[c].z, g4[c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 y = make_float2(__uint_as_float(o[8 * c + 2 * e]), __uint_as_float(o[8 * c + 2 * e + 1]));
              if (p.gate != nullptr) {
                const float2 gf = unpack_elem2<kF16>(gw[e]);
                y = mul2(y, gate_sigmoid2(gf.x, gf.y));
              }
              w[e] = pack_elem2<kF16>(y.x, y.y);
            }
            d[c] = make_uint4(w[0], w[1], w[2], w[3]);
            g4[c] = g_next[c];
          }
        }
      }
      if (any != 0u && mine && L != 0.f)
        put_back(p, sm.hit[set], x.b, x.g, x.base + x.rb * kPairRows / p.gqa + 1, lim, half * 128,
                 x.part < 0 ? nullptr : p.o_parts + (size_t(x.part) * kPairRows + int(rank) * 128 + row) * 256,
                 p.out + at * 256, kF16 ? 0x7E00u : 0x7FC0u);
      if (mine && half == 0) {
        if (x.part >= 0)
          p.lse_parts[size_t(x.part) * kPairRows + int(rank) * 128 + row] = lse;
        else if (p.lse != nullptr)
          p.lse[at] = lse;
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(&sm.o_free, lead);
      ++pc;
    }
    if (stop && lane == 0) {
      sm.abort = 1;
      record_status(p.ctl.status, GQA_ERR_TIMEOUT);
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other may still reach its shared or tensor memory
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
}

// Puts the parts of the segments that were cut together, gates and rounds them: a warp a row.
//   out = (sum_i w_i O_i) / (sum_i w_i) * sigmoid(g),  w_i = exp(lse_i - max lse)
// One wave of CTAs that read what is cut where, and go through the rows of those segments alone (eight rows a CTA, as
// many CTAs as all pairs may leave rows: 42 rows behind 4000 keys 47 us for 35, 1000 new ones 66 for 52; most of those CTAs
// found nothing to do, 16 to an SM).
constexpr int kMaxPairs = 96;
constexpr int kJoinCtas = 3;    // of an SM
constexpr int kAhead = 4;       // parts whose values are on their way together

template <bool kF16>
__global__ void __launch_bounds__(256, kJoinCtas) kv8_join_kernel(const ChunkArgs p) {
  __shared__ float s_w[8][kMaxPairs];
  __shared__ int4 s_cut[2 * kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  let_next_start();
  wait_for_last();
  if (threadIdx.x < 2 * kMaxPairs)
    s_cut[threadIdx.x] = int(threadIdx.x) < 2 * p.pairs
                             ? __ldcg(reinterpret_cast<const int4*>(p.cuts) + threadIdx.x) : make_int4(0, 0, 0, 0);
  __syncthreads();
  // parts: a pair's last piece and the first ones of the pairs behind it, up to the one that ends
  uint32_t starts[kMaxPairs / 32], off[kMaxPairs / 32], ends[kMaxPairs / 32];
#pragma unroll
  for (int k = 0; k < kMaxPairs / 32; ++k) {
    const int4 c = s_cut[2 * (32 * k + lane)];
    starts[k] = __ballot_sync(0xffffffffu, c.y != 0);
    off[k] = __ballot_sync(0xffffffffu, c.x != 1);
    ends[k] = __ballot_sync(0xffffffffu, c.x == 2);
  }
#pragma unroll 1
  for (int R = int(blockIdx.x) * 8 + warp;; R += int(gridDim.x) * 8) {
    int left = R / kPairRows, pair = -1;
    const int r = R % kPairRows;
#pragma unroll
    for (int k = 0; k < kMaxPairs / 32; ++k) {
      const uint32_t hit = __ballot_sync(0xffffffffu, ((starts[k] >> lane) & 1u) != 0u &&
                                                          __popc(starts[k] & ((1u << lane) - 1u)) == left);
      if (hit != 0u) pair = 32 * k + __ffs(hit) - 1;
      left -= __popc(starts[k]);
    }
    if (pair < 0) return;
    const int4 c0 = s_cut[2 * pair], c1 = s_cut[2 * pair + 1];
    const int g = c0.z, rb = c0.w, rows = c1.x, t0 = c1.y;
    const int p0 = rb * kPairRows, n_rows = min(kPairRows, rows * p.gqa - p0);
    if (r >= n_rows) continue;
    int stop = kMaxPairs, last = 0;
#pragma unroll
    for (int k = kMaxPairs / 32 - 1; k >= 0; --k) {
      const int from = pair + 1 - 32 * k;
      const uint32_t m = from >= 32 ? 0u : off[k] & (0xffffffffu << max(from, 0));
      if (m != 0u) {
        stop = 32 * k + __ffs(m) - 1;
        last = int((ends[k] >> (__ffs(m) - 1)) & 1u);
      }
    }
    const int cnt = stop - pair + last;
    const auto slot = [&](int i) { return size_t(i == 0 ? 2 * pair + 1 : 2 * (pair + i)) * kPairRows + r; };
    float4 v[kAhead][2];
    const auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k < cnt) {
          const float4* const o = reinterpret_cast<const float4*>(p.o_parts + slot(i0 + k) * 256) + lane * 2;
          v[k][0] = __ldcg(o);
          v[k][1] = __ldcg(o + 1);
        }
    };
    load(0);
    const int pk = p0 + r, i = pk / p.gqa;
    const size_t at = size_t(t0 + i) * p.Hq + g * p.gqa + (pk - i * p.gqa);
    uint4 gate = make_uint4(0u, 0u, 0u, 0u);
    if (p.gate != nullptr) gate = __ldg(reinterpret_cast<const uint4*>(p.gate + at * 256) + lane);
    float ls[kMaxPairs / 32], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMaxPairs / 32; ++k) {
      ls[k] = 32 * k + lane < cnt ? __ldcg(p.lse_parts + slot(32 * k + lane)) : -INFINITY;
      M = fmaxf(M, ls[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float msub = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxPairs / 32; ++k) {
      const float w = ls[k] == -INFINITY ? 0.f : __expf(ls[k] - msub);
      s_w[warp][32 * k + lane] = ls[k] == -INFINITY ? -1.f : w;   // -1: the part saw no key
      sum += w;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < cnt; i0 += kAhead) {
      if (i0 > 0) load(i0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float w = i0 + k < cnt ? s_w[warp][i0 + k] : -1.f;
        if (w < 0.f) continue;   // (a weight of 0 counts: its part may hold a NaN that the row sees)
        acc[0] += w * v[k][0].x;
        acc[1] += w * v[k][0].y;
        acc[2] += w * v[k][0].z;
        acc[3] += w * v[k][0].w;
        acc[4] += w * v[k][1].x;
        acc[5] += w * v[k][1].y;
        acc[6] += w * v[k][1].z;
        acc[7] += w * v[k][1].w;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const uint32_t gw[4] = {gate.x, gate.y, gate.z, gate.w};
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 y = make_float2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      if (p.gate != nullptr) {
        const float2 a = unpack_elem2<kF16>(gw[k]);
        y = make_float2(y.x * gate_sigmoid(a.x), y.y * gate_sigmoid(a.y));
      }
      w[k] = pack_elem2<kF16>(y.x, y.y);
    }
    reinterpret_cast<uint4*>(p.out + at * 256)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if (p.lse != nullptr && lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : msub + __logf(sum);
    __syncwarp();   // before the next row's weights
  }
}

int pair_count() {
  const int n = device_sm_count() / 2;
  return n < 1 ? 1 : n < kMaxPairs ? n : kMaxPairs;
}

struct Workspace {
  size_t lse, cuts, bytes;   // o_parts lie first
};
Workspace workspace_of(int pairs) {
  Workspace w;
  const size_t rows = size_t(2) * pairs * kPairRows;
  w.lse = rows * 256 * sizeof(float);
  w.cuts = w.lse + rows * sizeof(float);
  w.bytes = w.cuts + size_t(8) * pairs * sizeof(int);
  return w;
}

template <bool kF16>
cudaError_t launch_chunk(const CUtensorMap& tmK, const ChunkArgs& a, bool join, cudaStream_t stream) {
  const size_t smem = sizeof(ChunkSmem<kF16>) + 1024;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem_once(allowed, reinterpret_cast<const void*>(kv8_chunk_kernel<kF16>), smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv8_chunk_kernel<kF16>, dim3(unsigned(2 * a.pairs)), kThreadsC, smem, stream, 2, tmK, a);
  if (e != cudaSuccess) return e;
  note_launch(kF16 ? "kv8_chunk_kernel<fp16>" : "kv8_chunk_kernel<bf16>", 2 * a.pairs, kThreadsC, smem);
  if (!join) return cudaSuccess;
  const unsigned grid = unsigned(device_sm_count() * kJoinCtas);
  e = launch_dependent(kv8_join_kernel<kF16>, dim3(grid), 256, 0, stream, 1, a);
  if (e == cudaSuccess)
    note_launch(kF16 ? "kv8_join_kernel<fp16>" : "kv8_join_kernel<bf16>", grid, 256, 0);
  return e;
}

// K's pool by rows: boxes of 128 dims x a block's rows, 64 at most.
bool encode_k(CUtensorMap* map, const ChunkArgs& a) {
  EncodeTiledFn fn = get_encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {256, cuuint64_t(a.num_blocks) * cuuint64_t(a.Hkv) << a.bs_log2};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {128, cuuint32_t(1) << (a.bs_log2 < 6 ? a.bs_log2 : 6)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.k_pool), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int prefill_impl(bool f16, const void* Q, const void* k_pool, const void* v_pool, const float* k_scale,
                 const float* v_scale, const void* G, const int* block_tables, const int* kv_lens,
                 const int* cu_rows, void* out, float* lse_out, int B, int T, int Hq, int Hkv,
                 int num_blocks, int block_size, int max_blocks, int max_rows, int max_kv_len,
                 void* workspace, size_t workspace_bytes, gqa_stream_t stream) {
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_rows < 1 || max_kv_len < 1 ||
      max_rows > max_kv_len)
    return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, Hkv, block_size);
  if (st != GQA_OK) return st;
  if (max_blocks < 1 || max_kv_len > (long long)max_blocks * block_size) return GQA_ERR_INVALID_ARG;
  if ((long long)T * Hq >= (1LL << 31) || (long long)max_rows * Hq >= (1LL << 31) - kPairRows ||
      max_kv_len >= (1 << 30))
    return GQA_ERR_UNSUPPORTED;
  if (T == 0) return GQA_OK;
  if (Q == nullptr || k_pool == nullptr || v_pool == nullptr || k_scale == nullptr ||
      v_scale == nullptr || block_tables == nullptr || kv_lens == nullptr || cu_rows == nullptr ||
      out == nullptr)
    return GQA_ERR_INVALID_ARG;
  for (const void* q : {Q, k_pool, v_pool, G, (const void*)out})
    if (!aligned_to(q, 16)) return GQA_ERR_INVALID_ARG;
  for (const void* q : {(const void*)k_scale, (const void*)v_scale, (const void*)block_tables,
                        (const void*)kv_lens, (const void*)cu_rows, (const void*)lse_out})
    if (!aligned_to(q, 4)) return GQA_ERR_INVALID_ARG;
  // the kernel counts a launch's positions (a segment's tiles and a few more) in 31 bits
  const int gqa = Hq / Hkv;
  const long long max_rb = ((long long)max_rows * gqa + kPairRows - 1) / kPairRows;
  const long long tiles = (max_kv_len + kTile - 1LL) / kTile;
  const long long per_seq = (long long)Hkv * max_rb * (tiles + kLead);
  if (Hkv * max_rb >= (1LL << 31) || per_seq >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  const int most = pair_count();
  const Workspace ws = workspace_of(most);
  if (workspace == nullptr || workspace_bytes < ws.bytes) return GQA_ERR_WORKSPACE;
  if (!aligned_to(workspace, 16)) return GQA_ERR_INVALID_ARG;
  ChunkArgs a{};
  a.q = static_cast<const uint4*>(Q);
  a.k_pool = static_cast<const uint8_t*>(k_pool);
  a.v_pool = static_cast<const uint8_t*>(v_pool);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.gate = static_cast<const uint16_t*>(G);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse_out;
  a.o_parts = static_cast<float*>(workspace);
  a.lse_parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + ws.lse);
  a.cuts = reinterpret_cast<int*>(static_cast<char*>(workspace) + ws.cuts);
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.gqa = gqa;
  a.num_blocks = num_blocks;
  while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
  a.max_blocks = max_blocks;
  a.max_rows = max_rows;
  a.max_kv_len = max_kv_len;
  if (!make_launch_ctl(&a.ctl)) return GQA_ERR_CUDA;
  CUtensorMap tmK;
  if (!encode_k(&tmK, a)) return GQA_ERR_UNSUPPORTED;
  const long long fit = ((1LL << 31) - 1) / per_seq;
  const int step = fit < kKv8Seqs ? int(fit) : kKv8Seqs;
  for (int b0 = 0; b0 < B; b0 += step) {
    a.B = B - b0 < step ? B - b0 : step;
    a.tables = block_tables + (long long)b0 * max_blocks;
    a.kv_lens = kv_lens + b0;
    a.cu_rows = cu_rows + b0;
    const long long units = (long long)a.B * Hkv * max_rb * tiles;
    a.pairs = units < most ? int(units) : most;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // a cut lies more than kSnap tiles from either end of a segment: in shorter ones there is none; and none in
    // any where the kernel leaves them whole
    const bool join = tiles > 2 * kSnap + 1 && (tiles > int(kWhole) || (long long)a.B * Hkv * max_rb > a.pairs);
    if ((f16 ? launch_chunk<true>(tmK, a, join, s) : launch_chunk<false>(tmK, a, join, s)) != cudaSuccess)
      return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_kv8_prefill_workspace_size(void) { return workspace_of(pair_count()).bytes; }

int gqa_kv8_prefill(const void* Q, const void* k_pool, const void* v_pool, const float* k_scale,
                    const float* v_scale, const void* G, const int* block_tables, const int* kv_lens,
                    const int* cu_rows, void* out, float* lse_out, int B, int T, int Hq, int Hkv,
                    int num_blocks, int block_size, int max_blocks, int max_rows, int max_kv_len,
                    void* workspace, size_t workspace_bytes, gqa_stream_t stream) {
  return prefill_impl(false, Q, k_pool, v_pool, k_scale, v_scale, G, block_tables, kv_lens, cu_rows, out,
                      lse_out, B, T, Hq, Hkv, num_blocks, block_size, max_blocks, max_rows, max_kv_len,
                      workspace, workspace_bytes, stream);
}
int gqa_kv8_prefill_f16(const void* Q, const void* k_pool, const void* v_pool, const float* k_scale,
                        const float* v_scale, const void* G, const int* block_tables,
                        const int* kv_lens, const int* cu_rows, void* out, float* lse_out, int B, int T,
                        int Hq, int Hkv, int num_blocks, int block_size, int max_blocks, int max_rows,
                        int max_kv_len, void* workspace, size_t workspace_bytes, gqa_stream_t stream) {
  return prefill_impl(true, Q, k_pool, v_pool, k_scale, v_scale, G, block_tables, kv_lens, cu_rows, out,
                      lse_out, B, T, Hq, Hkv, num_blocks, block_size, max_blocks, max_rows, max_kv_len,
                      workspace, workspace_bytes, stream);
}

}  // extern "C"
