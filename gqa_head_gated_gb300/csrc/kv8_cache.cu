// Writing the paged 8-bit KV cache: kv8_append quantises new rows behind the keys that
// their blocks hold; kv8_keep moves the accepted draft rows of a sequence to the front
// of its draft region.
//
// The rule, per (block, KV head), K and V apart, for the run of rows written to a block:
//   a    = largest finite |x| of the run, E(a) = least e >= -126 with a <= 448 * 2^e
//   e    = E(a) when the run starts at the block's first row, else max(e_old, E(a))
//   rows before the run are rounded again by 2^(e_old - e) where the scale grew
//   q    = e4m3(x * 2^-e), nearest even; NaN and +-Inf are stored as NaN (e4m3 has no
//          infinity, and a saturated one would pass for a number)
// Several runs of a call in one block follow one another in order.
// keep is the same rule applied to the kept rows' values, as if they had been appended
// behind the first len - r keys.
//
// An append of a prompt should be bound by HBM (2 bytes read and 1 written a value) and is by
// issue slots and latency: 100 instructions a row of 256 values and warp, of which the conversions
// are a third, at 55 % of the slots.  8192 rows of 4 heads, K and V: 12.0 us for 50 MB (62 % of the
// copy rate; floor 7.4), 12 chunks of 2731 rows of 2 heads 23.7 for 101 MB (63 %; 20.5 when the
// ends of a sequence did not look for other rows of their block).  With 4 CTAs
// of 256 threads an SM each warp holds 8 rows between the maximum and the rounding; 5 and 6 CTAs
// spill (16.3, 19.0 us where 4 took 13.0), 512 threads with 4 rows a warp took 14.0.  A step's call, 16 rows, is
// bound by latency: 3.6 us on the GPU (a chain of reads: slot, scale, row, and a launch).
// keep of 128 sequences' drafts takes 7.1 us on the GPU for 8.4 MB, again such a chain: list,
// table, rows, and the block's rows once more where a scale grew.
#include <cuda_runtime.h>

#include "kv8_common.cuh"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 64;               // tokens whose runs a CTA writes
constexpr int kSpan = kWindow + 128;      // the last of them may reach a block further
constexpr int kRowsPerWarp = kWindow / kWarps;

// 16-bit magnitudes order as integers: the largest two of a lane's 8 elements, side by side.
__device__ __forceinline__ uint32_t lane_amax(uint4 u) {
  return __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                  __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
}

// The larger of the two over the warp.
__device__ __forceinline__ uint32_t warp_amax(uint32_t m) {
  return __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
}

// Largest |x| of a row, NaN and infinities left out.
template <bool kF16>
__device__ __forceinline__ uint32_t finite_row_amax(uint4 u) {
  constexpr uint32_t kInf = kF16 ? 0x7C00u : 0x7F80u;
  const uint32_t w[4] = {u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu, u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu};
  uint32_t m = 0u;
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0xFFFFu, b = w[i] >> 16;
    m = max(m, max(a < kInf ? a : 0u, b < kInf ? b : 0u));
  }
  return __reduce_max_sync(0xffffffffu, m);
}

template <bool kF16>
__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack_elem2<kF16>(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

struct AppendParams {
  const uint4* x[2];        // K, V new rows: 16-bit [T, Hkv, 256]
  uint2* pool[2];           // e4m3 [num_blocks, Hkv, bs, 256]
  float* scale[2];          // [num_blocks, Hkv]
  const int* slots;
  int T, Hkv, num_blocks, bs_log2;
  LaunchCtl ctl;
};

// Rounds a block's first n rows again, from scale `s_old` to 1 / inv (one warp a row).
__device__ __forceinline__ void rescale_rows(uint2* block, int n, float s_old, float inv) {
  for (int r = threadIdx.x >> 5; r < n; r += kWarps) {
    uint2* const a = block + r * 32 + (threadIdx.x & 31);
    float f[8];
    from_e4m3x8(*a, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * s_old * inv;
    *a = to_e4m3x8(f);
  }
}

// A call may have several runs in one block: rows that are skipped in the middle of a sequence,
// sequences whose tokens alternate.  Each rounds the rows before it again, so that they go one
// after another: the CTA that has the block's first run takes all of them, the others leave
// theirs to it.  A run that starts at the block's first row has none before it, one that ends at
// its last row none behind it (rows of a block increase with the token), so that a prompt's
// windows look at the call's other tokens only at the ends of a sequence.
constexpr int kHash = kThreads;           // lists of a window's runs by block
constexpr int kContinues = 1;             // there is an earlier run in the block: left to its CTA
constexpr int kFollowed = 2;              // a later token of the call is in the block
constexpr int kRepeats = 4;               // an earlier token has this row or one behind it: no place

constexpr int kFew = 2;                   // runs that are asked for one by one
constexpr int kAhead = 8, kAsk = 16;      // tokens whose slots a thread loads together

struct Ask {
  int lo, hi;                // tokens
  unsigned slot;             // first of the block
};

struct WindowRuns {
  int head[kHash];           // first run of the list, -1: none
  int next[kWindow];
  int end[kWindow];          // by run (its first token): the token behind its last
  int state[kWindow];
  uint32_t followed[kWindow / 32];   // runs whose blocks' later ones are taken here
  int found, len;                    // of such a block
  int n_asks;
  Ask ask[2 * kFew];
};

// All threads: is any token in one of the few ranges in the block asked for?  A load and one
// instruction a token, where look_around() takes about ten: 12 prompt chunks of 2731 rows, whose
// 24 ends each go through 32,772 slots, 23.7 us so and 28.7 by look_around() alone; 8 loads
// together 24.8, 24 (spills) 27.1.  (256 sequences of 128 rows 66.7, and 50.3 when nobody looked; 128
// of 32 rows, by look_around(), 17.5 and 13.4.  With the CTAs of a window as a cluster that shares
// its tokens, the same three: 23.9, 72.9, 17.5, and a prompt of 8192 rows 12.3 for 12.0.)
__device__ __noinline__ bool any_in_block(const int* slots, unsigned bs, const WindowRuns& w) {
  unsigned m = ~0u;
  const int n = min(w.n_asks, 2 * kFew);
  for (int a = 0; a < n; ++a) {
    const Ask q = w.ask[a];
    for (int t = q.lo + int(threadIdx.x); t < q.hi; t += kAsk * kThreads) {
      unsigned s[kAsk];
#pragma unroll
      for (int k = 0; k < kAsk; ++k)
        s[k] = t + k * kThreads < q.hi ? unsigned(__ldg(slots + t + k * kThreads)) : ~0u;
#pragma unroll
      for (int k = 0; k < kAsk; ++k) m = __viaddmin_u32(s[k], 0u - q.slot, m);
    }
  }
  return __syncthreads_or(m < bs);
}

// All threads: sets kContinues, kFollowed and kRepeats, from every token of the call, for the runs
// of this window (`mine`: one starts at token w0 + tid) that may have others in their block.
__device__ __noinline__ void look_around(const int* slots, int T, int w0, unsigned n_slots,
                                         int bs_log2, const int* s_slot, bool mine, WindowRuns& w) {
  const int tid = threadIdx.x;
  if (mine) w.next[tid] = atomicExch(&w.head[(s_slot[tid + 1] >> bs_log2) % kHash], tid);
  __syncthreads();
  for (int t0 = tid; t0 < T; t0 += kAhead * kThreads) {
    int slot[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      slot[k] = t0 + k * kThreads < T ? __ldg(slots + t0 + k * kThreads) : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int s = slot[k], i = t0 + k * kThreads - w0;
      if (unsigned(s) >= n_slots) continue;
      for (int f = w.head[(s >> bs_log2) % kHash]; f >= 0; f = w.next[f]) {
        const int first = s_slot[f + 1];
        if ((s >> bs_log2) != (first >> bs_log2)) continue;
        if (i >= w.end[f]) atomicOr(&w.state[f], kFollowed);
        if (i < f && (first & ((1 << bs_log2) - 1)) != 0)
          atomicOr(&w.state[f], s < first ? kContinues : kContinues | kRepeats);
      }
    }
  }
  __syncthreads();
}

// All threads: the later runs, from token `t` on, in the block of `slot`, whose rows up to that
// one are written.
template <bool kF16>
__device__ __noinline__ void follow_block(const AppendParams& p, const uint4* x, uint2* pool,
                                          float* scale, int slot, int t, int g, bool record,
                                          WindowRuns& w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = 1 << p.bs_log2, blk = slot >> p.bs_log2;
  const size_t block = size_t(blk) * p.Hkv + g;
  uint2* const rows = pool + (block << p.bs_log2) * 32;
  const auto inside = [&](int i) {
    const int s = __ldg(p.slots + i);
    return s >= 0 && (s >> p.bs_log2) == blk;
  };
  int most = slot & (bs - 1);              // last row that a token of the call had so far
  while (t < p.T) {
    __syncthreads();
    if (tid == 0) w.found = p.T;
    __syncthreads();
    for (; t < p.T; t += 8 * kThreads) {   // the next token in the block
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        const int i = t + k * kThreads + tid;
        if (i < p.T && inside(i)) {
          atomicMin(&w.found, i);
          break;
        }
      }
      __syncthreads();
      const bool hit = w.found < p.T;
      __syncthreads();                     // read by all before the next ones are looked at
      if (hit) break;
    }
    t = w.found;
    if (t >= p.T) return;
    const int row = __ldg(p.slots + t) & (bs - 1);
    const bool start = !inside(t - 1);     // (t > 0: it comes behind a run)
    if (tid == 0) w.len = bs - row;
    __syncthreads();
    if (tid < bs - row && (t + tid >= p.T || __ldg(p.slots + t + tid) != __ldg(p.slots + t) + tid))
      atomicMin(&w.len, tid);
    __syncthreads();
    const int n = w.len;
    if (start && row > most) {
      if (tid == 0) w.found = 0;           // here: largest |x|
      __syncthreads();
      for (int i = warp; i < n; i += kWarps) {
        const uint32_t a =
            finite_row_amax<kF16>(__ldg(x + (size_t(t + i) * p.Hkv + g) * 32 + lane));
        if (lane == 0) atomicMax(&w.found, int(a));
      }
      const float old = scale[block];
      __syncthreads();
      const int e = max(scale_exp(__float_as_uint(elem_to_float<kF16>(uint32_t(w.found)))), stored_exp(old));
      const float inv = inv_pow2f(e);
      if (tid == 0) scale[block] = pow2f(e);
      if (pow2f(e) != old) rescale_rows(rows, row, old, inv);
      for (int i = warp; i < n; i += kWarps) {
        float f[8];
        unpack8<kF16>(__ldg(x + (size_t(t + i) * p.Hkv + g) * 32 + lane), f);
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] *= inv;
        rows[(row + i) * 32 + lane] = to_e4m3x8(f);
      }
    } else if (start && row == 0 && record) {
      record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);   // the block is begun twice
    }
    most = max(most, row + n - 1);
    t += n;
  }
}

// One CTA: the runs that start in its window of 64 tokens, for one KV head of K or V.
// A token's run is the tokens before it in the same block; a run is at most one block.
// Every warp keeps 8 of the first 64 rows in registers between the maximum and the rounding;
// rows of the last run past them are read twice.
template <bool kF16>
__global__ void __launch_bounds__(kThreads, 4) kv8_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int s_slot[kSpan + 1];          // slot of token w0 - 1 + i
  __shared__ uint32_t s_start[kSpan / 32];   // bit i: token w0 + i starts a run
  __shared__ uint32_t s_break[kSpan / 32];   // bit i: token w0 + i starts a run or is in none
  __shared__ int s_run[kSpan];               // first token of token w0 + i's run, -1: none here
  __shared__ int s_row[kSpan];               // its pool row ((block * Hkv + g) * bs + row)
  __shared__ uint32_t s_max[kWindow];        // by run (its first token): largest |x|, 16 bits
  __shared__ float s_inv[kWindow];           // one over its scale
  __shared__ float s_old[kWindow];           // the scale that the rows before it have
  __shared__ int s_grown[kWindow];
  __shared__ int s_n_grown;
  __shared__ WindowRuns s_runs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w0 = blockIdx.x * kWindow, g = blockIdx.y, kv = blockIdx.z;
  const int bs = 1 << p.bs_log2;
  const int n_span = min(kWindow + bs, p.T - w0);   // tokens from w0 on that matter here
  const uint4* const x = kv == 0 ? p.x[0] : p.x[1];
  uint2* const pool = kv == 0 ? p.pool[0] : p.pool[1];

  let_next_start();
  wait_for_last();
  for (int i = tid; i < kSpan + 1; i += kThreads) {
    const int t = w0 - 1 + i;
    s_slot[i] = t >= 0 && i <= n_span ? __ldg(p.slots + t) : -1;
  }
  if (tid < kWindow) {
    s_max[tid] = 0u;
    s_runs.state[tid] = 0;
  }
  s_runs.head[tid] = -1;
  if (tid == 0) s_n_grown = s_runs.n_asks = 0;
  __syncthreads();
  const long long n_slots = (long long)p.num_blocks << p.bs_log2;
  if (tid < kSpan) {   // kSpan / 32 whole warps
    const int before = s_slot[tid], s = s_slot[tid + 1];
    bool in = s >= 0 && s < n_slots;
    bool start = in && (before < 0 || before >= n_slots || s != before + 1 || (s & (bs - 1)) == 0);
    // a token in the block of the one before it but not behind it has no place
    const bool bad = (s < -1 || s >= n_slots) ||
                     (start && before >= 0 && (s >> p.bs_log2) == (before >> p.bs_log2));
    if (bad) {
      in = start = false;
      if (tid < kWindow && g == 0 && kv == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    }
    const uint32_t st = __ballot_sync(0xffffffffu, start);
    const uint32_t br = __ballot_sync(0xffffffffu, start || !in);
    if (lane == 0) {
      s_start[warp] = st;
      s_break[warp] = br;
    }
  }
  __syncthreads();
  // Rows before the first run belong to the window before; the 64 from it on are loaded now.
  const uint64_t starts = (uint64_t(s_start[1]) << 32) | s_start[0];
  const bool starts_run = tid < kWindow && ((starts >> tid) & 1ull);
  const int i0 = starts == 0ull ? kSpan : __ffsll(static_cast<long long>(starts)) - 1;
  uint4 u[kRowsPerWarp];
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) {
    const int i = i0 + warp + k * kWarps;
    if (i < n_span) u[k] = __ldg(x + (size_t(w0 + i) * p.Hkv + g) * 32 + lane);
  }
  if (tid < kSpan) {
    int f = -1;
    if (tid < n_span) {
      int w = tid >> 5;
      uint32_t m = s_break[w] & (0xffffffffu >> (31 - (tid & 31)));
      while (m == 0u && w > 0) m = s_break[--w];
      if (m != 0u) f = w * 32 + 31 - __clz(m);
      if (f >= kWindow || (f >= 0 && !((s_start[f >> 5] >> (f & 31)) & 1u))) f = -1;
    }
    const int s = s_slot[tid + 1];
    s_run[tid] = f;
    s_row[tid] = f < 0 ? 0 : (((s >> p.bs_log2) * p.Hkv + g) << p.bs_log2) + (s & (bs - 1));
  }
  bool other = false;   // other tokens of the call may be in the block of the run that starts here
  if (starts_run) {
    int end = tid + 1;
    for (; end < kSpan; end = (end | 31) + 1) {
      const uint32_t m = s_break[end >> 5] >> (end & 31);
      if (m != 0u) {
        end += __ffs(int(m)) - 1;
        break;
      }
    }
    const int row = s_slot[tid + 1] & (bs - 1);
    s_runs.end[tid] = end;
    const int block = s_slot[tid + 1] - row;
    if (row != 0 && w0 + tid > 0) {
      other = true;
      const int a = atomicAdd(&s_runs.n_asks, 1);
      if (a < 2 * kFew) s_runs.ask[a] = Ask{0, w0 + tid, unsigned(block)};
    }
    if (row + end - tid < bs && w0 + end < p.T) {
      other = true;
      const int a = atomicAdd(&s_runs.n_asks, 1);
      if (a < 2 * kFew) s_runs.ask[a] = Ask{w0 + end, p.T, unsigned(block)};
    }
  }
  if (p.T <= 32 && warp == 0) {   // a small step: the lanes have all of its tokens
    const int s = s_slot[lane + 1];
    const uint32_t same = __match_any_sync(0xffffffffu, s >= 0 && s < n_slots ? s >> p.bs_log2 : -1 - lane);
    if (other) {
      const int end = s_runs.end[lane];
      other = ((same & ((1u << lane) - 1u)) | (end < 32 ? same >> end : 0u)) != 0u;
    }
  }
  const int n_other = __syncthreads_count(other);
  bool looked = n_other > 0;   // the same in all threads, as all of what follows
  if (looked) {
    // the rows' loads (32 lines a warp) wait behind this: they are on their way to L2 meanwhile
    const int i = i0 + warp + (lane >> 2) * kWarps;
    if (i < n_span)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(x + (size_t(w0 + i) * p.Hkv + g) * 32 + (lane & 3) * 8));
  }
  // (the list holds what kFew runs ask; a step of 32 tokens has its answer)
  if (looked && n_other <= kFew && p.T > 32) looked = any_in_block(p.slots, unsigned(bs), s_runs);
  if (looked) {
    look_around(p.slots, p.T, w0, unsigned(n_slots), p.bs_log2, s_slot, other, s_runs);
    if (starts_run && (s_runs.state[tid] & kRepeats) && g == 0 && kv == 0)
      record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    if (tid < n_span && s_run[tid] >= 0 && (s_runs.state[s_run[tid]] & kContinues)) s_run[tid] = -1;
    if (tid < kWindow) {
      const uint32_t m = __ballot_sync(
          0xffffffffu, starts_run && (s_runs.state[tid] & (kContinues | kFollowed)) == kFollowed);
      if (lane == 0) s_runs.followed[warp] = m;
    }
    __syncthreads();
  }
  const auto run_of = [&](int i) -> int { return i < n_span ? s_run[i] : -1; };
  int run[kRowsPerWarp];
  constexpr uint32_t kInf = kF16 ? 0x7C00u : 0x7F80u;
  bool finite = true;      // no row of this warp holds a NaN or an infinity
  uint32_t m = 0u;         // maxima of the lane's elements in the run of the last rows
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) run[k] = run_of(i0 + warp + k * kWarps);
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) {
    if (run[k] < 0) continue;
    m = __vmaxu2(m, lane_amax(u[k]));
    if (k + 1 < kRowsPerWarp && run[k + 1] == run[k]) continue;
    const uint32_t a = warp_amax(m);
    m = 0u;
    finite = finite && a < kInf;
    if (a < kInf && lane == 0) atomicMax(&s_max[run[k]], a);
  }
  if (!finite) {           // the same in all lanes: rows one by one, without such elements
#pragma unroll 1
    for (int i = i0 + warp; i < i0 + kWindow; i += kWarps) {
      const int r = run_of(i);
      if (r < 0) continue;
      const uint32_t a = finite_row_amax<kF16>(__ldg(x + (size_t(w0 + i) * p.Hkv + g) * 32 + lane));
      if (lane == 0) atomicMax(&s_max[r], a);
    }
  }
  for (int i = i0 + kWindow + warp; i < n_span; i += kWarps) {
    const int r = run_of(i);
    if (r < 0) break;   // past the last run
    const uint4 v = __ldg(x + (size_t(w0 + i) * p.Hkv + g) * 32 + lane);
    uint32_t a = warp_amax(lane_amax(v));
    if (a >= kInf) a = finite_row_amax<kF16>(v);
    if (lane == 0) atomicMax(&s_max[r], a);
  }
  __syncthreads();
  if (starts_run && !(s_runs.state[tid] & kContinues)) {
    const int s = s_slot[tid + 1];
    float* const sp = (kv == 0 ? p.scale[0] : p.scale[1]) + size_t(s >> p.bs_log2) * p.Hkv + g;
    int e = scale_exp(__float_as_uint(elem_to_float<kF16>(s_max[tid])));
    if ((s & (bs - 1)) != 0) {
      const float old = *sp;
      e = max(e, stored_exp(old));
      if (pow2f(e) != old) {
        s_old[tid] = old;
        s_grown[atomicAdd(&s_n_grown, 1)] = tid;
      }
    }
    s_inv[tid] = inv_pow2f(e);
    *sp = pow2f(e);
  }
  __syncthreads();
  const auto put = [&](int i, int r, uint4 v, bool all) {
    float f[8];
    unpack8<kF16>(v, f);
    const float inv = s_inv[r];
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      const float2 y = mul2(make_float2(f[c], f[c + 1]), make_float2(inv, inv));
      f[c] = y.x;
      f[c + 1] = y.y;
    }
    pool[size_t(s_row[i]) * 32 + lane] = all ? finite_to_e4m3x8(f) : to_e4m3x8(f);
  };
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k)
    if (run[k] >= 0) put(i0 + warp + k * kWarps, run[k], u[k], finite);
  for (int i = i0 + kWindow + warp; i < n_span; i += kWarps) {
    const int r = run_of(i);
    if (r < 0) break;
    put(i, r, __ldg(x + (size_t(w0 + i) * p.Hkv + g) * 32 + lane), false);
  }
  for (int j = 0; j < s_n_grown; ++j) {
    const int r = s_grown[j], n = s_row[r] & (bs - 1);
    rescale_rows(pool + size_t(s_row[r] - n) * 32, n, s_old[r], s_inv[r]);
  }
  if (!looked) return;
  for (uint64_t left = (uint64_t(s_runs.followed[1]) << 32) | s_runs.followed[0]; left != 0ull;
       left &= left - 1ull) {
    const int f = __ffsll(static_cast<long long>(left)) - 1;
    __syncthreads();   // the run's rows, those before them and its scale are written
    follow_block<kF16>(p, x, pool, kv == 0 ? p.scale[0] : p.scale[1],
                       s_slot[s_runs.end[f]], w0 + s_runs.end[f], g, g == 0 && kv == 0, s_runs);
  }
}

// ---------------------------------------------------------------- keep
constexpr int kMaxKeep = 64;                              // as many as a tree has rows
constexpr int kKeepPerWarp = kMaxKeep / kWarps;
constexpr int kMaxRuns = kMaxKeep / 16 + 1;               // blocks that they can touch

struct KeepParams {
  uint2* pool[2];
  float* scale[2];
  const int* tables;
  const int* kv_lens;
  const int* cu_rows;
  const int* keep_idx;
  const int* cu_keep;
  int* lens_out;
  int n_keep, B, Hkv, num_blocks, max_blocks, bs_log2;
  LaunchCtl ctl;
};

// One CTA: one sequence and KV head of K or V.  All kept rows are in registers before
// the first is written (a block's scale may change while later rows of it are due).
__global__ void __launch_bounds__(kThreads, 6) kv8_keep_kernel(const KeepParams p) {
  __shared__ int s_src[kMaxKeep];          // pool row (block * bs + row) of kept row k, and
  __shared__ int s_dst[kMaxKeep];          // its place
  __shared__ uint32_t s_max[kMaxRuns];
  __shared__ float s_inv[kMaxRuns];
  __shared__ float s_old;                  // scale of the rows that stay before the first run
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, g = blockIdx.y, kv = blockIdx.z;
  const int bs = 1 << p.bs_log2;
  let_next_start();
  wait_for_last();
  const int r = p.cu_rows[b + 1] - p.cu_rows[b];
  const int L = p.kv_lens[b];
  const int k0 = p.cu_keep[b], nk = p.cu_keep[b + 1] - k0;
  const int base = L - r;
  const int* const table = p.tables + (long long)b * p.max_blocks;
  const bool ok = r >= 0 && L >= r && nk >= 0 && nk <= r && nk <= kMaxKeep && k0 >= 0 &&
                  (long long)k0 + nk <= p.n_keep &&
                  (long long)L <= ((long long)p.max_blocks << p.bs_log2);
  bool bad = !ok;
  if (ok && tid < nk) {
    const int i = p.keep_idx[k0 + tid];
    const int before = tid == 0 ? -1 : p.keep_idx[k0 + tid - 1];
    const int dst = table[(base + tid) >> p.bs_log2];
    bad = i < 0 || i >= r || i <= before || dst < 0 || dst >= p.num_blocks;
    const int src = bad ? -1 : table[(base + i) >> p.bs_log2];
    bad = bad || src < 0 || src >= p.num_blocks;
    s_src[tid] = (src << p.bs_log2) + ((base + i) & (bs - 1));
    s_dst[tid] = (dst << p.bs_log2) + ((base + tid) & (bs - 1));
  }
  if (tid < kMaxRuns) s_max[tid] = 0u;
  if (__syncthreads_or(bad)) {
    if (tid == 0 && g == 0 && kv == 0) record_status(p.ctl.status, GQA_ERR_DEVICE_RANGE);
    return;
  }
  if (tid == 0 && g == 0 && kv == 0 && p.lens_out != nullptr) p.lens_out[b] = base + nk;
  if (nk == 0) return;
  uint2* const pool = kv == 0 ? p.pool[0] : p.pool[1];
  float* const scale = kv == 0 ? p.scale[0] : p.scale[1];
  // 8-byte units of pool row `at`, and its block's scale
  const auto row_of = [&](int at) {
    return ((size_t(at >> p.bs_log2) * p.Hkv + g) * bs + (at & (bs - 1))) * 32;
  };
  const auto scale_of = [&](int at) { return scale + size_t(at >> p.bs_log2) * p.Hkv + g; };
  const int run0 = base >> p.bs_log2;
  const int n_runs = ((base + nk - 1) >> p.bs_log2) - run0 + 1;
  uint2 q[kKeepPerWarp];
  float sc[kKeepPerWarp];
#pragma unroll
  for (int k = 0; k < kKeepPerWarp; ++k) {
    const int i = warp + k * kWarps;
    if (i >= nk) continue;
    q[k] = pool[row_of(s_src[i]) + lane];
    sc[k] = *scale_of(s_src[i]);
  }
  if (tid == 0) s_old = *scale_of(s_dst[0]);
#pragma unroll
  for (int k = 0; k < kKeepPerWarp; ++k) {
    const int i = warp + k * kWarps;
    if (i >= nk) continue;
    float f[8];
    from_e4m3x8(q[k], f);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] *= sc[k];
    const uint32_t m = __reduce_max_sync(0xffffffffu, finite_amax_bits(f));
    if (lane == 0) atomicMax(&s_max[((base + i) >> p.bs_log2) - run0], m);
  }
  __syncthreads();   // every kept row and its scale are read
  const int off0 = base & (bs - 1);
  if (tid < n_runs) {
    int e = scale_exp(s_max[tid]);
    if (tid == 0 && off0 != 0) e = max(e, stored_exp(s_old));
    s_inv[tid] = inv_pow2f(e);
    // the run's first row: kept row 0, or the first one of its block
    *scale_of(s_dst[tid == 0 ? 0 : ((run0 + tid) << p.bs_log2) - base]) = pow2f(e);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeepPerWarp; ++k) {
    const int i = warp + k * kWarps;
    if (i >= nk) continue;
    const float inv = s_inv[((base + i) >> p.bs_log2) - run0];
    float f[8];
    from_e4m3x8(q[k], f);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = f[c] * sc[k] * inv;
    pool[row_of(s_dst[i]) + lane] = to_e4m3x8(f);
  }
  if (off0 != 0 && s_old * s_inv[0] != 1.f)
    rescale_rows(pool + row_of(s_dst[0] - off0), off0, s_old, s_inv[0]);
}

int log2_of(int block_size) {
  int n = 0;
  while ((1 << n) < block_size) ++n;
  return n;
}

int append_impl(bool f16, const void* Knew, const void* Vnew, const int* slots, void* k_pool,
                void* v_pool, float* k_scale, float* v_scale, int T, int Hkv, int num_blocks,
                int block_size, gqa_stream_t stream) {
  if (T < 0) return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, Hkv, block_size);
  if (st != GQA_OK) return st;
  // (token indexes run a few windows past T)
  if (Hkv > 65535 || (long long)T * Hkv >= (1LL << 31) - kAsk * kThreads) return GQA_ERR_UNSUPPORTED;
  if (T == 0) return GQA_OK;
  if (Knew == nullptr || Vnew == nullptr || slots == nullptr || k_pool == nullptr ||
      v_pool == nullptr || k_scale == nullptr || v_scale == nullptr)
    return GQA_ERR_INVALID_ARG;
  if (!aligned_to(Knew, 16) || !aligned_to(Vnew, 16) || !aligned_to(k_pool, 16) ||
      !aligned_to(v_pool, 16) || !aligned_to(slots, 4) || !aligned_to(k_scale, 4) ||
      !aligned_to(v_scale, 4))
    return GQA_ERR_INVALID_ARG;
  AppendParams p;
  p.x[0] = static_cast<const uint4*>(Knew);
  p.x[1] = static_cast<const uint4*>(Vnew);
  p.pool[0] = static_cast<uint2*>(k_pool);
  p.pool[1] = static_cast<uint2*>(v_pool);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.slots = slots;
  p.T = T;
  p.Hkv = Hkv;
  p.num_blocks = num_blocks;
  p.bs_log2 = log2_of(block_size);
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  const dim3 grid((T + kWindow - 1) / kWindow, Hkv, 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_dependent(f16 ? kv8_append_kernel<true> : kv8_append_kernel<false>, grid, kThreads, 0,
                       s, 1, p) != cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch(f16 ? "kv8_append_kernel<fp16>" : "kv8_append_kernel<bf16>",
              (long long)grid.x * grid.y * grid.z, kThreads, 0);
  return GQA_OK;
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

int gqa_kv8_append(const void* Knew, const void* Vnew, const int* slots, void* k_pool, void* v_pool,
                   float* k_scale, float* v_scale, int T, int Hkv, int num_blocks, int block_size,
                   gqa_stream_t stream) {
  return append_impl(false, Knew, Vnew, slots, k_pool, v_pool, k_scale, v_scale, T, Hkv,
                     num_blocks, block_size, stream);
}
int gqa_kv8_append_f16(const void* Knew, const void* Vnew, const int* slots, void* k_pool,
                       void* v_pool, float* k_scale, float* v_scale, int T, int Hkv,
                       int num_blocks, int block_size, gqa_stream_t stream) {
  return append_impl(true, Knew, Vnew, slots, k_pool, v_pool, k_scale, v_scale, T, Hkv, num_blocks,
                     block_size, stream);
}

int gqa_kv8_keep(void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                 const int* block_tables, const int* kv_lens, const int* cu_rows,
                 const int* keep_idx, const int* cu_keep, int* kv_lens_out, int n_keep, int B,
                 int Hkv, int num_blocks, int block_size, int max_blocks, gqa_stream_t stream) {
  if (B < 1 || max_blocks < 1 || n_keep < 0) return GQA_ERR_INVALID_ARG;
  const int st = check_kv8_pool(num_blocks, Hkv, block_size);
  if (st != GQA_OK) return st;
  if (Hkv > 65535 || (long long)max_blocks * block_size >= (1LL << 31)) return GQA_ERR_UNSUPPORTED;
  if (k_pool == nullptr || v_pool == nullptr || k_scale == nullptr || v_scale == nullptr ||
      block_tables == nullptr || kv_lens == nullptr || cu_rows == nullptr ||
      (keep_idx == nullptr && n_keep > 0) || cu_keep == nullptr || kv_lens_out == kv_lens)
    return GQA_ERR_INVALID_ARG;
  if (!aligned_to(k_pool, 16) || !aligned_to(v_pool, 16)) return GQA_ERR_INVALID_ARG;
  for (const void* q : {(const void*)k_scale, (const void*)v_scale, (const void*)block_tables,
                        (const void*)kv_lens, (const void*)cu_rows, (const void*)keep_idx,
                        (const void*)cu_keep, (const void*)kv_lens_out})
    if (!aligned_to(q, 4)) return GQA_ERR_INVALID_ARG;
  KeepParams p;
  p.pool[0] = static_cast<uint2*>(k_pool);
  p.pool[1] = static_cast<uint2*>(v_pool);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.tables = block_tables;
  p.kv_lens = kv_lens;
  p.cu_rows = cu_rows;
  p.keep_idx = keep_idx;
  p.cu_keep = cu_keep;
  p.lens_out = kv_lens_out;
  p.n_keep = n_keep;
  p.B = B;
  p.Hkv = Hkv;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks;
  p.bs_log2 = log2_of(block_size);
  if (!make_launch_ctl(&p.ctl)) return GQA_ERR_CUDA;
  const dim3 grid(B, Hkv, 2);
  if (launch_dependent(kv8_keep_kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), 1, p) !=
      cudaSuccess)
    return GQA_ERR_CUDA;
  note_launch("kv8_keep_kernel", (long long)B * Hkv * 2, kThreads, 0);
  return GQA_OK;
}

}  // extern "C"
