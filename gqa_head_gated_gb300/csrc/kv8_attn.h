// The split kernel of the paged 8-bit cache's attention (kv8_attn.cu), launched by
// kv8_decode.cu.
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace gqa {

constexpr int kKv8Seqs = 256;   // sequences that one launch schedules

struct Kv8AttnArgs {
  const uint4* q;             // 16-bit [T, Hq, 256]
  const uint8_t* k_pool;      // e4m3 [num_blocks, Hkv, block_size, 256]
  const uint8_t* v_pool;
  const float* k_scale;       // [num_blocks, Hkv]
  const float* v_scale;
  const int* tables;          // this and the next two: from sequence b0 on
  const int* kv_lens;
  const int* cu_rows;         // null: one row per sequence
  const unsigned long long* tree_mask;
  float* o_parts;             // [parts, T * Hq, 256]
  float* lse_parts;           // [parts, T * Hq]
  int* n_parts;               // [B of the call, Hkv, max_rb]: parts written for each segment
  int b0, B, T, Hkv, Hq, gqa, num_blocks, bs_log2, max_blocks, max_rows, max_kv_len, max_rb, parts;
  LaunchCtl ctl;
};

// Packed rows (query heads of a group x new rows) that a segment of the kernel takes.
int kv8_rows_per_block(long long packed_rows);

// a.B <= kKv8Seqs, a.parts >= 3, B * Hkv * max_rb * (tiles of 128 keys in max_kv_len) < 2^31.
cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, bool f16, int sms, cudaStream_t stream,
                            bool* encode_failed);
// The kernel for 128 packed rows (launch_kv8_attn picks it).
cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, bool f16, int sms, cudaStream_t stream,
                            bool* encode_failed);

}  // namespace gqa
