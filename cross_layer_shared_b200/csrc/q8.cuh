// Launch interface of the kernels on an 8-bit cache (internal to libsa), and
// the code format they share.
//
// Format: x ~ s * c with c an e4m3 code and s = 2^e one scale per block of 64
// tokens and KV head; e is the smallest integer >= -126 with
// max|x| <= 448 * 2^e over the block's finite values.  e4m3 is a floating
// format, so a power-of-two scale keeps its relative step (2^-4) for all but
// the smallest values, every product with a scale is exact, and so is moving
// a block's codes to a larger scale, except where they become subnormal.
// Sequence b owns cap = seq_off[b+1] - seq_off[b] token places (a multiple of
// 64) laid out [Hkv, cap, d] from row seq_off[b]*Hkv on, so the scale of row r
// is scales[r / 64].
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "status.cuh"

namespace sa {

constexpr int kQ8Block = 64;
constexpr uint32_t kQ8MinScaleBits = 1u << 23;  // 2^-126

// tiles of `tile` tokens that hold len of them, for every len >= 0 an int holds
__host__ __device__ constexpr int q8_tiles(int len, int tile) { return len / tile + (len % tile != 0); }
static_assert(q8_tiles(0, 128) == 0 && q8_tiles(1, 128) == 1 && q8_tiles(128, 128) == 1 && q8_tiles(129, 128) == 2 &&
                  q8_tiles(0x7fffffc0, 128) == 1 << 24,
              "counted without passing 32 bits");

// One sequence's place in the cache; ok is false (and the sequence counts as
// empty) when the offsets do not describe one or len does not fit.
struct Q8Seq {
  int64_t off;  // first token place
  int cap, len;
  bool ok;
};

__device__ __forceinline__ Q8Seq q8_seq(const int64_t* seq_off, const int32_t* seq_len, int b, int64_t n_tokens,
                                        int S_max) {
  Q8Seq s;
  s.off = __ldcg(reinterpret_cast<const long long*>(seq_off) + b);
  const int64_t end = __ldcg(reinterpret_cast<const long long*>(seq_off) + b + 1);
  s.len = __ldcg(&seq_len[b]);
  const int64_t cap = end - s.off;
  s.ok = s.off >= 0 && cap >= 0 && end <= n_tokens && (s.off | end) % kQ8Block == 0 && s.len >= 0 && s.len <= cap &&
         s.len <= S_max;
  s.cap = s.ok ? (int)cap : 0;
  if (!s.ok) s.len = 0;
  return s;
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ---- conversions ----
// four e4m3 codes -> four halves (exact), two per register
__device__ __forceinline__ void q8_to_half4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}

// the e4m3 codes nearest to four floats (ties to even; beyond +-448 the
// largest code, NaN the NaN code), v0 in the lowest byte
__device__ __forceinline__ uint32_t q8_from_float4(float v0, float v1, float v2, float v3) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\tmov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
  return r;
}

// bits of the smallest power of two s >= 2^-126 with amax <= 448 s, from the
// bits of a finite amax >= 0: 448 = 1.75 * 2^8
__device__ __forceinline__ uint32_t q8_scale_bits(uint32_t amax_bits) {
  int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
  if (e < 1) e = 1;
  return (uint32_t)e << 23;
}

// ---- clusters ----
// shared memory of the cluster's CTA `rank`, at this CTA's address
__device__ __forceinline__ float4 ld_peer4(uint32_t addr, int rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr, int rank) {
  uint32_t at;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- cache_q8.cu ----
struct Q8Cache {
  uint8_t* codes[2];  // K and V (or one tensor: [1] null)
  float* scales[2];
};

struct Q8AppendArgs {
  const void* rows[2];    // new rows, token i of head h at element i*stride + h*d
  int64_t stride[2];      // elements
  int64_t n_rows;         // tokens in rows
  const int64_t* new_off; // [B+1], or null: one token per sequence
  int max_new;
  Q8Cache cache;
  const int64_t* seq_off;
  const int32_t* seq_len;
  int B, Hkv, d;
  int64_t n_tokens;
  int in_f32;
  DeviceStatus* status;
};
cudaError_t launch_cache_append_q8(const Q8AppendArgs& a, int num_sms, cudaStream_t stream);

struct Q8ReadArgs {
  Q8Cache cache;
  const int64_t* seq_off;
  const int32_t* seq_len;
  int B, Hkv, d, S_max;
  int64_t n_tokens;
  const int32_t* idx;      // [B, k], or null: whole sequences
  int k;
  const int64_t* out_off;  // whole sequences: [B+1] token offsets in the packed output
  int64_t n_out;
  void* out[2];
  int out_f32, out_wide;   // out_wide: both outputs are 32-byte aligned
  DeviceStatus* status;
};
cudaError_t launch_cache_read_q8(const Q8ReadArgs& a, cudaStream_t stream);

// ---- indexer_q8.cu ----
struct Q8IndexerArgs {
  const uint16_t* qI;  // bf16 [B, H_I, d_I]
  const float* w;
  const float* scales;
  const int64_t* seq_off;
  const int32_t* seq_len;
  int B;
  int64_t n_tokens;
  int S_max, H_I, d_I;
  float* scores;
  int64_t ld;
  DeviceStatus* status;
};
// tm_ki: codes as u8 [n_tokens, d_I], box (128, 128), 128-byte swizzle
cudaError_t launch_indexer_q8(const Q8IndexerArgs& a, const CUtensorMap& tm_ki, int num_sms, cudaStream_t stream);

// ---- attn_q8.cu ----
constexpr int kQ8RowTile = 128;     // query rows of a CTA of attn_q8_group.cu
// key slices of a unit: their (m, l) of `rows` rows fit the merging CTA's shared memory
__host__ __device__ constexpr int q8_max_splits(int rows) { return 8192 / rows < 256 ? 8192 / rows : 256; }
struct Q8AttnArgs {
  const uint16_t* Q;
  const uint8_t* K;
  const float* Ks;
  const uint8_t* V;
  const float* Vs;
  const int64_t* seq_off;
  const int32_t* seq_len;
  const int32_t* idx;  // [B, k], or null: every token
  int k;
  int B, Hq, Hkv, G, R, S_max;
  int64_t n_tokens;
  float scale_log2;
  void* O;
  int out_f32;
  int n_split, chunk;  // key slices of chunk keys (of the index entries, or of the tokens)
  int cluster;         // slices that merge as a cluster (0: through the workspace)
  // n_split > 1: counters per (b, g, row tile), zero between launches, and
  // the slices' partials [unit][n_split][rows][128], (m, l) [unit][n_split][rows]
  uint32_t* cnt;
  float* po;
  float2* pml;
  DeviceStatus* status;
};
struct Q8AttnPlan {
  bool group;  // attn_q8_group.cu
  int row_tiles, units, n_split, chunk, cluster;
  int parts, rows;  // partial results of a unit, and the query rows of each (padded)
};
Q8AttnPlan plan_attn_q8(int R, int B, int Hkv, int64_t n_tokens, int S_max, int k, int sms, int max_counters);
size_t attn_q8_scratch_bytes(const Q8AttnPlan& p);
cudaError_t launch_attn_q8(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream);

// ---- attn_q8_group.cu ----
void plan_attn_q8_group(Q8AttnPlan& p, int64_t n, int sms);
cudaError_t launch_attn_q8_group(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream);

}  // namespace sa
