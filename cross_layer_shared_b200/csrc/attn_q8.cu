// Decode attention over the 8-bit cache (format in q8.cuh), over the tokens
// of an index or over every token:
//   z_t = scale * ks_t (q . ck_t),  o = sum_t softmax(z)_t vs_t cv_t
// with ck, cv the token's codes and ks, vs its blocks' scales.
//
// What bounds it: 256 + 8/64 bytes per (token, KV head) for 4*128*R flops, R
// query rows.  A decode layer has R <= 8: HBM over long contexts, latency
// over a short index.  So the kernel is built to keep many independent copies
// in flight, and its products run on warp-level MMA tiles (a tcgen05 tile is
// at least 64 rows, and its TMEM and commit chain costs more than a whole
// pass here).
//
//   * One CTA of 8 warps per (sequence, KV head, 8 or 16 query rows, slice of
//     the keys), two CTAs per SM (much work of many rows: attn_q8_group.cu).
//     Each warp walks keys of its own 16 at a time with a ring of three stages
//     (K and V codes and scales by cp.async, two passes ahead): warps never
//     wait for one another.
//   * e4m3 codes become halves exactly (one conversion per two codes), in
//     registers: S^T = K Q^T and O^T = V^T P^T are m16n8k16 f16 MMAs with fp32
//     accumulators.  Queries are scaled per row by a power of two into the
//     upper half of f16's range, which keeps all 8 bits of a bf16 element
//     over 29 binades below the row's largest.
//   * The dims of a k-step are permuted (the dot product does not care) so
//     that a lane's K operands are two 16-byte pieces of a row.  V^T comes
//     from ldmatrix.trans on pairs of codes: a lane gets two dims of two keys,
//     one byte permute turns that into two operand registers' worth of codes.
//   * P^T's operand layout is one movmatrix away from S^T's accumulators.  For
//     fp32 outputs P is split into two halves (22 bits, down to 2^-10 of the
//     row's largest); for bf16 outputs one half (11 bits, eight times finer
//     than the output's rounding).
//   * The V scale vs = f 2^e (f = 1 for the powers of two an append writes)
//     joins the logit: o sums f 2^(z + e - m_o) cv with a reference m_o over
//     z + e of its own, l sums 2^(z - m_l).  So a key's weight is held
//     relative to the largest contribution, however far the scales are apart.
//   * m_o moves only when some key passes it by more than 14 (log2 units) and
//     is then set 7 below the maximum: weights, f < 2 included, stay below
//     2^15 and most of f16's range is above its subnormals: a weight times its
//     V scale keeps a half's 11 bits down to 2^-21 of the row's largest, is off
//     by at most 2^-32 of that in one half or two (f16's last subnormal bit,
//     2^-24, where the largest is 2^7 or more), and one below that is lost.  l
//     is a float: m_l moves past 60.
//   * Padding entries and tokens past the length have codes zero and weight
//     zero, whatever the cache holds there.
//   * Partial results travel normalised: (m, l, o / l).  A weighted mean of V
//     rows cannot leave V's own range, whatever the scales.
//   * The slices of a short unit are a cluster of up to 8 CTAs and merge in
//     shared memory.  More slices leave their results (a cluster's, or with
//     much work each slice's) in the workspace and count themselves on a
//     counter in its header; the last one merges them and puts the counter back
//     to zero.  Results do not depend on which is last.
//
// Measured (B200, warm graph replay): every token of 4 x 131072, 32 query and 8
// KV heads, 178 us = 92 % of the measured HBM rate; 8 sequences over 2048
// picked tokens, 32 / 4 heads, 10.2 us (17 MB: latency); two sequences of 333
// and 1021 tokens 5.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_warp.cuh"
#include "q8.cuh"
#include "sm100.cuh"
#include "status.cuh"

namespace sa {
namespace {
using namespace wm;

constexpr int kDq = 128;
constexpr int kWarpsQ = 8;
constexpr int kThreadsQ = kWarpsQ * 32;
constexpr int kKeysQ = 16;   // keys of a pass
constexpr int kStagesQ = 3;
constexpr float kRangeO = 14.f;  // log2 units z + e may pass m_o by: 2^14 f is finite in f16 for any f < 2
constexpr int kORow = kDq + 4;

struct StageQ {
  uint8_t k[kKeysQ * kDq];  // 16-byte piece c of row r at r*128 + ((c ^ (r & 7)) << 4)
  uint8_t v[kKeysQ * kDq];
  float ks[kKeysQ];
  float vs[kKeysQ];
};

template <int NT>
struct SmemQ {
  static constexpr int kRows = 8 * NT;  // query rows of the CTA
  static constexpr int kKW = kWarpsQ;   // key groups: the warps
  union {
    StageQ ring[kKW][kStagesQ];
    struct {
      float o[kKW][kRows][kORow];  // after the loop: each key group's o
      float f[kKW][kRows];         // .. and its weight
    } w;
    float2 sml[q8_max_splits(kRows)][kRows];  // the merging CTA: each slice's (m, l), then (weight, -)
  };
  uint4 q[NT][4][32];        // the query's B fragments: [8 rows][two k-steps][lane]
  float rf[kRows];                 // per row: softmax scale * log2(e) / query scale
  float2 ml[kKW][kRows];           // each key group's (m, l)
  float2 ML[kRows];                // each row's (reference, sum of weights)
  int64_t out_off[kRows];
  int last;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8x8 matrix of halves, transposed over the warp
__device__ __forceinline__ uint32_t transpose_half(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void cp_async4(void* dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(src_bytes)
               : "memory");
}

// a scale >= 0 as f 2^e: 1 <= f < 2, or from zero up to 2^-126 f < 1 and e =
// -126, so that a key without a contribution does not set the reference of
// those that have one (beside it 2^-32 of 448 2^-126 may be lost: nothing)
__device__ __forceinline__ void split_scale(float s, float& f, float& e) {
  const uint32_t u = __float_as_uint(s);
  const int x = (int)(u >> 23 & 0xff);
  f = x == 0 ? s * 0x1p126f : __uint_as_float((u & 0x7fffffu) | 0x3f800000u);
  e = (float)(max(x, 1) - 127);
}

// max over the 8 lanes that hold one query row's keys
__device__ __forceinline__ float warp_key_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

template <int NT, bool PRECISE>
__global__ void __launch_bounds__(kThreadsQ, 2) attn_q8_kernel(const Q8AttnArgs a, const int row_tiles) {
  using Smem = SmemQ<NT>;
  constexpr int kRows = Smem::kRows, kKW = Smem::kKW;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int slice = blockIdx.x % a.n_split;
  const int unit = blockIdx.x / a.n_split;  // (b, g, row tile)
  const int rt = unit % row_tiles;
  const int g = unit / row_tiles % a.Hkv, b = unit / row_tiles / a.Hkv;
  const int row_base = rt * kRows;
  pdl_trigger();
  pdl_wait();
  // loads that need nothing of the sequence come first: the warp's query rows
  // and the index entries of its first two passes
  uint2 qv[NT];
  int64_t q_off[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int row = row_base + warp + kWarpsQ * i;
    const int l = row < a.G ? 0 : row / a.G;
    q_off[i] = (((int64_t)l * a.B + b) * a.Hq + g * a.G + row - l * a.G) * kDq;
    qv[i] = make_uint2(0u, 0u);
    if (row < a.R) qv[i] = __ldcg(reinterpret_cast<const uint2*>(a.Q + q_off[i]) + lane);  // dims 4*lane ..
  }
  int t_first = -1, t_second = -1;
  if (a.idx) {
    const int64_t e = (int64_t)slice * a.chunk + warp * kKeysQ + (lane & 15);
    const int64_t end = min((int64_t)a.k, (int64_t)(slice + 1) * a.chunk);
    if (e < end) t_first = __ldcg(&a.idx[(int64_t)b * a.k + e]);
    if (e + kKW * kKeysQ < end) t_second = __ldcg(&a.idx[(int64_t)b * a.k + e + kKW * kKeysQ]);
  }
  const Q8Seq s = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
  if (!s.ok && tid == 0 && slice == 0) report(a.status, kErrDevice, kKernAttnQ8, b, s.len, s.cap);
  const int n_keys = !s.ok ? 0 : a.idx ? a.k : s.len;  // entries, or tokens
  const int e_beg = (int)min((int64_t)n_keys, (int64_t)slice * a.chunk);
  const int e_end = (int)min((int64_t)n_keys, (int64_t)e_beg + a.chunk);
  // slices of this unit that have keys (at least one): the others do nothing
  const int n_live = max(1, (int)(((int64_t)n_keys + a.chunk - 1) / a.chunk));
  if (slice >= n_live && !a.cluster) return;
  const int64_t row0 = s.off * a.Hkv + (int64_t)g * s.cap;
  const int e_grp = e_beg + warp * kKeysQ;  // this group's passes: e_grp + p * kKW * 16
  const int n_pass = e_grp < e_end ? (e_end - e_grp + kKW * kKeysQ - 1) / (kKW * kKeysQ) : 0;

  // token of entry lane (< 16) of pass p, or -1; entries past the length are
  // reported when they are used
  auto entry = [&](int p) -> int {
    const int e = e_grp + p * (kKW * kKeysQ) + (lane & 15);
    if (p >= n_pass || e >= e_end) return -1;
    return a.idx ? __ldcg(&a.idx[(int64_t)b * a.k + e]) : e;
  };
  // pass p's copies (t: its entries) into its stage; returns which entries are tokens
  auto issue = [&](int t, int p) -> uint32_t {
    if (t >= s.len) {
      if (g == 0 && rt == 0 && lane < 16)
        report(a.status, kErrDevice, kKernAttnQ8, (int64_t)b * a.k + e_grp + p * (kKW * kKeysQ) + lane, t, s.len);
      t = -1;
    }
    if (p < n_pass) {
      StageQ& st = sm.ring[warp][p % kStagesQ];
#pragma unroll
      for (int i = 0; i < kKeysQ * 8 / 32; ++i) {
        const int j = lane + i * 32;  // 16-byte piece of the 16 rows
        const int r = j >> 3, c = j & 7;
        const int tr = __shfl_sync(0xffffffffu, t, r);
        const int64_t at = (row0 + max(tr, 0)) * kDq + c * 16;
        const uint32_t to = r * kDq + ((c ^ (r & 7)) << 4);
        const uint32_t bytes = tr >= 0 ? 16u : 0u;
        cp_async16(st.k + to, a.K + at, bytes);
        cp_async16(st.v + to, a.V + at, bytes);
      }
      const int64_t at = (row0 + max(t, 0)) / kQ8Block;
      cp_async4(lane < 16 ? &st.ks[lane] : &st.vs[lane - 16], (lane < 16 ? a.Ks : a.Vs) + at, t >= 0 ? 4u : 0u);
    }
    cp_async_commit();
    return __ballot_sync(0xffffffffu, t >= 0);
  };
  if (!a.idx || !s.ok) t_first = entry(0), t_second = entry(1);
  uint32_t seen = issue(t_first, 0);  // of the pass computed next, and of the one after it
  int t_next = entry(2);
  uint32_t seen_after = issue(t_second, 1);

  // ---- the query rows as f16 fragments ----
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = warp + kWarpsQ * i;
    const uint2 v = qv[i];
    const float x0 = bf_lo(v.x), x1 = bf_hi(v.x), x2 = bf_lo(v.y), x3 = bf_hi(v.y);
    const float mx = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
    const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
    // 2^e with the largest element in [2^14, 2^15); 1 for zero or non-finite rows
    int e = mb == 0u || mb >= 0x7f800000u ? 127 : 127 + 14 + 127 - (int)(mb >> 23);
    e = min(e, 253);  // tiny rows: as large as a float scale goes
    const float up = __uint_as_float((uint32_t)e << 23);
    // dims 4*lane ..: lane tq' = lane / 8 of the fragment, k-step lane % 8
    uint2* dst = reinterpret_cast<uint2*>(&sm.q[r >> 3][(lane & 7) >> 1][(r & 7) * 4 + (lane >> 3)]) + (lane & 1);
    *dst = make_uint2(pack_half(x0 * up, x1 * up), pack_half(x2 * up, x3 * up));
    if (lane == 0) {
      sm.rf[r] = a.scale_log2 / up;
      sm.out_off[r] = q_off[i];
    }
  }
  __syncthreads();

  float rf[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    rf[n][0] = sm.rf[n * 8 + 2 * tq];
    rf[n][1] = sm.rf[n * 8 + 2 * tq + 1];
  }
  float m_l[NT][2], m_o[NT][2], l_run[NT][2], o[NT][8][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m_l[n][0] = m_l[n][1] = m_o[n][0] = m_o[n][1] = -INFINITY;
    l_run[n][0] = l_run[n][1] = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[n][c][0] = o[n][c][1] = o[n][c][2] = o[n][c][3] = 0.f;
  }

  for (int p = 0; p < n_pass; ++p) {
    cp_async_wait<1>();
    __syncwarp();  // pass p has landed; pass p - 1's stage is free
    const uint32_t here = seen;
    const bool seen0 = here >> gq & 1, seen1 = here >> (gq + 8) & 1;
    seen = seen_after;
    seen_after = issue(t_next, p + 2);
    t_next = entry(p + 3);
    if (here == 0u) continue;  // padding: the end of a short sequence's index
    const StageQ& st = sm.ring[warp][p % kStagesQ];
    // ---- S^T = K Q^T: lane holds keys gq, gq + 8 at rows 2tq, 2tq + 1 ----
    float sc[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[n][0][i] = sc[n][1][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = gq * kDq + (((2 * tq + i) ^ gq) << 4);
      const uint4 k0 = *reinterpret_cast<const uint4*>(st.k + at);
      const uint4 k1 = *reinterpret_cast<const uint4*>(st.k + at + 8 * kDq);
      const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t f[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          q8_to_half4(w0[2 * j + u], f[u][0], f[u][2]);
          q8_to_half4(w1[2 * j + u], f[u][1], f[u][3]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 q = sm.q[n][2 * i + j][lane];
          mma_f16(sc[n][0], f[0][0], f[0][1], f[0][2], f[0][3], q.x, q.y);
          mma_f16(sc[n][1], f[1][0], f[1][1], f[1][2], f[1][3], q.z, q.w);
        }
      }
    }
    // ---- online softmax (log2 units) ----
    const float ks0 = st.ks[gq], ks1 = st.ks[gq + 8];
    float f0, f1, e0, e1;  // V scales f 2^e of keys gq, gq + 8
    split_scale(st.vs[gq], f0, e0);
    split_scale(st.vs[gq + 8], f1, e1);
    float z[NT][4];  // [e] key gq, [2 + e] key gq + 8, row 2tq + e
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        z[n][e] = seen0 ? (sc[n][0][e] + sc[n][1][e]) * (ks0 * rf[n][e]) : -INFINITY;
        z[n][2 + e] = seen1 ? (sc[n][0][2 + e] + sc[n][1][2 + e]) * (ks1 * rf[n][e]) : -INFINITY;
        over |= fmaxf(z[n][e] + e0, z[n][2 + e] + e1) > m_o[n][e] + kRangeO;
        over |= fmaxf(z[n][e], z[n][2 + e]) > m_l[n][e] + 60.f;
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float alpha[2] = {1.f, 1.f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ml = warp_key_max(fmaxf(z[n][e], z[n][2 + e]));
          const float mo = warp_key_max(fmaxf(z[n][e] + e0, z[n][2 + e] + e1));
          if (ml > m_l[n][e] + 60.f) {  // also when the row has no reference yet
            l_run[n][e] *= m_l[n][e] == -INFINITY ? 0.f : ex2f(m_l[n][e] - ml);
            m_l[n][e] = ml;
          }
          if (mo > m_o[n][e] + kRangeO) {
            alpha[e] = m_o[n][e] == -INFINITY ? 0.f : ex2f(m_o[n][e] - (mo - 7.f));
            m_o[n][e] = mo - 7.f;
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          o[n][c][0] *= alpha[0];
          o[n][c][1] *= alpha[1];
          o[n][c][2] *= alpha[0];
          o[n][c][3] *= alpha[1];
        }
      }
    }
    uint32_t pb[NT][PRECISE ? 2 : 1][2];  // P^T's B fragments: b0 = row gq at keys 2tq, 2tq + 1, b1 = at keys + 8
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float pw[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l_run[n][e] += (seen0 ? ex2f(z[n][e] - m_l[n][e]) : 0.f) + (seen1 ? ex2f(z[n][2 + e] - m_l[n][e]) : 0.f);
        pw[e] = seen0 ? ex2f(z[n][e] + e0 - m_o[n][e]) * f0 : 0.f;
        pw[2 + e] = seen1 ? ex2f(z[n][2 + e] + e1 - m_o[n][e]) * f1 : 0.f;
      }
      const uint32_t h0 = pack_half(pw[0], pw[1]), h1 = pack_half(pw[2], pw[3]);
      pb[n][0][0] = transpose_half(h0);
      pb[n][0][1] = transpose_half(h1);
      if (PRECISE) {
        const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
        const float2 g1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
        pb[n][PRECISE ? 1 : 0][0] = transpose_half(pack_half(pw[0] - g0.x, pw[1] - g0.y));
        pb[n][PRECISE ? 1 : 0][1] = transpose_half(pack_half(pw[2] - g1.x, pw[3] - g1.y));
      }
    }
    // ---- O^T += V^T P^T: 16 dims (one 16-byte piece) per product ----
    const uint32_t vbase = smem_u32(st.v) + ((lane & 15)) * kDq;  // row of this lane's ldmatrix address
#pragma unroll
    for (int c2 = 0; c2 < 4; ++c2) {
      uint32_t r0, r1, r2, r3;  // keys 0-7 / 8-15 of piece 2*c2, then of piece 2*c2 + 1
      ldsm_x4_trans(vbase + (((2 * c2 + (lane >> 4)) ^ (lane & 7)) << 4), r0, r1, r2, r3);
      const uint32_t rr[4] = {r0, r1, r2, r3};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t f0, f1, f2, f3;  // dims 2gq, 2gq + 1 of the piece (rows gq, gq + 8 of the operand)
        q8_to_half4(__byte_perm(rr[2 * u], 0u, 0x3120), f0, f1);
        q8_to_half4(__byte_perm(rr[2 * u + 1], 0u, 0x3120), f2, f3);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(o[n][2 * c2 + u], f0, f1, f2, f3, pb[n][0][0], pb[n][0][1]);
          if (PRECISE) mma_f16(o[n][2 * c2 + u], f0, f1, f2, f3, pb[n][PRECISE ? 1 : 0][0], pb[n][PRECISE ? 1 : 0][1]);
        }
      }
    }
  }
  cp_async_wait<0>();
  // the row sums over the 8 lanes that share each row
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float v = l_run[n][e];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      l_run[n][e] = v;
    }
  __syncthreads();  // every group is done with its ring (w shares its space)
  // ---- the key groups' (m, l, o / l) into the CTA's ----
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = n * 8 + 2 * tq + e;
      const float inv = l_run[n][e] == 0.f ? 0.f : 1.f / l_run[n][e];  // a NaN sum stays one
      // 2^(m_o - m_l) in two halves: it may pass a float's range where the result does not
      const float half_up = m_l[n][e] == -INFINITY ? 0.f : ex2f(0.5f * (m_o[n][e] - m_l[n][e]));
      const auto value = [&](float x) { return x * inv * half_up * half_up; };
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float2*>(&sm.w.o[warp][r][16 * c + 2 * gq]) =
            make_float2(value(o[n][c][e]), value(o[n][c][2 + e]));
      if (gq == 0) sm.ml[warp][r] = make_float2(m_l[n][e], l_run[n][e]);
    }
  __syncthreads();
  const int rows = min(kRows, a.R - row_base);
  if (tid < rows) {
    float M = -INFINITY, L = 0.f, f[kKW];
#pragma unroll
    for (int i = 0; i < kKW; ++i) M = fmaxf(M, sm.ml[i][tid].x);
#pragma unroll
    for (int i = 0; i < kKW; ++i) {
      const float2 ml = sm.ml[i][tid];
      f[i] = (ml.x == -INFINITY ? 0.f : ex2f(ml.x - M)) * ml.y;
      L += f[i];
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < kKW; ++i) sm.w.f[i][tid] = f[i] * inv;
    sm.ML[tid] = make_float2(M, L);
  }
  __syncthreads();
  auto store_out = [&](int r, int c, float4 v) {
    const int64_t off = sm.out_off[r] + c;
    if (a.out_f32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.O) + off) = v;
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.O) + off) =
          make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  };
  // what meets in the workspace: slices, or clusters of them (all of which
  // count there, with keys or without); a single one is the result
  const int sh = a.cluster ? 31 - __clz(a.cluster) : 0;
  const int n_parts = a.cluster ? a.n_split >> sh : n_live;
  const int part = slice >> sh;
  const int64_t part0 = (int64_t)unit * (a.cluster ? n_parts : a.n_split);
  auto store_part = [&](int r, int c, float4 v) {
    if (n_parts == 1)
      store_out(r, c, v);
    else
      __stcg(reinterpret_cast<float4*>(a.po + ((part0 + part) * kRows + r) * kDq + c), v);
  };
  for (int i = tid; i < rows * (kDq / 4); i += kThreadsQ) {
    const int r = i / (kDq / 4), c = i % (kDq / 4) * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kKW; ++j) {
      const float f = sm.w.f[j][r];
      const float4 v = *reinterpret_cast<const float4*>(&sm.w.o[j][r][c]);
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    if (a.cluster > 1)
      *reinterpret_cast<float4*>(&sm.w.o[0][r][c]) = acc;  // only this thread reads or writes it
    else
      store_part(r, c, acc);
  }
  if (a.cluster > 1) {
    // ---- the cluster's rows: this CTA merges every a.cluster-th 16 bytes of
    // them, a lane per CTA of the cluster.  (This runs once: what it costs is its
    // code's first fetch, so it is short.  Eight loads a thread took 1.7 us.)
    const int n = a.cluster, mine = slice & (n - 1), j = tid & (n - 1);
    cluster_sync();
    for (int base = 0; base < rows * (kDq / 4); base += kThreadsQ) {
      const int i = base + (tid & ~(n - 1)) + mine;
      const bool in = i < rows * (kDq / 4);
      const int r = in ? i / (kDq / 4) : 0, c = i % (kDq / 4) * 4;
      const float2 ml = ld_peer2(smem_u32(&sm.ML[r]), j);
      float4 v = ld_peer4(smem_u32(&sm.w.o[0][r][c]), j);
      float M = ml.x;
      for (int d = 1; d < n; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
      float L = (ml.x == -INFINITY ? 0.f : ex2f(ml.x - M)) * ml.y;
      v = make_float4(v.x * L, v.y * L, v.z * L, v.w * L);
#pragma unroll 1
      for (int d = 1; d < n; d <<= 1) {
        L += __shfl_xor_sync(0xffffffffu, L, d);
        v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, d);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
      }
      if (in && j == 0) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        store_part(r, c, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        if (c == 0 && n_parts > 1) __stcg(&a.pml[(part0 + part) * kRows + r], make_float2(M, L));
      }
    }
    cluster_sync();  // no CTA goes on while its rows are read
  } else if (tid < rows && n_parts > 1) {
    __stcg(&a.pml[(part0 + part) * kRows + tid], sm.ML[tid]);
  }
  if (n_parts == 1) return;
  // ---- count this CTA; the last one merges ----
  __threadfence();
  __syncthreads();
  if (tid == 0) sm.last = atomicAdd(&a.cnt[unit], 1u) == (unsigned)((a.cluster ? a.n_split : n_live) - 1);
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  for (int i = tid; i < n_parts * kRows; i += kThreadsQ)
    if (i % kRows < rows) (&sm.sml[0][0])[i] = __ldcg(&a.pml[part0 * kRows + i]);
  __syncthreads();
  for (int r = warp; r < rows; r += kWarpsQ) {
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < n_parts; i += 32) M = fmaxf(M, sm.sml[i][r].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    for (int i = lane; i < n_parts; i += 32) {
      const float2 ml = sm.sml[i][r];
      const float f = (ml.x == -INFINITY ? 0.f : ex2f(ml.x - M)) * ml.y;
      sm.sml[i][r].x = f;
      L += f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    if (lane == 0) sm.ML[r] = make_float2(M, L == 0.f ? 0.f : 1.f / L);
  }
  __syncthreads();
  for (int i = tid; i < rows * (kDq / 4); i += kThreadsQ) {
    const int r = i / (kDq / 4), c = i % (kDq / 4) * 4;
    const float* src = a.po + (part0 * kRows + r) * kDq + c;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < n_parts; ++j) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)j * kRows * kDq));
      const float f = sm.sml[j][r].x;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    const float inv = sm.ML[r].y;
    store_out(r, c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  if (tid == 0) a.cnt[unit] = 0;  // ready for the next launch on this workspace
}

template <int NT>
cudaError_t launch_nt(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream) {
  auto kern = a.out_f32 ? attn_q8_kernel<NT, true> : attn_q8_kernel<NT, false>;
  const size_t smem = sizeof(SmemQ<NT>);
  cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.units * p.n_split));
  cfg.blockDim = dim3(kThreadsQ);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster ? p.cluster : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, p.row_tiles);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {
constexpr int kRound = kKeysQ * kWarpsQ;  // keys a CTA takes per round of its warps

// How a unit's keys are split where all slices run at once: in one cluster of
// 1, 2, 4 or 8 CTAs, in several of 8, or one by one through the workspace.
// What counts is the rounds a CTA takes (about a microsecond each) and what
// the merge adds to them: a cluster's barrier and reads 1, a meeting in the
// workspace 2, and one CTA reading s partial results s / 16 more.
// (One head of 1500, 2500 and 4000 tokens: one cluster of 8 takes 7.2, 8.2 and
// 9.2 us, more slices through the workspace 9.1, 9.4 and 9.6.)
struct Split {
  int cluster = 1;       // CTAs of a cluster (0: none, every slice on its own)
  int64_t slices = 1;
  double cost = 1e30;
  int64_t rounds = 0;    // of a CTA
};

Split split_once(int64_t units, int64_t rounds, int sms, bool counters) {
  // whole clusters that run at once, two CTAs an SM: a GPC holds no parts of
  // one (33 of 8 and 71 of 4 CTAs on 148 SMs)
  const int64_t fit[4] = {2ll * sms, sms, 8ll * sms / 17, 2ll * sms / 9};
  Split best;
  auto offer = [&](int cluster, int64_t slices, double merge) {
    const int64_t r = (rounds + slices - 1) / slices;
    if ((double)r + merge < best.cost) best = {cluster, slices, (double)r + merge, r};
  };
  offer(1, 1, 0);
  for (int i = 1; i < 4; ++i)
    if (units <= fit[i] && rounds > 1 << (i - 1)) offer(1 << i, 1ll << i, 1);
  if (counters) {
    int64_t m = fit[3] / units;
    if (m > (rounds + 7) / 8) m = (rounds + 7) / 8;
    if (m > 1) offer(8, 8 * m, 3 + m / 16.0);
    int64_t one = fit[0] / units;
    if (one > rounds) one = rounds;
    if (one > 1) offer(0, one, 2 + one / 16.0);
  }
  return best;
}
}  // namespace

Q8AttnPlan plan_attn_q8(int R, int B, int Hkv, int64_t n_tokens, int S_max, int k, int sms, int max_counters) {
  Q8AttnPlan p;
  // keys of the longest unit (S_max may be a bound that bounds nothing)
  const int64_t n = k > 0 ? k : S_max < n_tokens ? S_max : n_tokens;
  const int64_t rounds = n > kRound ? (n + kRound - 1) / kRound : 1;
  const int64_t slots = 2ll * sms;      // CTAs the GPU holds at once
  // More than 16 rows: 16 a CTA, K and V read again for every 16, where all
  // CTAs run at once for two rounds at most; else tiles of 128 rows.  (20 rows
  // of 16 heads, 2048 keys: 13.8 and 22.7 us; 96 rows of 8 heads: 16.8 in
  // three rounds and 14.1.)
  const int64_t tiles16 = (R + 15) / 16;
  const int64_t units16 = B * (int64_t)Hkv * tiles16;
  Split split = split_once(units16, rounds, sms, units16 <= max_counters);
  p.group = R > 16 && (units16 > slots || split.rounds > 2);
  p.row_tiles = p.group ? (R + kQ8RowTile - 1) / kQ8RowTile : (int)tiles16;
  p.units = B * Hkv * p.row_tiles;
  if (p.group) {
    plan_attn_q8_group(p, n, sms);
    return p;
  }
  p.rows = R <= 8 ? 8 : 16;
  // Much work (from 2048 keys per slot): about four slices per slot, so that
  // ragged sequences and the last wave even out.  What counts is the keys there
  // can be, not the cache's places: a cache with room to grow may hold short
  // sequences.
  int64_t keys = B * n;
  if (k == 0 && keys > n_tokens) keys = n_tokens;
  keys *= (int64_t)Hkv * p.row_tiles;
  int64_t chunk = (n + split.slices - 1) / split.slices;
  if (keys >= slots * 2048) {
    split.cluster = 0;
    chunk = p.units > max_counters ? n : (keys + slots * 4 - 1) / (slots * 4);
  }
  const int most = q8_max_splits(p.rows);
  const int64_t least = split.cluster ? 0 : (n + most - 1) / most;
  if (chunk < least) chunk = least;
  chunk = (chunk + kRound - 1) / kRound * kRound;
  if (chunk < kRound) chunk = kRound;
  p.chunk = (int)chunk;
  p.cluster = split.cluster;
  p.n_split = p.cluster ? (int)split.slices : (int)((n + chunk - 1) / chunk);
  if (p.n_split < 1) p.n_split = 1;
  p.parts = p.cluster ? p.n_split / p.cluster : p.n_split;
  return p;
}

size_t attn_q8_scratch_bytes(const Q8AttnPlan& p) {
  if (p.parts <= 1) return 0;
  const size_t n = (size_t)p.units * p.parts * p.rows;
  return (n * kDq * 4 + 255) / 256 * 256 + (n * 8 + 255) / 256 * 256;
}

cudaError_t launch_attn_q8(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream) {
  if (p.group) return launch_attn_q8_group(a, p, stream);
  return p.rows == 8 ? launch_nt<1>(a, p, stream) : launch_nt<2>(a, p, stream);
}

}  // namespace sa
