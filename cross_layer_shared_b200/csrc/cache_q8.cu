// Writing tokens into the 8-bit cache (format in q8.cuh) and reading them
// back.  Both are one pass over their data: HBM-bound for many tokens,
// launch-latency-bound for a decode step's single tokens.
//
// Append.  Sequence b's n_b new tokens go to places seq_len[b] - n_b ..
// seq_len[b] - 1.  One CTA per (sequence, touched block of 64 tokens, head,
// tensor): it holds the block's new rows in registers from the one time they
// are read, reduces max|x|, picks the block's scale and stores the codes.  A
// block that already holds tokens keeps its scale unless the new ones need a
// larger one; then the CTA also moves the old codes to it.
//
// Consecutive CTAs take the heads of one block: a token's row of heads is one
// piece of memory, and heads read far apart in time cost DRAM pages.
//
// A CTA's block is (blockIdx.y's sequence, block blockIdx.x / units behind its
// first new token) where the sequences' counts are alike.  Ragged counts would
// leave many such CTAs without work, each a place on the GPU for the time of a
// load (16 prompts of 517 .. 16384 tokens: half of them, 20 of 165 us); there
// the touched blocks are numbered through, and each warp finds its CTA's block
// by a scan over the sequences, 32 at a time.
//
// Measured (B200, warm graph replay): those 16 prompts, fp32, 4 heads of 128, K
// and V, 124 us = 85 % of the measured HBM rate; 2048 bf16 tokens of 8 heads
// 6.1 us; one token of 4 sequences 2.4 us.  Reading 131009 tokens of 8 heads
// back as bf16 takes 121.7 us = the measured HBM rate.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "q8.cuh"
#include "sm100.cuh"
#include "status.cuh"

namespace sa {
namespace {

constexpr int kThreadsC = 256;

// 8 elements of a row as floats; kept raw until they are used.  New rows are
// read once: marked so, they leave the L2 to the codes (16 fp32 prompts
// 145 -> 122 us).
template <bool F32>
struct Raw8;
template <>
struct Raw8<false> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  // largest |element| as bits, infinities and NaN included: pairs compared as integers
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
};
template <>
struct Raw8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float get(int i) const {
    const float4& q = i < 4 ? a : b;
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(get(i)) & 0x7fffffffu);
    return m;
  }
};

struct NewTokens {  // of one sequence; n = 0 when it has none or is not as described
  Q8Seq s;
  int64_t src0;   // first row
  int n, first;   // count, and the first touched block
  __device__ __forceinline__ int blocks() const { return n == 0 ? 0 : (s.len - 1) / kQ8Block - first + 1; }
};

__device__ __forceinline__ NewTokens new_tokens(const Q8AppendArgs& a, int b, bool rep) {
  NewTokens t;
  t.s = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, 0x7fffffff);
  t.src0 = a.new_off ? __ldcg(reinterpret_cast<const long long*>(a.new_off) + b) : b;
  const int64_t src1 = a.new_off ? __ldcg(reinterpret_cast<const long long*>(a.new_off) + b + 1) : b + 1;
  const int64_t n = src1 - t.src0;
  const bool ok = t.s.ok && n >= 0 && n <= t.s.len && n <= a.max_new && t.src0 >= 0 && src1 <= a.n_rows;
  if (!ok && rep) report(a.status, kErrDevice, kKernCacheQ8, b, t.s.ok ? n : -1, t.s.len);
  t.n = ok ? (int)n : 0;
  t.first = (t.s.len - t.n) / kQ8Block;
  return t;
}

// (tensor, head) units a CTA takes at once, with much to do: as many as make
// 128 bytes a thread in flight
template <bool F32, int D>
constexpr int kUnits = 128 / (kQ8Block * D / kThreadsC * (F32 ? 4 : 2)) > 1
                           ? 128 / (kQ8Block * D / kThreadsC * (F32 ? 4 : 2))
                           : 1;

// registers for as many CTAs an SM as hold what the memory needs in flight
template <bool F32, int D, int U>
constexpr int kAppendCtas = kQ8Block * D / kThreadsC * (F32 ? 4 : 2) * U < 96    ? 1
                            : kQ8Block * D / kThreadsC * (F32 ? 4 : 2) * U <= 128 ? 4
                            : D == 192                                            ? 3
                                                                                  : 2;

template <bool F32, int D, bool FLAT, int U>
__global__ void __launch_bounds__(kThreadsC, kAppendCtas<F32, D, U>) cache_append_q8_kernel(const Q8AppendArgs a) {
  constexpr int kPieces = D / 8;                           // 8-element pieces of a row
  constexpr int kPer = kQ8Block * kPieces / kThreadsC;     // pieces a thread holds
  __shared__ uint32_t warp_max[U][kThreadsC / 32];
  const int tid = threadIdx.x;
  const int units = a.Hkv * (a.cache.codes[1] ? 2 : 1);  // (tensor, head)
  const int groups = (units + U - 1) / U;
  const int unit0 = blockIdx.x % groups * U;
  pdl_trigger();
  pdl_wait();
  NewTokens nt;
  int blk = blockIdx.x / groups;  // block behind the sequence's first touched one
  if (FLAT) {
    const int lane = tid & 31;
    // one CTA more than there can be blocks: it meets every sequence
    const bool rep = blockIdx.x == gridDim.x - 1 && tid < 32;
    bool found = false;
    for (int base = 0; base < a.B && !found; base += 32) {
      int cnt = 0;
      if (base + lane < a.B) {
        nt = new_tokens(a, base + lane, rep);
        cnt = nt.blocks();
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > blk);
      if (past) {
        const int l = __ffs(past) - 1;
        blk -= __shfl_sync(0xffffffffu, incl - cnt, l);
        nt.s.off = __shfl_sync(0xffffffffu, nt.s.off, l);
        nt.s.cap = __shfl_sync(0xffffffffu, nt.s.cap, l);
        nt.s.len = __shfl_sync(0xffffffffu, nt.s.len, l);
        nt.src0 = __shfl_sync(0xffffffffu, nt.src0, l);
        nt.n = __shfl_sync(0xffffffffu, nt.n, l);
        nt.first = __shfl_sync(0xffffffffu, nt.first, l);
        found = true;
      } else {
        blk -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (!found) return;
  } else {
    nt = new_tokens(a, blockIdx.y, tid == 0 && blockIdx.x == 0);
    if (blk >= nt.blocks()) return;
  }
  const Q8Seq& s = nt.s;
  const int64_t src0 = nt.src0;
  const int pos0 = s.len - nt.n;
  const int t0 = (nt.first + blk) * kQ8Block;  // the block's first token
  const int lo = max(pos0 - t0, 0), hi = min(s.len - t0, kQ8Block);  // new tokens [lo, hi) of the block
  constexpr int kElem = F32 ? 4 : 2;
  Raw8<F32> x[U][kPer];
  uint32_t old_bits[U];  // of the scale of the tokens already there (0: none, or not a positive scale)
  auto first_row = [&](int h) { return s.off * a.Hkv + (int64_t)h * s.cap + t0; };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int unit = unit0 + u, which = unit >= a.Hkv, h = unit - which * a.Hkv;
    old_bits[u] = 0;
    if (lo > 0 && unit < units) {
      const float old = __ldcg(a.cache.scales[which] + first_row(h) / kQ8Block);
      if (old > 0.f && old < INFINITY) old_bits[u] = __float_as_uint(old);
    }
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.rows[which]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreadsC) / kPieces, p = (tid + i * kThreadsC) % kPieces;
      if (r >= lo && r < hi && unit < units)
        x[u][i].load(src + ((src0 + (t0 + r - pos0)) * a.stride[which] + (int64_t)h * D + p * 8) * kElem);
      else
        x[u][i].clear();
    }
  }
  // max|x| over the finite values, as bits (ordered like the floats)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mx = max(mx, x[u][i].largest());
    if (mx >= 0x7f800000u) {  // an infinity or NaN among them
      mx = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t v = __float_as_uint(x[u][i].get(j)) & 0x7fffffffu;
          mx = max(mx, v < 0x7f800000u ? v : 0u);
        }
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((tid & 31) == 0) warp_max[u][tid >> 5] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int unit = unit0 + u, which = unit >= a.Hkv, h = unit - which * a.Hkv;
    if (unit >= units) return;
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kThreadsC / 32; ++i) mx = max(mx, warp_max[u][i]);
    const uint32_t bits = max(q8_scale_bits(mx), old_bits[u]);
    // exact for a power of two; a kept scale from elsewhere need not be one, and
    // then this and the products below round once each, 2^-24 beside a code's 2^-4
    const float inv = 1.f / __uint_as_float(bits);
    const int64_t row0 = first_row(h);
    uint8_t* dst = a.cache.codes[which] + row0 * D;
    const bool move = lo > 0 && bits != old_bits[u];  // the tokens already there go to the larger scale
    const float ratio = move ? __uint_as_float(old_bits[u]) * inv : 1.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreadsC) / kPieces, p = (tid + i * kThreadsC) % kPieces;
      uint2* out = reinterpret_cast<uint2*>(dst + r * D + p * 8);
      if (r >= lo && r < hi) {
        const Raw8<F32>& v = x[u][i];
        *out = make_uint2(q8_from_float4(v.get(0) * inv, v.get(1) * inv, v.get(2) * inv, v.get(3) * inv),
                          q8_from_float4(v.get(4) * inv, v.get(5) * inv, v.get(6) * inv, v.get(7) * inv));
      } else if (r < lo && move) {
        const uint2 c = *out;
        uint32_t q[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t l, u2;
          q8_to_half4(q[j], l, u2);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&l));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&u2));
          q[j] = q8_from_float4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio);
        }
        *out = make_uint2(q[0], q[1]);
      }
    }
    if (tid == 0 && bits != old_bits[u]) a.cache.scales[which][row0 / kQ8Block] = __uint_as_float(bits);
  }
}

// ---------------------------------------------------------------- reading back
// A thread takes kReadPer pieces of 16 codes, all their loads before the first
// conversion: 16 bytes in, 32 (bf16) or 64 (fp32) out, in whole 32-byte
// sectors.  A CTA takes kReadPieces consecutive pieces of one (sequence, head,
// tensor), so the split needs no whole rows.  A code times its scale is exact
// in fp32; bf16 rounds it only below 2^-133.  Pieces a thread, for 131009 tokens
// x 8 heads of K and V (806 MB) and for 131072 picked rows (51 MB): 2 take 185
// and 15.1 us, 4 take 129 and 11.6, 6 take 121 and 10.9, 8 take 124 and 11.9.
constexpr int kReadPer = 6;
constexpr int kReadPieces = kReadPer * kThreadsC;

__device__ __forceinline__ void store32(void* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {  // an output that starts between two sectors
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

template <bool F32, int D>
__global__ void __launch_bounds__(kThreadsC) cache_read_q8_kernel(const Q8ReadArgs a) {
  constexpr int kPieces = D / 16;
  const int tid = threadIdx.x;
  const int b = blockIdx.z, h = blockIdx.y % a.Hkv, which = blockIdx.y / a.Hkv;
  pdl_trigger();
  pdl_wait();
  const Q8Seq s = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
  const bool first = tid == 0 && blockIdx.x == 0 && blockIdx.y == 0;
  if (!s.ok && first) report(a.status, kErrDevice, kKernCacheQ8, b, s.len, s.cap);
  const int64_t row0 = s.off * a.Hkv + (int64_t)h * s.cap;
  int n;           // entries of this sequence
  int64_t out0;    // its first output row for this head
  if (a.idx) {
    n = a.k;
    out0 = ((int64_t)b * a.Hkv + h) * a.k;
  } else {
    n = s.len;
    const int64_t o = __ldcg(reinterpret_cast<const long long*>(a.out_off) + b);
    const int64_t o1 = __ldcg(reinterpret_cast<const long long*>(a.out_off) + b + 1);
    if (o < 0 || o1 > a.n_out || o1 - o != s.len) {
      if (first && s.ok) report(a.status, kErrDevice, kKernCacheQ8, b, o1 - o, s.len);
      return;
    }
    out0 = o * a.Hkv + (int64_t)h * s.len;
  }
  const int64_t base = (int64_t)blockIdx.x * kReadPieces;
  const int64_t e_base = base / kPieces;
  const int rem = (int)(base % kPieces);
  const uint8_t* codes = a.cache.codes[which];
  const float* scales = a.cache.scales[which];
  int e[kReadPer], t[kReadPer];  // entry, token (-1: zeros)
#pragma unroll
  for (int i = 0; i < kReadPer; ++i) {
    const int64_t at = e_base + (rem + tid + i * kThreadsC) / kPieces;
    e[i] = at < n ? (int)at : -1;
    t[i] = e[i];
    if (a.idx && e[i] >= 0) t[i] = __ldcg(&a.idx[(int64_t)b * a.k + e[i]]);
  }
  uint4 c[kReadPer];
  float sc[kReadPer];
#pragma unroll
  for (int i = 0; i < kReadPer; ++i) {
    const int p = (rem + tid + i * kThreadsC) % kPieces;
    if (t[i] >= s.len) {
      if (p == 0 && blockIdx.y == 0)
        report(a.status, kErrDevice, kKernCacheQ8, (int64_t)b * a.k + e[i], t[i], s.len);
      t[i] = -1;
    }
    c[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.f;
    if (t[i] >= 0) {
      c[i] = __ldcg(reinterpret_cast<const uint4*>(codes + (row0 + t[i]) * D + p * 16));
      sc[i] = __ldcg(scales + (row0 + t[i]) / kQ8Block);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadPer; ++i) {
    if (e[i] < 0) continue;
    const int p = (rem + tid + i * kThreadsC) % kPieces;
    const uint32_t q[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    const int64_t at = (out0 + e[i]) * D + p * 16;
    uint32_t w[F32 ? 16 : 8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t l, u;
      q8_to_half4(q[j], l, u);
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&l));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&u));
      const float v[4] = {f0.x * sc[i], f0.y * sc[i], f1.x * sc[i], f1.y * sc[i]};
      if (F32) {
#pragma unroll
        for (int x = 0; x < 4; ++x) w[4 * j + x] = __float_as_uint(v[x]);
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[2 * j + x]) : "f"(v[2 * x + 1]), "f"(v[2 * x]));
      }
    }
    if (F32) {
      float* o = reinterpret_cast<float*>(a.out[which]) + at;
      store32(o, w, a.out_wide);
      store32(o + 8, w + (F32 ? 8 : 0), a.out_wide);
    } else {
      store32(reinterpret_cast<uint16_t*>(a.out[which]) + at, w, a.out_wide);
    }
  }
}

template <typename Kernel, typename Args>
cudaError_t launch_grid(Kernel kern, const Args& a, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreadsC);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool F32, int D>
cudaError_t launch_append(const Q8AppendArgs& a, int num_sms, cudaStream_t stream) {
  // blocks a sequence's new tokens can touch: one more than full blocks when they start inside one
  const int64_t blocks = ((int64_t)a.max_new + kQ8Block - 2) / kQ8Block + 1;
  // and all of them together: less than two more than full blocks each
  const int64_t all = a.n_rows / kQ8Block + 2ll * a.B + 1;
  const int units = a.Hkv * (a.cache.codes[1] ? 2 : 1);
  const bool flat = blocks * a.B > all + all / 4;
  constexpr int U = kUnits<F32, D>;
  // several units a CTA from two waves on: a CTA's fixed second half of its
  // time (place, reduction, launch) then moves more bytes (22 sequences of
  // 1107 .. 2215 bf16 tokens, 4 heads of 128: 32 us, 37 with one)
  const bool many = U > 1 && units > 1 && (flat ? all : blocks * a.B) * units > 12ll * num_sms;
  const int groups = many ? (units + U - 1) / U : units;
  const dim3 grid((unsigned)((flat ? all : blocks) * groups), flat ? 1 : a.B);
  if (many)
    return flat ? launch_grid(cache_append_q8_kernel<F32, D, true, U>, a, grid, stream)
                : launch_grid(cache_append_q8_kernel<F32, D, false, U>, a, grid, stream);
  return flat ? launch_grid(cache_append_q8_kernel<F32, D, true, 1>, a, grid, stream)
              : launch_grid(cache_append_q8_kernel<F32, D, false, 1>, a, grid, stream);
}

}  // namespace

cudaError_t launch_cache_append_q8(const Q8AppendArgs& a, int num_sms, cudaStream_t stream) {
#define SA_APPEND_CASE(DD) \
  if (a.d == DD) return a.in_f32 ? launch_append<true, DD>(a, num_sms, stream) : launch_append<false, DD>(a, num_sms, stream);
  SA_APPEND_CASE(64) SA_APPEND_CASE(128) SA_APPEND_CASE(192) SA_APPEND_CASE(256)
#undef SA_APPEND_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_cache_read_q8(const Q8ReadArgs& a, cudaStream_t stream) {
  const int64_t pieces = (int64_t)(a.idx ? a.k : a.S_max) * (a.d / 16);
  const dim3 grid((unsigned)((pieces + kReadPieces - 1) / kReadPieces), a.Hkv * (a.out[1] ? 2 : 1), a.B);
#define SA_READ_CASE(DD)                                                                     \
  if (a.d == DD)                                                                             \
    return a.out_f32 ? launch_grid(cache_read_q8_kernel<true, DD>, a, grid, stream)          \
                     : launch_grid(cache_read_q8_kernel<false, DD>, a, grid, stream);
  SA_READ_CASE(64) SA_READ_CASE(128) SA_READ_CASE(192) SA_READ_CASE(256)
#undef SA_READ_CASE
  return cudaErrorInvalidValue;
}

}  // namespace sa
