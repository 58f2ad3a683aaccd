// Indexer scores over an 8-bit key cache (format in q8.cuh):
//   score[b,t] = sum_j w[b,j] max(0, q_j . K_t) = ks_t sum_j w[b,j] max(0, q_j . c_t)
// with c_t the token's codes and ks_t >= 0 its block's scale.
//
// HBM-bound: a key is d_I + 4/64 bytes in and 4 out, half of what bf16 keys
// need, for 2 H_I d_I flops.  The codes go from HBM to the tensor cores as they
// are: tcgen05 kind::f8f6f4 multiplies e4m3 by e4m3, so only the bf16 queries
// have to change.  Each query row is scaled by a power of two into (224, 448]
// and split into two e4m3 parts, hi + lo: a bf16 element has 8 significant
// bits and each part holds 4.  lo's smallest step is 2^-9, the last bit of an
// element of 2^-2, so the split is exact down to 2^-9 of the row's largest
// element (over all mantissas: down to 2^-9.8), and below it is off by less
// than 2^-17 of that element.
// Both parts are columns of one B operand, so a key tile is read from shared
// memory once for them; the epilogue adds the two columns of a head.
//
// Persistent CTAs take equal contiguous ranges of the ragged list of
// (sequence, 128-key tile) pairs, so that a CTA meets few sequences.  Warp 0
// issues TMA of key tiles into a ring, warp 1 the MMAs (M = 128 keys, N = two
// parts of H_I heads padded to a multiple of 8, K = 32 per instruction) into
// one of several TMEM accumulators, warps 2-5 apply ReLU, weights and the key
// scale and store one score per thread, warps 6-7 split the next sequence's
// queries into one of two buffers while the tiles of the last one run.  Two
// CTAs share an SM where each still has four stages: a tile passes TMA, MMA
// and epilogue one after another, and a second chain fills the gaps (32 ragged
// sequences of 8192 .. 131072: 90, 54 and 61 us with 1, 2 and 3 CTAs an SM).
//
// Measured (B200, warm graph replay, 16 heads of 128): those 32 sequences 54 us
// = 84 % of the measured HBM rate, 4 x 131072 keys 17.0 us; one sequence of 4096
// keys, 4 heads of 64, 3.5 us.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "q8.cuh"
#include "sm100.cuh"
#include "status.cuh"

namespace sa {
namespace {

constexpr int kTile = 128;
constexpr int kMaxAcc = 4;
constexpr int kThreadsI = 256;
constexpr int kMaxStagesI = 8;
constexpr int kSmemMaxI = 232448;   // of a CTA alone on its SM
constexpr int kSmemHalfI = 115712;  // of each of two

// instruction descriptor, kind::f8f6f4: e4m3 A and B (both K-major), fp32 accumulate
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// shared memory: barriers | tmem slot | weights of two query buffers |
// prefix[B+1] | (1024-aligned) two query buffers | ring
constexpr int kBarBytes = 8 * (2 * kMaxStagesI + 2 * kMaxAcc + 4);
constexpr int kSlotOffset = kBarBytes;
constexpr int kWOffset = kSlotOffset + 16;

template <int NH, int NPAD>  // 128-byte halves of a key row, padded heads
struct LayoutI {
  static constexpr int kCols = 2 * NPAD;              // of one accumulator
  static constexpr int kAcc = kCols <= 64 ? 4 : 2;
  static constexpr int kTmemCols = kAcc * kCols <= 64 ? 64 : kAcc * kCols <= 128 ? 128 : 256;
  static constexpr int kStageBytes = NH * kTile * 128;
  static constexpr int kQHalf = kCols * 128;          // [hi heads | lo heads] x 128 bytes
  static constexpr int kQBytes = NH * kQHalf;
  static constexpr int kPrefixOffset = kWOffset + 2 * NPAD * 4;
  static int q_offset(int B) { return (kPrefixOffset + 4 * (B + 1) + 1023) / 1024 * 1024; }
  static int stages(int B, int smem) {
    const int n = (smem - 1024 - q_offset(B) - 2 * kQBytes) / kStageBytes;
    return n > kMaxStagesI ? kMaxStagesI : n;
  }
  static size_t smem_bytes(int B, int n_st) {
    return 1024 + (size_t)q_offset(B) + 2 * kQBytes + (size_t)n_st * kStageBytes;
  }
};

// largest b with prefix[b] <= t (prefix[0] = 0, prefix[B] > t)
__device__ __forceinline__ int tile_sequence(const int* prefix, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int NH, int NPAD>
__global__ void __launch_bounds__(kThreadsI, 2)
indexer_q8_kernel(const __grid_constant__ CUtensorMap tm_ki, const Q8IndexerArgs a, int n_st, int q_off) {
  using Lay = LayoutI<NH, NPAD>;
  constexpr int kAcc = Lay::kAcc;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded address: the compiler then knows it for shared
  // memory; generic loads would queue behind the global ones)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kMaxStagesI;
  uint64_t* tfull = empty + kMaxStagesI;
  uint64_t* tempty = tfull + kMaxAcc;
  uint64_t* qfull = tempty + kMaxAcc;
  uint64_t* qempty = qfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOffset);
  float* wq = reinterpret_cast<float*>(smem + kWOffset);  // [2][NPAD]: w times the query scale's inverse
  int* prefix = reinterpret_cast<int*>(smem + Lay::kPrefixOffset);
  uint8_t* qbuf = smem + q_off;
  uint8_t* ring = qbuf + 2 * Lay::kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ksteps = a.d_I / 32;

  pdl_trigger();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < n_st; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int c = 0; c < kAcc; ++c) { mbar_init(&tfull[c], 1); mbar_init(&tempty[c], 4); }
    // a query buffer is free once its MMAs are done and the four epilogue warps have passed its tiles
    for (int c = 0; c < 2; ++c) { mbar_init(&qfull[c], 2); mbar_init(&qempty[c], 5); }
    fence_mbar_init();
    tma_prefetch_desc(&tm_ki);
  } else if (warp == 1) {
    tmem_alloc(tmem_slot, Lay::kTmemCols);
  }
  pdl_wait();
  if (warp == 0) {
    // prefix[b] = tiles of the sequences before b
    int carry = 0;
    for (int base = 0; base < a.B; base += 32) {
      const int b = base + lane;
      int n = 0;
      if (b < a.B) {
        const Q8Seq s = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
        if (!s.ok && blockIdx.x == 0) report(a.status, kErrDevice, kKernIndexerQ8, b, a.seq_len[b], a.S_max);
        n = q8_tiles(s.len, kTile);
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (b < a.B) prefix[b] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[a.B] = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // this CTA's tiles [g_beg, g_end), and the sequence of the first
  const int total = prefix[a.B];
  const int g_beg = (int)((int64_t)total * blockIdx.x / gridDim.x);
  const int g_end = (int)((int64_t)total * (blockIdx.x + 1) / gridDim.x);
  int b = g_beg < g_end ? tile_sequence(prefix, a.B, g_beg) : 0;

  if (warp == 0) {
    // ---------------- key tiles ----------------
    if (lane == 0) {
      // (stages are counted, not divided for: a division takes as long as the rest of a turn)
      int st = 0, issued = 0;
      uint32_t phase = 1;  // of the stage's `empty` that frees it: passed at once on the first turn
      int64_t off = g_beg < g_end ? a.seq_off[b] : 0;
      for (int g = g_beg; g < g_end; ++g) {
        if (g >= prefix[b + 1]) {
          do ++b; while (g >= prefix[b + 1]);
          off = a.seq_off[b];
        }
        if (!mbar_wait(&empty[st], phase, kWaitLimitNs)) {
          report(a.status, kErrTimeout, kKernIndexerQ8, blockIdx.x, 0, g);
          break;
        }
        const int64_t row = off + (int64_t)(g - prefix[b]) * kTile;
        mbar_arrive_expect_tx(&full[st], Lay::kStageBytes);
#pragma unroll
        for (int h = 0; h < NH; ++h)
          tma_load_2d(ring + st * Lay::kStageBytes + h * kTile * 128, &tm_ki, &full[st], h * 128, (int)row);
        ++issued;
        if (++st == n_st) st = 0, phase ^= 1;
      }
      // drain: every load issued by this thread has landed before the CTA exits
      for (int k = 0; k < n_st && k < issued; ++k) {
        if (--st < 0) st = n_st - 1, phase ^= 1;
        mbar_wait(&full[st], phase ^ 1, kWaitLimitNs);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    // the warp stays together and one elected lane issues: a product's operands
    // are then known to be one value per warp
    const bool lead = elect_one();
    auto wait = [](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitLimitNs));
    };
    constexpr uint32_t idesc = idesc_e4m3(128, Lay::kCols);
    const uint64_t a0 = umma_desc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t b0 = umma_desc_sw128(smem_u32(qbuf), 16, 1024);
    int st = 0, nseq = 0;
    uint32_t phase = 0;
    int next = g_beg;  // first tile of the next sequence
    for (int g = g_beg, i = 0; g < g_end; ++g, ++i) {
      const int c = i % kAcc;
      bool ok = true;
      if (g == next) {
        while (g >= prefix[b + 1]) ++b;
        next = prefix[b + 1];
        if (nseq > 0 && lead) umma_commit(&qempty[(nseq - 1) & 1]);  // the last sequence's products
        ok = wait(&qfull[nseq & 1], (nseq >> 1) & 1);
        ++nseq;
      }
      if (!ok || !wait(&full[st], phase) || !wait(&tempty[c], ((i / kAcc) & 1) ^ 1)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernIndexerQ8, blockIdx.x, 1, i);
        break;
      }
      tc_fence_after();
      // descriptors count 16-byte units
      const uint64_t ad = a0 + (uint32_t)(st * (Lay::kStageBytes / 16));
      const uint64_t bd = b0 + ((nseq - 1) & 1) * (uint32_t)(Lay::kQBytes / 16);
      const uint32_t d = tmem_base + c * Lay::kCols;
      if (lead) {
#pragma unroll
        for (int k = 0; k < NH * 4; ++k) {
          if (k >= ksteps) break;
          const int h = k / 4, kk = k % 4;
          umma_e4m3(d, ad + h * (kTile * 128 / 16) + kk * 2, bd + h * (Lay::kQHalf / 16) + kk * 2, idesc, k != 0);
        }
        umma_commit(&empty[st]);
        umma_commit(&tfull[c]);
      }
      __syncwarp();
      if (++st == n_st) st = 0, phase ^= 1;
    }
  } else if (warp < 6) {
    // ---------------- epilogue: ReLU, head weights, sum, key scale ----------------
    const int quarter = warp & 3;  // TMEM lanes this warp may read
    const int r = quarter * 32 + lane;
    int nseq = 0;
    bool fresh = true;
    Q8Seq seq = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
    // scale of this thread's key of tile g of the sequence: loaded a tile ahead
    // (unsigned: the tile ahead of a sequence's last may start at 2^31)
    auto key_scale = [&](uint32_t t) {
      return t < (uint32_t)seq.len ? __ldcg(&a.scales[(seq.off + t) / kQ8Block]) : 0.f;
    };
    float ks = g_beg < g_end ? key_scale((g_beg - prefix[b]) * kTile + r) : 0.f;
    for (int g = g_beg, i = 0; g < g_end; ++g, ++i) {
      const int c = i % kAcc;
      bool ok = true;
      if (g >= prefix[b + 1]) {
        do ++b; while (g >= prefix[b + 1]);
        seq = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
        ks = key_scale((g - prefix[b]) * kTile + r);
        fresh = true;
      }
      const int t = (g - prefix[b]) * kTile + r;
      const float ks_next = key_scale((uint32_t)t + kTile);
      if (lane == 0) {
        if (fresh) {
          if (nseq > 0) mbar_arrive(&qempty[(nseq - 1) & 1]);
          ok = mbar_wait(&qfull[nseq & 1], (nseq >> 1) & 1, kWaitLimitNs);
        }
        if (ok) ok = mbar_wait(&tfull[c], (i / kAcc) & 1, kWaitLimitNs);
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernIndexerQ8, blockIdx.x, 2, i);
        break;
      }
      if (fresh) ++nseq;
      fresh = false;
      tc_fence_after();
      const float* w = wq + ((nseq - 1) & 1) * NPAD;
      const uint32_t acc_col = tmem_base + ((uint32_t)(quarter * 32) << 16) + c * Lay::kCols;
      float acc = 0.f;
#pragma unroll 1  // 16 heads at a time: more would spill
      for (int j0 = 0; j0 < NPAD; j0 += 16) {
        uint32_t v[32];  // 16 heads of the hi part, then of the lo part (or 8 of each)
        tmem_ld16(acc_col + j0, v);
        if (NPAD > 8) tmem_ld16(acc_col + NPAD + j0, v + 16);
        tmem_wait_ld();
        constexpr int kN = NPAD > 8 ? 16 : 8;
#pragma unroll
        for (int j = 0; j < kN; j += 4) {
          const float4 wj = *reinterpret_cast<const float4*>(w + j0 + j);
          const float ww[4] = {wj.x, wj.y, wj.z, wj.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            acc = fmaf(ww[u], fmaxf(__uint_as_float(v[j + u]) + __uint_as_float(v[kN + j + u]), 0.f), acc);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[c]);
      if (t < seq.len) a.scores[(int64_t)b * a.ld + t] = __fadd_rn(acc * ks, 0.f);  // canonical +0
      ks = ks_next;
    }
  } else {
    // ---------------- queries: scale, split, swizzled K-major tiles ----------------
    int nseq = 0;
    for (; g_beg < g_end && b < a.B && prefix[b] < g_end; ++b) {
      if (prefix[b + 1] <= g_beg || prefix[b + 1] == prefix[b]) continue;  // no tiles here
      bool ok = true;
      if (lane == 0) ok = mbar_wait(&qempty[nseq & 1], ((nseq >> 1) & 1) ^ 1, kWaitLimitNs);
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernIndexerQ8, blockIdx.x, 3, nseq);
        break;
      }
      uint8_t* hi = qbuf + (nseq & 1) * Lay::kQBytes;
      uint8_t* lo = hi + NPAD * 128;
      // four heads at a time, 8 lanes a head, 16 dims (one 16-byte chunk of codes) a lane
      const int ch = lane & 7;
#pragma unroll 2
      for (int j = (warp - 6) * 4 + (lane >> 3); j < NPAD; j += 8) {
        // a padding head is zero: its columns add nothing
        const uint16_t* q = a.qI + ((int64_t)b * a.H_I + j) * a.d_I;
        uint4 v[NH][2];
        uint32_t mx = 0;  // largest |element|, as bf16 bits (ordered like the values)
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const bool in = j < a.H_I && h * 128 + ch * 16 < a.d_I;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            v[h][u] = in ? __ldcg(reinterpret_cast<const uint4*>(q + h * 128 + ch * 16) + u) : make_uint4(0, 0, 0, 0);
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[h][u].x & 0x7fff7fffu, v[h][u].y & 0x7fff7fffu),
                                       __vmaxu2(v[h][u].z & 0x7fff7fffu, v[h][u].w & 0x7fff7fffu)));
          }
        }
        const float wj = j < a.H_I ? __ldcg(&a.w[(int64_t)b * a.H_I + j]) : 0.f;
        mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const uint32_t sb = mx >= 0x7f80u ? 0x3f800000u : q8_scale_bits(mx << 16);
        const float inv = 1.f / __uint_as_float(sb);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint32_t w[8] = {v[h][0].x, v[h][0].y, v[h][0].z, v[h][0].w, v[h][1].x, v[h][1].y, v[h][1].z, v[h][1].w};
          uint32_t ch_hi[4], ch_lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float y0 = __uint_as_float(w[2 * u] << 16) * inv, y1 = __uint_as_float(w[2 * u] & 0xffff0000u) * inv;
            const float y2 = __uint_as_float(w[2 * u + 1] << 16) * inv;
            const float y3 = __uint_as_float(w[2 * u + 1] & 0xffff0000u) * inv;
            ch_hi[u] = q8_from_float4(y0, y1, y2, y3);
            uint32_t p0, p1;
            q8_to_half4(ch_hi[u], p0, p1);
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&p0));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&p1));
            ch_lo[u] = q8_from_float4(y0 - f0.x, y1 - f0.y, y2 - f1.x, y3 - f1.y);
          }
          const uint32_t to = h * Lay::kQHalf + sw128_offset(j, ch);
          *reinterpret_cast<uint4*>(hi + to) = make_uint4(ch_hi[0], ch_hi[1], ch_hi[2], ch_hi[3]);
          *reinterpret_cast<uint4*>(lo + to) = make_uint4(ch_lo[0], ch_lo[1], ch_lo[2], ch_lo[3]);
        }
        if (ch == 0) wq[(nseq & 1) * NPAD + j] = wj * __uint_as_float(sb);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&qfull[nseq & 1]);
      ++nseq;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Lay::kTmemCols);
  }
}

template <int NH, int NPAD>
cudaError_t launch_nh(const Q8IndexerArgs& a, const CUtensorMap& tm_ki, int num_sms, cudaStream_t stream) {
  using Lay = LayoutI<NH, NPAD>;
  auto kern = indexer_q8_kernel<NH, NPAD>;
  // two CTAs an SM where each has four stages or more, else one with all there is
  const int half = Lay::stages(a.B, kSmemHalfI);
  const int per_sm = half >= 4 ? 2 : 1;
  const int n_st = per_sm == 2 ? half : Lay::stages(a.B, kSmemMaxI);
  if (n_st < 2) return cudaErrorInvalidValue;  // the prefix table would crowd out the ring
  const size_t smem = Lay::smem_bytes(a.B, n_st);
  cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)a.B * q8_tiles(a.S_max, kTile);
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (int64_t)num_sms * per_sm;
  cfg.gridDim = dim3((unsigned)(tiles < ctas ? tiles : ctas));
  cfg.blockDim = dim3(kThreadsI);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm_ki, a, n_st, Lay::q_offset(a.B));
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_indexer_q8(const Q8IndexerArgs& a, const CUtensorMap& tm_ki, int num_sms, cudaStream_t stream) {
  const int nh = (a.d_I + 127) / 128, npad = a.H_I <= 8 ? 8 : (a.H_I + 15) / 16 * 16;
#define SA_IDX_CASE(NH, NP) \
  if (nh == NH && npad == NP) return launch_nh<NH, NP>(a, tm_ki, num_sms, stream);
  SA_IDX_CASE(1, 8) SA_IDX_CASE(2, 8)
  SA_IDX_CASE(1, 16) SA_IDX_CASE(1, 32) SA_IDX_CASE(1, 48) SA_IDX_CASE(1, 64)
  SA_IDX_CASE(2, 16) SA_IDX_CASE(2, 32) SA_IDX_CASE(2, 48) SA_IDX_CASE(2, 64)
#undef SA_IDX_CASE
  return cudaErrorInvalidValue;
}

}  // namespace sa
