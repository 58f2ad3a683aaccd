// Decode attention over the 8-bit cache for many query rows per KV head (the
// layers of a group that share an index, or many heads): the operator of
// attn_q8.cu on tcgen05 tiles of 128 query rows x 128 keys.
//
// What bounds it: with R rows a (token, KV head) costs 256 + 8/64 bytes and
// 512 R flops.  From about 16 rows the warp-level MMAs of attn_q8.cu, whose
// warps each convert all codes they multiply, are issue-bound; here each code
// is converted once per 128 rows and the products run on tcgen05 (S and both
// halves of O in TMEM), so what is left is latency: a slice of an index is a
// handful of tiles.
//
//   * Warps 9-12 (producers) load the codes of a tile straight into registers
//     (16 bytes a lane, the next K and V pieces in flight while the last ones
//     are stored), make halves of them (exact) and write them as 128-byte
//     swizzled tiles, K as [keys, d] K-major, V the same rows read MN-major.
//   * Warp 8 issues S = Q K^T and, per key half h, O_h += P_h V_h.
//   * Warps 0-7: softmax, one query row per thread and key half, P written
//     over the consumed K tile.  The V scale joins P, not V: with l the sum of
//     p = 2^(z - m), O sums p * (vs 2^lc).  m and lc are whole numbers, m moves
//     when a logit passes it by 14 and lc keeps the largest p vs 2^lc between
//     2^7 and 2^14: halves hold a weight's 11 bits, however far the scales are
//     apart, and moving m costs no pass over O (lc takes it up).  (lc stops at
//     67: V scales below 2^-60 lose their weights' bits towards f16's
//     subnormals.)  fp32 outputs use two halves per weight (22 bits).
//   * Queries enter as halves scaled per row by a power of two (as in
//     attn_q8.cu); each row leaves its slice's (m, l, o / l) in the workspace,
//     and a second kernel merges them.  It is launched with
//     programmatic dependence and reads one row per warp, so the merge uses
//     the whole GPU and no counters.
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

constexpr int kDg = 128;
constexpr int kKeysG = 128;     // keys of a tile
constexpr int kSoftWarps = 8, kMmaWarp = 8, kProdWarp = 9, kProdWarps = 4;
constexpr int kThreadsG = 32 * (kProdWarp + kProdWarps);
constexpr int kPer = 128 * 8 / (32 * kProdWarps);  // 16-byte pieces of a K (or V) tile a producer holds
static_assert(32 * kProdWarps == kKeysG, "one producer thread per key's scales");
constexpr int kRowStep = 128 / kPer;
constexpr int kHalfG = 16384;   // 128 rows x 128 bytes
constexpr int kTileG = 2 * kHalfG;
constexpr int kStagesG = 2;
constexpr int kORowG = kDg + 4;  // floats of an output row in shared memory

constexpr int kMinExp = -60;
constexpr float kMaxLc = 7.f - kMinExp;

struct alignas(16) MetaG {
  float ks[kKeysG], vs[kKeysG], ve[kKeysG];  // scales, and the exponent of vs (at least kMinExp)
  uint32_t seen[4];                          // bit c of word w: key 32w + c is a token
  float emax[4];                             // largest ve of the word
};

template <bool PRECISE>
struct SmemG {
  static constexpr int kStage = kTileG;                           // after Q: K then V of each stage
  static constexpr int kPlo = kStage + kStagesG * 2 * kTileG;     // low halves of P
  static constexpr int kMeta = kPlo + (PRECISE ? kTileG : 0);
  static constexpr int kRf = kMeta + kStagesG * (int)sizeof(MetaG);
  static constexpr int kBar = kRf + kQ8RowTile * 4;
  // k_full[2] v_full[2] kv_empty[2] s_full[2] s_free[2] p_full[2] o_done[4] q_full
  static constexpr int kSlot = kBar + 8 * 17;
  static constexpr size_t kBytes = 1024 + kSlot + 16;
  static_assert(kBytes <= 232448, "shared memory budget");
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two floats at once
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return pair(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ bool warp_wait_g(uint64_t* bar, uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, kWaitLimitNs);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// 16 codes (dims 16c ..) of key row r as halves into a [128, 128] tile at `tile`.
// A half row is 64 dims; the two 16-byte chunks are stored in the order that
// keeps the 8 lanes of a row on different banks.
__device__ __forceinline__ void store_codes(uint32_t tile, int r, int c, const uint4& v) {
  uint32_t h[8];
  q8_to_half4(v.x, h[0], h[1]);
  q8_to_half4(v.y, h[2], h[3]);
  q8_to_half4(v.z, h[4], h[5]);
  q8_to_half4(v.w, h[6], h[7]);
  const int up = c >> 2;
  const uint32_t base = tile + up * kHalfG;
  const uint32_t a0 = base + sw128_offset(r, (c & 3) * 2), a1 = base + sw128_offset(r, (c & 3) * 2 + 1);
  sts16(up ? a1 : a0, up ? h[4] : h[0], up ? h[5] : h[1], up ? h[6] : h[2], up ? h[7] : h[3]);
  sts16(up ? a0 : a1, up ? h[0] : h[4], up ? h[1] : h[5], up ? h[2] : h[6], up ? h[3] : h[7]);
}

template <bool PRECISE>
__global__ void __launch_bounds__(kThreadsG, 1) attn_q8_group_kernel(const Q8AttnArgs a, const int row_tiles) {
  using Lay = SmemG<PRECISE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  MetaG* meta = reinterpret_cast<MetaG*>(smem + Lay::kMeta);
  float* rf_s = reinterpret_cast<float*>(smem + Lay::kRf);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* v_full = k_full + 2;
  uint64_t* kv_empty = v_full + 2;
  uint64_t* s_full = kv_empty + 2;
  uint64_t* s_free = s_full + 2;
  uint64_t* p_full = s_free + 2;
  uint64_t* o_done = p_full + 2;  // [4]: PV of tile i on o_done[i % 4]
  uint64_t* q_full = o_done + 4;
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + Lay::kSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % a.n_split;
  const int unit = blockIdx.x / a.n_split;  // (b, g, row tile)
  const int rt = unit % row_tiles;
  const int g = unit / row_tiles % a.Hkv, b = unit / row_tiles / a.Hkv;
  const int row_base = rt * kQ8RowTile;

  pdl_trigger();
  if (warp == kMmaWarp) {
    tmem_alloc(slot, 512);
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&k_full[i], kProdWarps);
        mbar_init(&v_full[i], kProdWarps);
        mbar_init(&kv_empty[i], 1);
        mbar_init(&s_full[i], 1);
        mbar_init(&s_free[i], kSoftWarps);
        mbar_init(&p_full[i], kSoftWarps);
      }
      for (int i = 0; i < 4; ++i) mbar_init(&o_done[i], 1);
      mbar_init(q_full, kSoftWarps);
      fence_mbar_init();
    }
  }
  pdl_wait();
  const Q8Seq s = q8_seq(a.seq_off, a.seq_len, b, a.n_tokens, a.S_max);
  if (!s.ok && tid == 0 && slice == 0) report(a.status, kErrDevice, kKernAttnQ8, b, s.len, s.cap);
  const int n_keys = !s.ok ? 0 : a.idx ? a.k : s.len;  // entries, or tokens
  const int e_beg = min(n_keys, slice * a.chunk), e_end = min(n_keys, e_beg + a.chunk);
  const int nt = (e_end - e_beg + kKeysG - 1) / kKeysG;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int64_t part = (int64_t)unit * a.n_split + slice;

  if (warp >= kProdWarp) {
    // =============== producers ===============
    const int pt = tid - kProdWarp * 32;
    const int pr = pt >> 3, pc = pt & 7;  // rows pr + kRowStep i, 16-byte piece pc
    const int64_t row0 = s.off * a.Hkv + (int64_t)g * s.cap;
    const bool rep = g == 0 && rt == 0;
    // token of key r of tile j, or -1
    auto token = [&](int j, int r) -> int {
      const int e = e_beg + j * kKeysG + r;
      if (e >= e_end) return -1;
      return a.idx ? __ldcg(&a.idx[(int64_t)b * a.k + e]) : e;
    };
    auto fetch = [&](const uint8_t* codes, const int (&t)[kPer], uint4 (&v)[kPer]) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        v[i] = t[i] >= 0 && t[i] < s.len
                   ? __ldcg(reinterpret_cast<const uint4*>(codes + (row0 + t[i]) * kDg + pc * 16))
                   : make_uint4(0, 0, 0, 0);
    };
    int tok[kPer], tok_next[kPer], tm, tm_next;  // tm: the key whose scales this thread loads
    uint4 kv[kPer], vv[kPer];
    float ks = 0.f, vs = 0.f;
    auto scales = [&]() {
      ks = vs = 0.f;
      if (tm >= 0 && tm < s.len) {
        ks = __ldcg(a.Ks + (row0 + tm) / kQ8Block);
        vs = __ldcg(a.Vs + (row0 + tm) / kQ8Block);
      }
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) tok[i] = token(0, pr + kRowStep * i);
    tm = token(0, pt);  // producers are as many as keys
#pragma unroll
    for (int i = 0; i < kPer; ++i) tok_next[i] = token(1, pr + kRowStep * i);
    tm_next = token(1, pt);
    fetch(a.K, tok, kv);
    scales();
    fetch(a.V, tok, vv);
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      if (j >= kStagesG && !warp_wait_g(&kv_empty[st], ((j >> 1) & 1) ^ 1)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 0, j);
        break;
      }
      const uint32_t kst = sbase + Lay::kStage + st * 2 * kTileG;
#pragma unroll
      for (int i = 0; i < kPer; ++i) store_codes(kst, pr + kRowStep * i, pc, kv[i]);
      if (tm >= s.len) {
        if (rep) report(a.status, kErrDevice, kKernAttnQ8, (int64_t)b * a.k + e_beg + j * kKeysG + pt, tm, s.len);
        tm = -1;
      }
      meta[st].ks[pt] = ks;
      const int ex = (int)(__float_as_uint(vs) >> 23 & 0xff);
      meta[st].vs[pt] = ex == 0 ? 0.f : vs;  // below 2^-126: zero
      const int ve = max(ex - 127, kMinExp);
      meta[st].ve[pt] = (float)ve;
      const uint32_t seen = __ballot_sync(0xffffffffu, tm >= 0);
      const int top = __reduce_max_sync(0xffffffffu, ve);
      if (lane == 0) {
        meta[st].seen[pt >> 5] = seen;
        meta[st].emax[pt >> 5] = (float)top;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
#pragma unroll
      for (int i = 0; i < kPer; ++i) tok[i] = tok_next[i];
      tm = tm_next;
      fetch(a.K, tok, kv);
      scales();
#pragma unroll
      for (int i = 0; i < kPer; ++i) store_codes(kst + kTileG, pr + kRowStep * i, pc, vv[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
      fetch(a.V, tok, vv);
#pragma unroll
      for (int i = 0; i < kPer; ++i) tok_next[i] = token(j + 2, pr + kRowStep * i);
      tm_next = token(j + 2, pt);
    }
  } else if (warp == kMmaWarp) {
    // =============== MMA issuer ===============
    if (lane == 0 && nt > 0) {
      constexpr uint32_t idesc_qk = idesc_f16(128, 128, false), idesc_pv = idesc_f16(128, 128, true);
      auto pv = [&](int i) -> bool {
        const int st = i & 1;
        if (!mbar_wait(&v_full[st], (i >> 1) & 1, kWaitLimitNs) || !mbar_wait(&p_full[st], (i >> 1) & 1, kWaitLimitNs))
          return false;
        tc_fence_after();
        const uint32_t kst = sbase + Lay::kStage + st * 2 * kTileG;  // P lives here now
        const uint32_t vst = kst + kTileG;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // keys 64h + 16kk ..
            const uint64_t vd = umma_desc_sw128(vst + h * 8192 + kk * 2048, kHalfG, 1024);
            umma_bf16(tmem + 256 + 128 * h, umma_desc_sw128(kst + h * kHalfG + kk * 32, 16, 1024), vd, idesc_pv,
                      (i | kk) != 0);
            if (PRECISE)
              umma_bf16(tmem + 256 + 128 * h, umma_desc_sw128(sbase + Lay::kPlo + h * kHalfG + kk * 32, 16, 1024), vd,
                        idesc_pv, 1);
          }
        umma_commit(&kv_empty[st]);
        umma_commit(&o_done[i & 3]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, kWaitLimitNs);
      for (int j = 0; j < nt && ok; ++j) {
        const int st = j & 1;
        ok = mbar_wait(&k_full[st], (j >> 1) & 1, kWaitLimitNs) &&
             mbar_wait(&s_free[st], ((j >> 1) & 1) ^ 1, kWaitLimitNs);
        if (!ok) break;
        tc_fence_after();
        const uint32_t kst = sbase + Lay::kStage + st * 2 * kTileG;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem + st * 128, umma_desc_sw128(sbase + h * kHalfG + kk * 32, 16, 1024),
                      umma_desc_sw128(kst + h * kHalfG + kk * 32, 16, 1024), idesc_qk, (h | kk) != 0);
        umma_commit(&s_full[st]);
        if (j >= 1) ok = pv(j - 1);
      }
      if (ok) ok = pv(nt - 1);
      if (!ok) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 1, 0);
    }
  } else {
    // =============== queries, then softmax ===============
    if (nt > 0) {
      constexpr int kRowsWarp = kQ8RowTile / kSoftWarps;
      uint2 qv[kRowsWarp];  // rows warp + 8 i, dims 4*lane ..: every load before the first use
#pragma unroll
      for (int i = 0; i < kRowsWarp; ++i) {
        const int row = row_base + warp + kSoftWarps * i;
        const int64_t off = (((int64_t)(row / a.G) * a.B + b) * a.Hq + g * a.G + row % a.G) * kDg;
        qv[i] = row < a.R ? __ldcg(reinterpret_cast<const uint2*>(a.Q + off) + lane) : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kRowsWarp; ++i) {
        const int r = warp + kSoftWarps * i;
        const uint2 v = qv[i];
        const float x0 = bf_lo(v.x), x1 = bf_hi(v.x), x2 = bf_lo(v.y), x3 = bf_hi(v.y);
        const float mx = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
        const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
        // 2^e with the largest element in [2^14, 2^15); 1 for zero or non-finite rows
        int e = mb == 0u || mb >= 0x7f800000u ? 127 : 127 + 14 + 127 - (int)(mb >> 23);
        e = min(e, 253);  // tiny rows: as large as a float scale goes
        const float up = __uint_as_float((uint32_t)e << 23);
        const uint32_t at = sbase + (lane >> 4) * kHalfG + sw128_offset(r, (lane & 15) >> 1) + (lane & 1) * 8;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(pack_half2(x0 * up, x1 * up)),
                     "r"(pack_half2(x2 * up, x3 * up))
                     : "memory");
        if (lane == 0) rf_s[r] = fmaxf(a.scale_log2 / up, 1e-45f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int half = warp >> 2;
    const int r_loc = (warp & 3) * 32 + lane;
    const bool active = row_base + (warp & 3) * 32 < a.R;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tmem_o = tmem + 256 + 128 * half + lane_base;
    float m = -INFINITY, lc = 0.f, l_run = 0.f, rf = 0.f;
    bool failed = false;
    for (int j = 0; j < nt; ++j) {
      const int st = j & 1;
      if (!warp_wait_g(&s_full[st], (j >> 1) & 1) || !warp_wait_g(&k_full[st], (j >> 1) & 1) ||
          (j == 0 && !warp_wait_g(q_full, 0))) {
        failed = true;
        break;
      }
      tc_fence_after();
      if (active) {
        if (j == 0) rf = rf_s[r_loc];
        const MetaG& mt = meta[st];
        const uint32_t tmem_s = tmem + st * 128 + 64 * half + lane_base;
        const uint32_t vis[2] = {mt.seen[2 * half], mt.seen[2 * half + 1]};
        const uint64_t* ks2 = reinterpret_cast<const uint64_t*>(mt.ks + 64 * half);
        const uint64_t* vs2 = reinterpret_cast<const uint64_t*>(mt.vs + 64 * half);
        // ---- the largest logit ----
        float wm[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) wm[i] = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32];
          tmem_ld32(tmem_s + 32 * c, sv);
          tmem_wait_ld();
          const bool all = vis[c] == 0xffffffffu;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float2 w = unpair(mul2(pair(sv[2 * q], sv[2 * q + 1]), ks2[16 * c + q]));
            wm[q & 3] = fmaxf(wm[q & 3], all || (vis[c] >> (2 * q) & 1u) ? w.x : -INFINITY);
            wm[4 + (q & 3)] = fmaxf(wm[4 + (q & 3)], all || (vis[c] >> (2 * q + 1) & 1u) ? w.y : -INFINITY);
          }
        }
        const float zmax = rf * fmaxf(fmaxf(fmaxf(wm[0], wm[1]), fmaxf(wm[2], wm[3])),
                                      fmaxf(fmaxf(wm[4], wm[5]), fmaxf(wm[6], wm[7])));
        float alpha = 1.f;
        bool look = false;  // whether P may leave its range: then the largest weight decides
        if (zmax > m + 14.f) {  // also when the row has no reference yet
          const float to = ceilf(zmax);
          if (m == -INFINITY) {
            lc = 1000.f;  // O is empty: the rule below picks the unit
          } else {
            l_run *= ex2f(m - to);
            lc += to - m;  // O keeps its unit
          }
          m = to;
        }
        look = zmax > -INFINITY && (zmax - m + fmaxf(mt.emax[2 * half], mt.emax[2 * half + 1]) + lc > 14.f || lc > kMaxLc);
        if (__any_sync(0xffffffffu, look)) {
          float ymax = -INFINITY;  // the largest logit + exponent of its V scale
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t sv[16];
            tmem_ld16(tmem_s + 16 * c, sv);
            tmem_wait_ld();
            const uint32_t see = vis[c >> 1] >> (16 * (c & 1));
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int at = 64 * half + 16 * c + e;
              const float y = fmaf(__uint_as_float(sv[e]) * mt.ks[at], rf, mt.ve[at]);
              if (see >> e & 1u) ymax = fmaxf(ymax, y);
            }
          }
          if (look && (ymax - m + lc > 14.f || lc > kMaxLc)) {
            const float to = fmaxf(fminf(fminf(lc, m - ceilf(ymax) + 7.f), kMaxLc), -126.f);
            alpha = ex2f(to - lc);
            lc = to;
          }
          if (__any_sync(0xffffffffu, alpha != 1.f) && j > 0) {
            // the last tile's PV must have landed before O is rescaled
            if (!warp_wait_g(&o_done[(j - 1) & 3], ((j - 1) >> 2) & 1)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t ov[16];
              tmem_ld16(tmem_o + c * 16, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st16(tmem_o + c * 16, ov);
            }
            tmem_wait_st();
          }
        }
        // ---- P over this half of the consumed K tile ----
        if (PRECISE && j > 0 && !warp_wait_g(&o_done[(j - 1) & 3], ((j - 1) >> 2) & 1)) {
          failed = true;  // the low halves of the last tile are still being read
          break;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
        const float unit_c = __int_as_float(((int)lc + 127) << 23);  // 2^lc
        const uint64_t rf2 = pair(rf, rf), neg2 = pair(neg_m, neg_m), unit2 = pair(unit_c, unit_c);
        const uint32_t pst = sbase + Lay::kStage + st * 2 * kTileG + half * kHalfG;
        uint64_t ls[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32];
          tmem_ld32(tmem_s + 32 * c, sv);
          tmem_wait_ld();
          const bool all = vis[c] == 0xffffffffu;
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // 8 keys: one 16-byte chunk of the row's P
            uint64_t pv[4];
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = 4 * q + i;
              const float2 x = unpair(fma2(mul2(pair(sv[2 * at], sv[2 * at + 1]), ks2[16 * c + at]), rf2, neg2));
              float2 y = make_float2(ex2f(x.x), ex2f(x.y));
              if (!all) {
                y.x = vis[c] >> (2 * at) & 1u ? y.x : 0.f;
                y.y = vis[c] >> (2 * at + 1) & 1u ? y.y : 0.f;
              }
              const uint64_t y2 = pair(y.x, y.y);
              ls[i & 1] = add2(ls[i & 1], y2);
              pv[i] = mul2(y2, mul2(vs2[16 * c + at], unit2));
              const float2 f = unpair(pv[i]);
              h[i] = pack_half2(f.x, f.y);
            }
            const uint32_t off = sw128_offset(r_loc, 4 * c + q);
            sts16(pst + off, h[0], h[1], h[2], h[3]);
            if (PRECISE) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpair(pv[i]), t = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                h[i] = pack_half2(f.x - t.x, f.y - t.y);
              }
              sts16(sbase + Lay::kPlo + half * kHalfG + off, h[0], h[1], h[2], h[3]);
            }
          }
        }
        const float2 l0 = unpair(ls[0]), l1 = unpair(ls[1]);
        l_run += (l0.x + l0.y) + (l1.x + l1.y);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_free[st]);
        mbar_arrive(&p_full[st]);
      }
    }
    // ---- the row's two key halves into one (m, l, o / l) in shared memory ----
    if (nt > 0 && !failed) failed = !warp_wait_g(&o_done[(nt - 1) & 3], ((nt - 1) >> 2) & 1);
    if (failed && lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 2, warp);
    tc_fence_after();
    // every MMA is done (the barrier): the stages are free for the rows
    float2* ml_s = reinterpret_cast<float2*>(smem + Lay::kMeta);  // [2][128]
    float* o_s = reinterpret_cast<float*>(smem + Lay::kStage);
    ml_s[half * kQ8RowTile + r_loc] = make_float2(m, l_run);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float2 other = ml_s[(half ^ 1) * kQ8RowTile + r_loc];
    const float M = fmaxf(m, other.x);
    const float mine = m == -INFINITY ? l_run : ex2f(m - M);  // an empty half: 0, or a NaN sum
    const float L = mine * l_run + (other.x == -INFINITY ? other.y : ex2f(other.x - M) * other.y);
    // o's unit is 2^lc
    const float f = (L == 0.f ? 0.f : mine / L) * __int_as_float((127 - (int)fmaxf(lc, -126.f)) << 23);
    auto rows = [&](bool add) {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t ov[32];
        tmem_ld32(tmem_o + c * 32, ov);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          float4* at = reinterpret_cast<float4*>(o_s + r_loc * kORowG + c * 32 + e);
          float4 v = make_float4(__uint_as_float(ov[e]) * f, __uint_as_float(ov[e + 1]) * f,
                                 __uint_as_float(ov[e + 2]) * f, __uint_as_float(ov[e + 3]) * f);
          if (add) {
            const float4 t = *at;
            v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
          }
          *at = v;
        }
      }
    };
    if (half == 1 && active && nt > 0) rows(false);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (half == 0 && active) {
      if (nt > 0) rows(true);
      if (row_base + r_loc < a.R) __stcg(&a.pml[part * kQ8RowTile + r_loc], make_float2(M, L));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (nt > 0) {
    const float* o_s = reinterpret_cast<const float*>(smem + Lay::kStage);
    const int n = min(kQ8RowTile, a.R - row_base) * (kDg / 4);
    float4* dst = reinterpret_cast<float4*>(a.po + part * kQ8RowTile * kDg);
    for (int i = tid; i < n; i += kThreadsG)
      __stcg(dst + i, *reinterpret_cast<const float4*>(o_s + i / (kDg / 4) * kORowG + i % (kDg / 4) * 4));
  }
}

// One warp per query row: the parts' (m, l, o / l) into the output row.
__global__ void __launch_bounds__(256) attn_q8_merge_kernel(const Q8AttnArgs a, const int row_tiles, const int n_rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x * 8 + warp;  // (b, g, row)
  if (i >= n_rows) return;
  const int row = i % a.R, bg = i / a.R;
  const int g = bg % a.Hkv, b = bg / a.Hkv;
  const int n = a.n_split;
  const int64_t p0 = ((int64_t)bg * row_tiles + row / kQ8RowTile) * n * kQ8RowTile + row % kQ8RowTile;
  float M = -INFINITY;
  for (int p = lane; p < n; p += 32) M = fmaxf(M, __ldcg(&a.pml[p0 + (int64_t)p * kQ8RowTile]).x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < n; base += 32) {
    float w = 0.f;
    if (base + lane < n) {
      const float2 ml = __ldcg(&a.pml[p0 + (int64_t)(base + lane) * kQ8RowTile]);
      w = (ml.x == -INFINITY ? 0.f : ex2f(ml.x - M)) * ml.y;
    }
    const int m = min(32, n - base);
#pragma unroll 8
    for (int p = 0; p < m; ++p) {
      const float f = __shfl_sync(0xffffffffu, w, p);
      L += f;
      if (f == 0.f) continue;  // nothing of this part is in the workspace
      const float4 v = __ldcg(reinterpret_cast<const float4*>(a.po + (p0 + (int64_t)(base + p) * kQ8RowTile) * kDg) + lane);
      acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t off = (((int64_t)(row / a.G) * a.B + b) * a.Hq + g * a.G + row % a.G) * kDg + 4 * lane;
  if (a.out_f32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.O) + off) =
        make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.O) + off) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

template <typename... Exp, typename... Act>
cudaError_t launch_pdl(void (*kern)(Exp...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                       Act... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// One CTA per SM and one wave, at most the 128-key tiles there are.
void plan_attn_q8_group(Q8AttnPlan& p, int64_t n, int sms) {
  const int64_t tiles = n > 0 ? (n + kKeysG - 1) / kKeysG : 1;
  int64_t split = sms / p.units > 1 ? sms / p.units : 1;
  if (split > tiles) split = tiles;
  p.chunk = (int)((tiles + split - 1) / split) * kKeysG;
  p.n_split = (int)((tiles * kKeysG + p.chunk - 1) / p.chunk);
  p.parts = p.n_split;
  p.rows = kQ8RowTile;
}

cudaError_t launch_attn_q8_group(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream) {
  auto kern = a.out_f32 ? attn_q8_group_kernel<true> : attn_q8_group_kernel<false>;
  const size_t smem = a.out_f32 ? SmemG<true>::kBytes : SmemG<false>::kBytes;
  cudaError_t e = ensure_smem(kern, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, (unsigned)(p.units * p.n_split), kThreadsG, smem, stream, a, p.row_tiles);
  if (e != cudaSuccess) return e;
  const int n_rows = a.B * a.Hkv * a.R;
  return launch_pdl(attn_q8_merge_kernel, (unsigned)((n_rows + 7) / 8), 256, 0, stream, a, p.row_tiles, n_rows);
}

}  // namespace sa
