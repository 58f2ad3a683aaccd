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
//   * Warps 9-16 (producers) load the codes of a tile straight into registers
//     (16 bytes a lane, the next K and V pieces in flight while the last ones
//     are stored), make halves of them (exact) and write them as 128-byte
//     swizzled tiles, K as [keys, d] K-major, V the same rows read MN-major.
//   * Warp 8 issues S = Q K^T and, per key half h, O_h += P_h V_h.
//   * Warps 0-7: softmax, one query row per thread and key half, P written
//     over the consumed K tile.  The V scale joins P, not V: with l the sum of
//     p = 2^(z - m), O sums p * (vs 2^lc).  m and lc are whole numbers, m moves
//     when a logit passes it by 14 and lc keeps the largest p vs 2^lc between
//     2^7 and 2^14: halves hold a weight's 11 bits, whatever the scales, and
//     moving m costs no pass over O (lc takes it up).  fp32 outputs use two
//     halves per weight (22 bits).
//   * Queries enter as halves scaled per row by a power of two (as in
//     attn_q8.cu), each row and key half leaves (m, l, o / l) of its slice in
//     the workspace, and a second kernel merges them.  It is launched with
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
constexpr int kSoftWarps = 8, kMmaWarp = 8, kProdWarp = 9, kProdWarps = 8;
constexpr int kThreadsG = 32 * (kProdWarp + kProdWarps);
constexpr int kHalfG = 16384;   // 128 rows x 128 bytes
constexpr int kTileG = 2 * kHalfG;
constexpr int kStagesG = 2;

struct MetaG {
  float ks[kKeysG], vs[kKeysG], ve[kKeysG];  // scales, and the exponent of vs
  uint32_t seen[4];                          // bit c of word w: key 32w + c is a token
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
  const int64_t part0 = ((int64_t)unit * a.n_split + slice) * 2;  // two key halves

  if (warp >= kProdWarp) {
    // =============== producers ===============
    const int pt = tid - kProdWarp * 32;
    const int pr = pt >> 3, pc = pt & 7;  // rows pr + 32 i, 16-byte piece pc
    const int64_t row0 = s.off * a.Hkv + (int64_t)g * s.cap;
    const bool rep = g == 0 && rt == 0;
    // token of key r of tile j, or -1
    auto token = [&](int j, int r) -> int {
      const int e = e_beg + j * kKeysG + r;
      if (e >= e_end) return -1;
      return a.idx ? __ldcg(&a.idx[(int64_t)b * a.k + e]) : e;
    };
    auto fetch = [&](const uint8_t* codes, const int (&t)[4], uint4 (&v)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = t[i] >= 0 && t[i] < s.len
                   ? __ldcg(reinterpret_cast<const uint4*>(codes + (row0 + t[i]) * kDg + pc * 16))
                   : make_uint4(0, 0, 0, 0);
    };
    int tok[4], tok_next[4], tm = -1, tm_next = -1;  // tm: the key whose scales this thread loads
    uint4 kv[4], vv[4];
    float ks = 0.f, vs = 0.f;
    auto scales = [&]() {
      ks = vs = 0.f;
      if (tm >= 0 && tm < s.len) {
        ks = __ldcg(a.Ks + (row0 + tm) / kQ8Block);
        vs = __ldcg(a.Vs + (row0 + tm) / kQ8Block);
      }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) tok[i] = token(0, pr + 32 * i);
    if (pt < kKeysG) tm = token(0, pt);
#pragma unroll
    for (int i = 0; i < 4; ++i) tok_next[i] = token(1, pr + 32 * i);
    if (pt < kKeysG) tm_next = token(1, pt);
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
      for (int i = 0; i < 4; ++i) store_codes(kst, pr + 32 * i, pc, kv[i]);
      if (pt < kKeysG) {
        if (tm >= s.len) {
          if (rep) report(a.status, kErrDevice, kKernAttnQ8, (int64_t)b * a.k + e_beg + j * kKeysG + pt, tm, s.len);
          tm = -1;
        }
        meta[st].ks[pt] = ks;
        const int ex = (int)(__float_as_uint(vs) >> 23 & 0xff);
        meta[st].vs[pt] = ex == 0 ? 0.f : vs;  // below 2^-126: zero
        meta[st].ve[pt] = ex == 0 ? 0.f : (float)(ex - 127);
        const uint32_t seen = __ballot_sync(0xffffffffu, tm >= 0);
        if (lane == 0) meta[st].seen[pt >> 5] = seen;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[st]);
#pragma unroll
      for (int i = 0; i < 4; ++i) tok[i] = tok_next[i];
      tm = tm_next;
      fetch(a.K, tok, kv);
      scales();
#pragma unroll
      for (int i = 0; i < 4; ++i) store_codes(kst + kTileG, pr + 32 * i, pc, vv[i]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[st]);
      fetch(a.V, tok, vv);
#pragma unroll
      for (int i = 0; i < 4; ++i) tok_next[i] = token(j + 2, pr + 32 * i);
      if (pt < kKeysG) tm_next = token(j + 2, pt);
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
      for (int r = warp; r < kQ8RowTile; r += kSoftWarps) {
        const int row = row_base + r;
        uint2 v = make_uint2(0u, 0u);
        if (row < a.R) {
          const int64_t off = (((int64_t)(row / a.G) * a.B + b) * a.Hq + g * a.G + row % a.G) * kDg;
          v = __ldcg(reinterpret_cast<const uint2*>(a.Q + off) + lane);  // dims 4*lane ..
        }
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
        if (lane == 0) rf_s[r] = a.scale_log2 / up;
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
        // ---- the largest logit, and the largest logit + exponent of its V scale ----
        float zm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        float ym[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32];
          tmem_ld32(tmem_s + 32 * c, sv);
          tmem_wait_ld();
          const float4* ks4 = reinterpret_cast<const float4*>(mt.ks + 64 * half + 32 * c);
          const float4* ve4 = reinterpret_cast<const float4*>(mt.ve + 64 * half + 32 * c);
          if (vis[c] == 0xffffffffu) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 k = ks4[q], v = ve4[q];
              const float z0 = __uint_as_float(sv[4 * q]) * (k.x * rf), z1 = __uint_as_float(sv[4 * q + 1]) * (k.y * rf);
              const float z2 = __uint_as_float(sv[4 * q + 2]) * (k.z * rf), z3 = __uint_as_float(sv[4 * q + 3]) * (k.w * rf);
              zm[0] = fmaxf(zm[0], z0), zm[1] = fmaxf(zm[1], z1), zm[2] = fmaxf(zm[2], z2), zm[3] = fmaxf(zm[3], z3);
              ym[0] = fmaxf(ym[0], z0 + v.x), ym[1] = fmaxf(ym[1], z1 + v.y);
              ym[2] = fmaxf(ym[2], z2 + v.z), ym[3] = fmaxf(ym[3], z3 + v.w);
            }
          } else if (vis[c] != 0u) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (vis[c] >> e & 1u) {
                const float z = __uint_as_float(sv[e]) * (mt.ks[64 * half + 32 * c + e] * rf);
                zm[e & 3] = fmaxf(zm[e & 3], z);
                ym[e & 3] = fmaxf(ym[e & 3], z + mt.ve[64 * half + 32 * c + e]);
              }
          }
        }
        const float zmax = fmaxf(fmaxf(zm[0], zm[1]), fmaxf(zm[2], zm[3]));
        const float ymax = fmaxf(fmaxf(ym[0], ym[1]), fmaxf(ym[2], ym[3]));
        float alpha = 1.f;
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
        if (ymax - m + lc > 14.f || lc > 126.f) {
          const float to = fmaxf(fminf(fminf(lc, m - ceilf(ymax) + 7.f), 126.f), -126.f);
          alpha = ex2f(fminf(to - lc, 126.f));
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
          for (int c = 0; c < 4; ++c) {
            uint32_t ov[32];
            tmem_ld32(tmem_o + c * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tmem_o + c * 32, ov);
          }
          tmem_wait_st();
        }
        // ---- P over this half of the consumed K tile ----
        if (PRECISE && j > 0 && !warp_wait_g(&o_done[(j - 1) & 3], ((j - 1) >> 2) & 1)) {
          failed = true;  // the low halves of the last tile are still being read
          break;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
        const float unit_c = __int_as_float(((int)lc + 127) << 23);  // 2^lc
        const uint32_t pst = sbase + Lay::kStage + st * 2 * kTileG + half * kHalfG;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t sv[32];
          tmem_ld32(tmem_s + 32 * c, sv);
          tmem_wait_ld();
          const bool all = vis[c] == 0xffffffffu;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float p[8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int at = 64 * half + 32 * c + 8 * q + 4 * u;
              const float4 k = *reinterpret_cast<const float4*>(mt.ks + at);
              const float4 v = *reinterpret_cast<const float4*>(mt.vs + at);
              const float kk[4] = {k.x, k.y, k.z, k.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int col = 8 * q + 4 * u + e;
                float x = ex2f(fmaf(__uint_as_float(sv[col]), kk[e] * rf, neg_m));
                if (!all && !(vis[c] >> col & 1u)) x = 0.f;
                ls[e] += x;
                p[4 * u + e] = x * fminf(vv[e] * unit_c, 0x1p126f);
              }
            }
            const uint32_t off = sw128_offset(r_loc, 4 * c + q);
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = pack_half2(p[2 * i], p[2 * i + 1]);
            sts16(pst + off, h[0], h[1], h[2], h[3]);
            if (PRECISE) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                h[i] = pack_half2(p[2 * i] - f.x, p[2 * i + 1] - f.y);
              }
              sts16(sbase + Lay::kPlo + half * kHalfG + off, h[0], h[1], h[2], h[3]);
            }
          }
        }
        l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_free[st]);
        mbar_arrive(&p_full[st]);
      }
    }
    // ---- this slice's (m, l, o / l) of the row and key half ----
    if (nt > 0 && !failed) failed = !warp_wait_g(&o_done[(nt - 1) & 3], ((nt - 1) >> 2) & 1);
    if (failed) {
      if (lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 2, warp);
    } else if (active) {
      const int64_t at = (part0 + half) * kQ8RowTile + r_loc;
      if (row_base + r_loc < a.R) __stcg(&a.pml[at], make_float2(m, l_run));
      if (nt > 0) {
        tc_fence_after();
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;  // a NaN sum stays one
        const float f = inv * __int_as_float((127 - (int)lc) << 23);  // o's unit is 2^lc
        float* dst = a.po + at * kDg;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t ov[32];
          tmem_ld32(tmem_o + c * 32, ov);
          tmem_wait_ld();
          if (row_base + r_loc < a.R) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              __stcg(reinterpret_cast<float4*>(dst + c * 32 + e),
                     make_float4(__uint_as_float(ov[e]) * f, __uint_as_float(ov[e + 1]) * f,
                                 __uint_as_float(ov[e + 2]) * f, __uint_as_float(ov[e + 3]) * f));
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
  const int n = 2 * a.n_split;
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
  p.parts = 2 * p.n_split;
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
