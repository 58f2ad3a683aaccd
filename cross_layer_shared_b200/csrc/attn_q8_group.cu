// Decode attention over the 8-bit cache for many query rows per KV head (the
// layers of a group that share an index, or many heads): the operator of
// attn_q8.cu on tcgen05 tiles of 128 query rows x 128 keys.
//
// What bounds it: with R rows a (token, KV head) costs 256 + 8/64 bytes and
// 512 R flops.  From about 16 rows the warp-level MMAs of attn_q8.cu, whose
// warps each convert all codes they multiply, are issue-bound; here each code
// is converted once per 128 rows and the products run on tcgen05 (S and O in
// TMEM).  What is left is latency around a slice's handful of tiles, and for
// each tile the conversion.
//
//   * Warps 9-16 (producers) load the codes of a tile straight into registers
//     (16 bytes a lane, the next K and V pieces in flight while the last ones
//     are stored) and write scale * code as bf16: exact for the powers of two
//     an append writes (4 significant bits), so S and PV see the cache's own
//     values and the softmax no scales.  K as [keys, d] K-major, V the same
//     rows read MN-major, 128-byte swizzled.
//   * Warp 8 issues S = Q K^T and O += P V.
//   * Warps 0-7: softmax, one query row per thread and key half, P written
//     over the consumed K tile.  One pass: weights are 2^(z - m) with m the
//     row's first logit until one passes it by 30 (fp32 and bf16 have the
//     exponents for that); only then the row's sums move to a new m and the
//     tile's weights are made again.  Both halves of a row keep one m: its two
//     warps meet once a tile to agree on that.
//   * l is a column of its own in the products: P times ones.  It is the sum of
//     the weights as they were rounded, so that they add up to one, and costs
//     the softmax nothing.  bf16 outputs: weights of 8 bits, the output's own.
//     fp32 outputs: three bf16 parts (24 bits), for whose shared memory K has
//     one stage instead of three.
//   * The key slices of 128 rows are a cluster of up to 8 CTAs: each leaves its
//     rows' (m, l, o / l) in its shared memory and merges 128 / 8 rows of all
//     of them.  More slices than that (few rows over a long context) go
//     through the workspace and a second kernel, one row per warp.
//
// Measured (B200, warm graph replay): 24 layers of 32 query and 8 KV heads (96
// rows) over 2048 picked tokens of 4 sequences 18.2 us, of which 4.3 go by
// before the first S, 7 over four tiles and 5 on the last products, the
// cluster's barrier and the merge.  Many tiles take 2.1 us each, and the
// producers set that pace: about 3200 cycles for a tile's loads and stores of K,
// then V, and the memory behind them; the softmax needs 2100, the products 1500.
// Four producer warps for K and four for V, without barriers among them, are
// faster over many tiles (246 for 278 us, 20 rows over 65,536 tokens of 32
// sequences and heads) and slower over the four of a picked step (18.8): not taken.
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
constexpr int kPer = 128 * 8 / (32 * kProdWarps);  // 16-byte pieces of a K (or V) tile a producer holds
constexpr int kRowStep = 128 / kPer;
static_assert(32 * kProdWarps >= kKeysG, "one producer thread per key's token and scales");
constexpr int kHalfG = 16384;   // 128 rows x 128 bytes
constexpr int kTileG = 2 * kHalfG;
constexpr float kRangeG = 30.f;  // log2 units a logit may pass its row's m by
constexpr int kORowG = kDg + 4;  // floats of an output row in shared memory

template <bool PRECISE>
struct SmemG {
  static constexpr int kStagesK = PRECISE ? 1 : 3, kStagesV = 2;
  static constexpr int kParts = PRECISE ? 3 : 1;         // of P: the first over the K tile
  static constexpr int kK = kTileG;                      // after Q
  static constexpr int kV = kK + kStagesK * kTileG;
  static constexpr int kPlo = kV + kStagesV * kTileG;
  static constexpr int kOnes = kPlo + (kParts - 1) * kTileG; // 16 x 128 ones, in two halves of 64 keys
  static constexpr int kTok = kOnes + 4096;                  // [2][128]: tokens of a tile's keys, -1 for none
  static constexpr int kScale = kTok + 2 * kKeysG * 4;       // [2][128]: their (K, V) scales
  static constexpr int kSeen = kScale + 2 * kKeysG * 8;      // [4 tiles][4]: bit c of word w: key 32w + c is a token
  static constexpr int kMove = kSeen + 4 * 4 * 4;            // [2 tiles][8 warps]: a row of the warp leaves its range
  static constexpr int kMl = kMove + 2 * 8 * 4;              // [2][128] floats of the rows' halves, [128] (m, l)
  // k_full[3] k_empty[3] v_full[2] v_empty[2] s_full[2] s_free[2] p_full[2] o_done[4] q_full
  static constexpr int kBar = kMl + 2 * kQ8RowTile * 8;
  static constexpr int kSlot = kBar + 8 * 21;
  static constexpr size_t kBytes = 1024 + kSlot + 16;
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kQ8RowTile * kORowG * 4 <= kTok, "the output rows fit over Q and the stages");
};

// two floats at once
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Operand tiles are only ever read by the MMAs, behind a fence: no "memory"
// clobber, so that other shared-memory loads may pass these stores.
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

// Waits for the TMEM loads so far; the values of v are used only behind it.
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// One column of TMEM: 32 lanes, one value each.
__device__ __forceinline__ float tmem_get(uint32_t at) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(v) : : "memory");
  return __uint_as_float(v);
}
__device__ __forceinline__ void tmem_set(uint32_t at, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(__float_as_uint(v)) : "memory");
}

// Both phases, by every lane: no broadcast, and most often no wait.
__device__ __forceinline__ bool warp_wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
  const bool ready = mbar_try_wait(a, pa) & mbar_try_wait(b, pb);
  if (__all_sync(0xffffffffu, ready)) return true;
  const bool ok = mbar_wait(a, pa, kWaitLimitNs) && mbar_wait(b, pb, kWaitLimitNs);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool warp_wait_g(uint64_t* bar, uint32_t parity) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, kWaitLimitNs);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// 16 codes (dims 16c ..) of key row r times their scale as bf16 into a
// [128, 128] tile at `tile` (a half row is 64 dims).  The 8 lanes of a store
// phase hold pieces 0-3 of one row and 4-7 of its neighbour: different banks.
__device__ __forceinline__ void store_codes(uint32_t tile, int r, int c, const uint4& v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint64_t sc = pair(scale, scale);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo, hi;
    q8_to_half4(w[i], lo, hi);
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const float2 g0 = unpair(mul2(pair(f0.x, f0.y), sc)), g1 = unpair(mul2(pair(f1.x, f1.y), sc));
    b[2 * i] = pack_bf16(g0.x, g0.y);
    b[2 * i + 1] = pack_bf16(g1.x, g1.y);
  }
  const uint32_t base = tile + (c >> 2) * kHalfG;
  sts16(base + sw128_offset(r, (c & 3) * 2), b[0], b[1], b[2], b[3]);
  sts16(base + sw128_offset(r, (c & 3) * 2 + 1), b[4], b[5], b[6], b[7]);
}

// dims 4 * lane .. of a query row's output
__device__ __forceinline__ void store_row(const Q8AttnArgs& a, int b, int g, int row, int lane, const float4& v) {
  const int64_t off = (((int64_t)(row / a.G) * a.B + b) * a.Hq + g * a.G + row % a.G) * kDg + 4 * lane;
  if (a.out_f32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.O) + off) = v;
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.O) + off) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <bool PRECISE>
__global__ void __launch_bounds__(kThreadsG, 1) attn_q8_group_kernel(const Q8AttnArgs a, const int row_tiles) {
  using Lay = SmemG<PRECISE>;
  constexpr int SK = Lay::kStagesK, SV = Lay::kStagesV;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, not a rounded address: the compiler then knows it for shared
  // memory; generic loads would queue behind the global ones)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint32_t* seen_s = reinterpret_cast<uint32_t*>(smem + Lay::kSeen);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Lay::kBar);
  uint64_t* k_empty = k_full + 3;
  uint64_t* v_full = k_empty + 3;
  uint64_t* v_empty = v_full + 2;
  uint64_t* s_full = v_empty + 2;
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
  const int64_t part = (int64_t)unit * a.n_split + slice;

  pdl_trigger();
  if (warp == kMmaWarp) {
    tmem_alloc(slot, 512);
    if (lane == 0) {
      for (int i = 0; i < 3; ++i) {
        mbar_init(&k_full[i], kProdWarps);
        mbar_init(&k_empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&v_full[i], kProdWarps);
        mbar_init(&v_empty[i], 1);
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
  const int e_beg = (int)min((int64_t)n_keys, (int64_t)slice * a.chunk), 
            e_end = (int)min((int64_t)n_keys, (int64_t)e_beg + a.chunk);
  const int nt = (e_end - e_beg + kKeysG - 1) / kKeysG;
  // every role meets here once its first loads are on their way: barriers and TMEM are ready
  auto ready = [] {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };

  if (warp >= kProdWarp) {
    // =============== producers ===============
    const int pt = tid - kProdWarp * 32;
    const int pc = pt & 7, pr = (pt >> 3) ^ (pc >> 2);  // rows pr + kRowStep i, 16-byte piece pc
    const int64_t row0 = s.off * a.Hkv + (int64_t)g * s.cap;
    int* tok_s = reinterpret_cast<int*>(smem + Lay::kTok);
    float2* scale_s = reinterpret_cast<float2*>(smem + Lay::kScale);
    // this thread's key of tile j: its token as listed (it loads the key's scales too)
    // (an index's entries need nothing of the sequence: their loads do not wait for it)
    const int64_t first = (int64_t)slice * a.chunk + pt;
    const int64_t end = pt < kKeysG ? min((int64_t)(a.idx ? a.k : s.len), (int64_t)(slice + 1) * a.chunk) : 0;
    auto token = [&](int j) -> int {
      const int64_t e = first + j * kKeysG;
      if (e >= end) return -1;
      return a.idx ? __ldcg(&a.idx[(int64_t)b * a.k + e]) : (int)e;
    };
    auto sync = [] { asm volatile("bar.sync 2, %0;" ::"n"(32 * kProdWarps) : "memory"); };
    auto fetch = [&](const uint8_t* codes, int j, uint4 (&v)[kPer]) {
      const uint8_t* from = codes + row0 * kDg + pc * 16;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int t = tok_s[(j & 1) * kKeysG + pr + kRowStep * i];
        v[i] = make_uint4(0, 0, 0, 0);
        if (t >= 0) v[i] = __ldcg(reinterpret_cast<const uint4*>(from + (int64_t)t * kDg));
      }
    };
    uint4 kv[kPer], vv[kPer];
    float ks = 0.f, vs = 0.f;
    auto scales = [&](int t) {
      ks = vs = 0.f;
      if (t >= 0 && t < s.len) {
        ks = __ldcg(a.Ks + (row0 + t) / kQ8Block);
        vs = __ldcg(a.Vs + (row0 + t) / kQ8Block);
      }
    };
    int tm = token(0), tm_next = token(1);
    if (pt < kKeysG) tok_s[pt] = tm < s.len ? tm : -1;
    sync();
    fetch(a.K, 0, kv);
    scales(tm);
    fetch(a.V, 0, vv);
    ready();
    bool dead = false;
    for (int j = 0; j < nt; ++j) {
      const int sk = j % SK, sv = j % SV;
      if (tm >= s.len) {
        if (g == 0 && rt == 0)
          report(a.status, kErrDevice, kKernAttnQ8, (int64_t)b * a.k + e_beg + j * kKeysG + pt, tm, s.len);
        tm = -1;
      }
      if (pt < kKeysG) scale_s[(j & 1) * kKeysG + pt] = make_float2(ks, vs);
      const uint32_t seen = __ballot_sync(0xffffffffu, tm >= 0);
      if (!dead && j >= SK && !warp_wait_g(&k_empty[sk], (j / SK - 1) & 1)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 0, j);
        dead = true;  // only meets the other producers from here on
      }
      if (pt < kKeysG && lane == 0 && !dead) seen_s[(j & 3) * 4 + (pt >> 5)] = seen;
      tm = tm_next;
      if (pt < kKeysG) tok_s[((j + 1) & 1) * kKeysG + pt] = tm < s.len ? tm : -1;
      sync();
      if (dead) continue;
      const float2* sc = scale_s + (j & 1) * kKeysG + pr;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        store_codes(sbase + Lay::kK + sk * kTileG, pr + kRowStep * i, pc, kv[i], sc[kRowStep * i].x);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[sk]);
      fetch(a.K, j + 1, kv);
      scales(tm);
      tm_next = token(j + 2);
      if (j >= SV && !warp_wait_g(&v_empty[sv], (j / SV - 1) & 1)) {
        if (lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 3, j);
        dead = true;
        continue;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        store_codes(sbase + Lay::kV + sv * kTileG, pr + kRowStep * i, pc, vv[i], sc[kRowStep * i].y);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[sv]);
      fetch(a.V, j + 1, vv);
    }
  } else if (warp == kMmaWarp) {
    // =============== MMA issuer ===============
    ready();
    // The whole warp stays together and one elected lane issues: operands of a
    // product are then known to be one value per warp.
    const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
    const bool lead = elect_one();
    auto wait = [](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitLimitNs));
    };
    if (nt > 0) {
      constexpr uint32_t idesc_qk = umma_idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_l = umma_idesc_bf16(128, 16, false, false);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(128, 128, false, true);
      auto pv = [&](int i) -> bool {
        if (!wait(&v_full[i % SV], (i / SV) & 1) || !wait(&p_full[i & 1], (i >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t pst = sbase + Lay::kK + i % SK * kTileG;  // P lives here now
        const uint32_t vst = sbase + Lay::kV + i % SV * kTileG;
        if (lead) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // keys 64h + 16kk ..
              const uint64_t vd = umma_desc_sw128(vst + h * 8192 + kk * 2048, kHalfG, 1024);
#pragma unroll
              for (int q = 0; q < Lay::kParts; ++q) {
                const uint64_t pd = umma_desc_sw128(
                    (q == 0 ? pst : sbase + Lay::kPlo + (q - 1) * kTileG) + h * kHalfG + kk * 32, 16, 1024);
                umma_bf16(tmem + 256, pd, vd, idesc_pv, (i | h | kk | q) != 0);
                umma_bf16(tmem + 384, pd, umma_desc_sw128(sbase + Lay::kOnes + h * 2048 + kk * 32, 16, 1024), idesc_l,
                          (i | h | kk | q) != 0);
              }
            }
          umma_commit(&k_empty[i % SK]);
          umma_commit(&v_empty[i % SV]);
          umma_commit(&o_done[i & 3]);
        }
        __syncwarp();
        return true;
      };
      bool ok = wait(q_full, 0);
      for (int j = 0; j < nt && ok; ++j) {
        if (PRECISE && j >= 1 && !(ok = pv(j - 1))) break;  // the next K tile follows it
        ok = wait(&k_full[j % SK], (j / SK) & 1) && wait(&s_free[j & 1], ((j >> 1) & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t kst = sbase + Lay::kK + j % SK * kTileG;
        if (lead) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_bf16(tmem + (j & 1) * 128, umma_desc_sw128(sbase + h * kHalfG + kk * 32, 16, 1024),
                        umma_desc_sw128(kst + h * kHalfG + kk * 32, 16, 1024), idesc_qk, (h | kk) != 0);
          umma_commit(&s_full[j & 1]);
        }
        __syncwarp();
        if (!PRECISE && j >= 1) ok = pv(j - 1);
      }
      if (ok) ok = pv(nt - 1);
      if (!ok && lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 1, 0);
    }
  } else {
    // =============== queries, then softmax ===============
    {
      const int r = tid >> 1, qh = tid & 1;  // half a query row: dims 64 qh ..
      const int row = row_base + r;
      uint4 qv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) qv[i] = make_uint4(0, 0, 0, 0);
      if (row < a.R) {
        const int64_t off = (((int64_t)(row / a.G) * a.B + b) * a.Hq + g * a.G + row % a.G) * kDg + 64 * qh;
#pragma unroll
        for (int i = 0; i < 8; ++i) qv[i] = __ldcg(reinterpret_cast<const uint4*>(a.Q + off) + i);
      }
      ready();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sts16(sbase + qh * kHalfG + sw128_offset(r, i), qv[i].x, qv[i].y, qv[i].z, qv[i].w);
      sts16(sbase + Lay::kOnes + 16 * tid, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const uint32_t tmem = *slot;
    const int half = warp >> 2;
    const int r_loc = (warp & 3) * 32 + lane;
    const bool active = row_base + (warp & 3) * 32 < a.R;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tmem_o = tmem + 256 + 64 * half + lane_base;  // this thread's columns of O
    const uint32_t tmem_l = tmem + 384 + lane_base;
    volatile float* up_s = reinterpret_cast<volatile float*>(smem + Lay::kMl) + r_loc;  // [2][128], by half
    volatile uint32_t* move_s = reinterpret_cast<volatile uint32_t*>(smem + Lay::kMove);  // [2 tiles][8 warps]
    auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(3 + (warp & 3)) : "memory"); };  // the rows' two warps
    const uint64_t scale2 = pair(a.scale_log2, a.scale_log2);
    float m = -INFINITY;
    // a wait that gave up: the warp goes on without waiting (on garbage, which
    // the status tells), so that no other warp waits for it at a barrier
    bool failed = false;
    for (int j = 0; j < nt; ++j) {
      if (!failed) failed = !warp_wait_both(&s_full[j & 1], (j >> 1) & 1, &k_full[j % SK], (j / SK) & 1);
      tc_fence_after();
      const uint32_t* seen = seen_s + (j & 3) * 4;
      const uint32_t* vis = seen + 2 * half;
      if (active) {
        const uint32_t tmem_s = tmem + (j & 1) * 128 + 64 * half + lane_base;
        uint32_t sa[16], sb[16];
        tmem_ld16(tmem_s, sa);
        const uint32_t vis0 = vis[0], vis1 = vis[1];
        const bool all = (vis0 & vis1) == 0xffffffffu;
        const uint32_t pst = sbase + Lay::kK + j % SK * kTileG + half * kHalfG + r_loc * 128;
        const uint32_t plo = sbase + Lay::kPlo + half * kHalfG + r_loc * 128;
        if (__any_sync(0xffffffffu, m == -INFINITY) && (seen[0] | seen[1] | seen[2] | seen[3])) {
          // the rows' first key: their reference
          int c = 0;
          while (seen[c] == 0u) ++c;
          const float z = tmem_get(tmem_s - 64 * half + 32 * c + __ffs(seen[c]) - 1) * a.scale_log2;
          if (m == -INFINITY) m = fabsf(z) < 1e30f ? z : 0.f;
        }
#pragma unroll 1
        for (int tries = 0; tries < 2; ++tries) {
          const float neg_m = m == -INFINITY ? 0.f : -m;
          const uint64_t neg2 = pair(neg_m, neg_m);
          float top[2] = {-INFINITY, -INFINITY};
          auto weights = [&](uint32_t (&sv)[16], int c) {  // of keys 16c .. of this half
            if (!all) {
              const uint32_t see = (c < 2 ? vis0 : vis1) >> (16 * (c & 1));
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!(see >> e & 1u)) sv[e] = 0xff800000u;  // -inf
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // 8 keys: one 16-byte chunk of the row's P
              float2 y[4];
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int at = 8 * q + 2 * i;
                const float2 x = unpair(fma2(pair(__uint_as_float(sv[at]), __uint_as_float(sv[at + 1])), scale2, neg2));
                top[i & 1] = fmaxf(fmaxf(x.x, x.y), top[i & 1]);
                y[i] = make_float2(ex2f(x.x), ex2f(x.y));
                h[i] = pack_bf16(y[i].x, y[i].y);
              }
              const uint32_t off = (uint32_t)((2 * c + q) ^ (r_loc & 7)) << 4;
              sts16(pst + off, h[0], h[1], h[2], h[3]);
              if (PRECISE) {
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // what the parts before leave
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    y[i] = make_float2(y[i].x - bf_lo(h[i]), y[i].y - bf_hi(h[i]));
                    h[i] = pack_bf16(y[i].x, y[i].y);
                  }
                  sts16(plo + part * kTileG + off, h[0], h[1], h[2], h[3]);
                }
              }
            }
          };
          // a load of TMEM takes about as long as 16 keys' weights: one ahead
          if (tries) tmem_ld16(tmem_s, sa);
          tmem_wait(sa);
          tmem_ld16(tmem_s + 16, sb);
          weights(sa, 0);
          tmem_wait(sb);
          tmem_ld16(tmem_s + 32, sa);
          weights(sb, 1);
          tmem_wait(sa);
          tmem_ld16(tmem_s + 48, sb);
          weights(sa, 2);
          tmem_wait(sb);
          weights(sb, 3);
          if (tries) break;
          const float mine = fmaxf(top[0], top[1]);
          const bool move = __any_sync(0xffffffffu, mine > kRangeG);
          if (lane == 0) move_s[(j & 1) * 8 + warp] = move;
          meet();
          if (!move && !move_s[(j & 1) * 8 + (warp ^ 4)]) break;
          // ---- some row's logits have left the range of its m: its sums move ----
          up_s[half * kQ8RowTile] = mine;
          meet();
          const float up = fmaxf(mine, up_s[(half ^ 1) * kQ8RowTile]);
          const float alpha = up > kRangeG ? ex2f(-up) : 1.f;
          if (up > kRangeG) m += up;
          if (j > 0) {
            // the last tile's PV must have landed before O is rescaled
            if (!failed) failed = !warp_wait_g(&o_done[(j - 1) & 3], ((j - 1) >> 2) & 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              uint32_t ov[16];
              tmem_ld16(tmem_o + c, ov);
              tmem_wait(ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st16(tmem_o + c, ov);
            }
            if (half == 0) tmem_set(tmem_l, tmem_get(tmem_l) * alpha);
            tmem_wait_st();
          }
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_free[j & 1]);
        mbar_arrive(&p_full[j & 1]);
      }
    }
    // ---- the row's (m, l, o / l) into shared memory ----
    if (nt > 0 && !failed) failed = !warp_wait_g(&o_done[(nt - 1) & 3], ((nt - 1) >> 2) & 1);
    if (failed && lane == 0) report(a.status, kErrTimeout, kKernAttnQ8, blockIdx.x, 2, warp);
    tc_fence_after();
    // every MMA is done (the barrier below): Q and the stages are free for the rows
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float L = active && nt > 0 ? tmem_get(tmem_l) : 0.f;
    const float f = L == 0.f ? 0.f : 1.f / L;
    if (active && nt > 0) {
      float* dst = reinterpret_cast<float*>(smem) + r_loc * kORowG + 64 * half;  // [128][kORowG]
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        uint32_t oa[16], ob[16];
        tmem_ld16(tmem_o + c, oa);
        tmem_ld16(tmem_o + c + 16, ob);
        tmem_wait(oa);
        tmem_wait(ob);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          *reinterpret_cast<float4*>(dst + c + e) =
              make_float4(__uint_as_float(oa[e]) * f, __uint_as_float(oa[e + 1]) * f, __uint_as_float(oa[e + 2]) * f,
                          __uint_as_float(oa[e + 3]) * f);
          *reinterpret_cast<float4*>(dst + c + 16 + e) =
              make_float4(__uint_as_float(ob[e]) * f, __uint_as_float(ob[e + 1]) * f, __uint_as_float(ob[e + 2]) * f,
                          __uint_as_float(ob[e + 3]) * f);
        }
      }
    }
    if (half == 0) reinterpret_cast<float2*>(smem + Lay::kMl)[kQ8RowTile + r_loc] = make_float2(m, L);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(*slot, 512);
  }
  const int rows = min(kQ8RowTile, a.R - row_base);
  if (a.cluster) {
    // ---- the slices' rows: this CTA merges every a.cluster-th part of them ----
    if (a.cluster > 1) cluster_sync();  // every slice's rows are in its shared memory
    const int n = a.cluster, per = kQ8RowTile / n;
    const uint32_t ml_at = smem_u32(smem + Lay::kMl) + kQ8RowTile * 8;
    for (int r = slice * per + warp; r < min(rows, (slice + 1) * per); r += kThreadsG / 32) {
      // every load before the first use, four slices at a time: a peer's
      // memory is several hundred cycles away
      float2 ml[8];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ml[i] = i < n ? ld_peer2(ml_at + r * 8, i) : make_float2(-INFINITY, 0.f);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += 4) {
        if (i0 >= n) break;
        const uint32_t at = sbase + (r * kORowG + 4 * lane) * 4;
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int from = min(i0 + i, n - 1);
          x[i] = ld_peer4(at, from);
        }
        if (i0 == 0)
#pragma unroll
          for (int i = 0; i < 8; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = (ml[i0 + i].x == -INFINITY ? 0.f : ex2f(ml[i0 + i].x - M)) * ml[i0 + i].y;
          L += w;
          if (w != 0.f) {  // else that slice has no row there
            acc.x += w * x[i].x, acc.y += w * x[i].y;
            acc.z += w * x[i].z, acc.w += w * x[i].w;
          }
        }
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      store_row(a, b, g, row_base + r, lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
    if (a.cluster > 1) cluster_sync();  // no CTA leaves while its rows are read
    return;
  }
  const float2* ml_s = reinterpret_cast<const float2*>(smem + Lay::kMl) + kQ8RowTile;
  if (tid < rows) __stcg(&a.pml[part * kQ8RowTile + tid], ml_s[tid]);
  if (nt > 0) {
    const float* o_s = reinterpret_cast<const float*>(smem);
    float4* dst = reinterpret_cast<float4*>(a.po + part * kQ8RowTile * kDg);
    for (int i = tid; i < rows * (kDg / 4); i += kThreadsG) {
      const float* at = o_s + i / (kDg / 4) * kORowG + i % (kDg / 4) * 4;
      __stcg(dst + i, *reinterpret_cast<const float4*>(at));
    }
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
  store_row(a, b, g, row, lane, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

}  // namespace

// One CTA per SM and one wave, at most the 128-key tiles there are.  A cluster
// of 1, 2, 4 or 8 slices merges in shared memory; more slices only where the
// cluster's would be longer than four tiles.  A cluster takes whole SMs of one
// GPC: 15 of 8 and 33 of 4 CTAs run at once on 148 SMs (16 of 8 take 22.7 us
// where 8 take 14.1).
void plan_attn_q8_group(Q8AttnPlan& p, int64_t n, int sms) {
  const int64_t tiles = n > 0 ? (n + kKeysG - 1) / kKeysG : 1;
  const int cluster = p.units <= sms / 10 ? 8 : p.units <= 2 * sms / 9 ? 4 : p.units <= sms / 2 ? 2 : 1;
  p.cluster = cluster;
  while (p.cluster > 1 && p.cluster / 2 >= tiles) p.cluster /= 2;
  int64_t split = sms / p.units > 1 ? sms / p.units : 1;
  if (split > tiles) split = tiles;
  if (split > cluster && tiles > 4 * cluster)
    p.cluster = 0;
  else
    split = p.cluster;
  p.chunk = (int)((tiles + split - 1) / split) * kKeysG;
  p.n_split = p.cluster ? p.cluster : (int)((tiles * kKeysG + p.chunk - 1) / p.chunk);
  p.parts = p.cluster ? 0 : p.n_split;
  p.rows = kQ8RowTile;
}

cudaError_t launch_attn_q8_group(const Q8AttnArgs& a, const Q8AttnPlan& p, cudaStream_t stream) {
  auto kern = a.out_f32 ? attn_q8_group_kernel<true> : attn_q8_group_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.units * p.n_split));
  cfg.blockDim = dim3(kThreadsG);
  cfg.dynamicSmemBytes = a.out_f32 ? SmemG<true>::kBytes : SmemG<false>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster ? p.cluster : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = ensure_smem(kern, cfg.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, kern, a, p.row_tiles);
  if (e != cudaSuccess || p.cluster) return e != cudaSuccess ? e : cudaGetLastError();
  const int n_rows = a.B * a.Hkv * a.R;
  cfg.gridDim = dim3((unsigned)((n_rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_q8_merge_kernel, a, p.row_tiles, n_rows);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sa
