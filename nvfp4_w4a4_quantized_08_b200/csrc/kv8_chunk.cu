// kv8_chunk.cu -- attention of many rows per request over the paged 8-bit cache, on the
// sm_100a tensor cores (chunks of new tokens, prompts).
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k[j]) v[j],  k = codes * page scale
//
// Bound by the softmax (one exponential for each row and token: 16 a clock and SM) and the
// tensor core (bf16 S = Q K^T and P V), which take about the same time per tile of 128 x
// 128; so both have to run all the time.  One CTA of 16 warps takes 256 packed rows (two
// tiles of 128) of one request and KV head and a range of its tokens:
//   warps 0..7   softmax: warpgroup g owns row tile g, one row a thread.  A row's 128
//                scores of a tile are read from tensor memory once, into registers
//                (200 a thread, moved over from the other warps by setmaxnreg); the
//                probabilities go back as bf16, in two halves, so that P V starts on the
//                first while the second is computed.
//   warps 8..11  decoders: E4M3 codes -> bf16 K and V operands in 128-byte-swizzled shared
//                memory (two stages each).  A code is shifted into place and multiplied by
//                2^120, two at a time: exact.  The order of 8 dims is the one in which that
//                needs no byte permutes (0 2 1 3 4 6 5 7); Q is stored in the same order, the
//                output is read in it.  Every byte decodes to something finite, so tokens past
//                the end need no clearing: their probabilities are 0.
//   warp 12      issues the MMAs: ... PV0_j, S0_{j+1}, PV1_j, S1_{j+1}, PV0_{j+1} ..., so
//                the tensor core works on one row tile while the other's softmax runs.
//   warp 13      copies the codes of a tile ahead (one bulk copy for the 16 tokens of a group,
//                which share a page).
// Tensor memory (512 columns): O0, O1, S0, S1; P_g takes S_g's place.
//
// The codes go into the products without their page scales.  Scores of a group of 16 tokens
// are multiplied by the page's K scale in fp32; its V scale is an exponent added to the
// probabilities' (P is bf16, which holds it), and the normaliser takes the group's sum times
// 2^-exponent: exact, and one multiplication a group.  The running maximum is raised lazily:
// only a step of more than 2^16 rescales O and the sum.
//
// Every wait is bounded: one that runs out records NVFP4_ERR_TIMEOUT in the status word, and
// the CTA drains its MMAs, frees tensor memory and returns.
#include "common.cuh"
#include "kernels.h"
#include "kv8_batch.cuh"
#include "tc.cuh"

namespace nvfp4 {
namespace kv8_chunk {

using namespace tc;
using kv8::Args;
using kv8::Request;

constexpr int kRows = 128;                 // rows of a tile
constexpr int kTiles = 2;                  // row tiles of a CTA
constexpr int kKeys = 128;                 // tokens of a tile
constexpr int kGroups = kKeys / 16;        // groups of tokens that share a page
constexpr int kSoftWarps = 8;              // warps 0..7
constexpr int kDecWarps = 4;               // warps 8..11
constexpr int kMmaWarp = kSoftWarps + kDecWarps;
constexpr int kThreads = 512;              // four warpgroups; the last has the MMA warp only
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr int kStages = 2;                 // decoded tiles of K, and of V
constexpr int kMetaStages = 4;             // page scales: read later than K
constexpr int kMetaFloats = 3 * kGroups;
// registers a thread at launch, and after the warpgroups have shared them out anew
constexpr int kLaunchRegs = 128, kSoftRegs = 200, kDecRegs = 56, kMmaRegs = 56;
static_assert(2 * kSoftRegs + kDecRegs + kMmaRegs == 4 * kLaunchRegs, "register split");
static_assert(kThreads * kLaunchRegs <= 65536, "registers of an SM");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol0 = 0, kSCol0 = 256;   // O_g at 128 g, S_g (then P_g) at 256 + 128 g
constexpr float kLazyLog2 = 16.0f;

template <int kD>
struct Layout {
  static constexpr int kChunks = kD / 64;
  static constexpr int kOp = kChunks * kChunkBytes;        // 128 rows x kD bf16
  static constexpr int kQ = 0, kK = kTiles * kOp, kV = kK + kStages * kOp;
  static constexpr int kRaw = kD == 64 ? 3 : 1;            // tiles of codes ahead
  static constexpr int kRawBytes = kKeys * kD;             // of one plane
  static constexpr int kRawK = kV + kStages * kOp, kRawV = kRawK + kRaw * kRawBytes;
  static constexpr int kMeta = kRawV + kRaw * kRawBytes;   // [stage][3][group] floats
  static constexpr int kBar = kMeta + kMetaStages * kMetaFloats * 4;
  // q[2], k_full, k_empty, v_full, v_empty [stage], s_full[2], p_ready[2][2], pv_done[2],
  // meta_full[4], raw K full, empty, raw V full, empty [raw stage], o_full, drain
  static constexpr int kNumBars = 2 + 4 * kStages + 2 + 4 + 2 + kMetaStages + 4 * kRaw + 2;
  static constexpr int kTmemPtr = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemPtr + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

// kind::f16: fp32 D (bit 4), bf16 A and B (bits 7 and 10), N >> 3 at 17, M >> 4 at 24; B
// MN-major: bit 16.
__host__ __device__ constexpr uint32_t idesc(uint32_t n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
}

// Four E4M3 bytes -> bf16 of bytes (0, 2) and (1, 3): sign and the 7 other bits into place,
// which is the value times 2^-120 (subnormals too), then times 2^120.
__device__ __forceinline__ uint2 decode4(uint32_t w) {
  uint32_t lo = ((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u);
  uint32_t hi = ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u);
  const uint32_t k120 = 0x7B807B80u;
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(k120));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(k120));
  return make_uint2(lo, hi);
}

template <int kRegs>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// All 128 columns of a thread's row.
__device__ __forceinline__ void load_scores(uint32_t addr, uint32_t (&r)[4][32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32_async(addr + 32 * c, r[c]);
  tmem_wait_ld(r[0], r[1]);
  regs_after_wait(r[2]);
  regs_after_wait(r[3]);
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Args a) {
  using L = Layout<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_q = sbase + L::kBar;                      // + 8 g
  const uint32_t bar_k_full = bar_q + 8 * kTiles;              // + 8 stage
  const uint32_t bar_k_empty = bar_k_full + 8 * kStages;
  const uint32_t bar_v_full = bar_k_empty + 8 * kStages;
  const uint32_t bar_v_empty = bar_v_full + 8 * kStages;
  const uint32_t bar_s_full = bar_v_empty + 8 * kStages;       // + 8 g
  const uint32_t bar_p_ready = bar_s_full + 8 * kTiles;        // + 16 g + 8 half
  const uint32_t bar_pv_done = bar_p_ready + 16 * kTiles;      // + 8 g
  const uint32_t bar_meta = bar_pv_done + 8 * kTiles;          // + 8 stage
  const uint32_t bar_rk_full = bar_meta + 8 * kMetaStages;     // + 8 raw stage
  const uint32_t bar_rk_empty = bar_rk_full + 8 * L::kRaw;
  const uint32_t bar_rv_full = bar_rk_empty + 8 * L::kRaw;
  const uint32_t bar_rv_empty = bar_rv_full + 8 * L::kRaw;
  const uint32_t bar_o_full = bar_rv_empty + 8 * L::kRaw;
  const uint32_t bar_drain = bar_o_full + 8;
  uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + L::kTmemPtr);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  float* meta = reinterpret_cast<float*>(smem + L::kMeta);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the row tiles with the most tokens to see come first
  const int h = blockIdx.x % a.kv_heads, b = blockIdx.y, split = blockIdx.z;
  const int tile = int(gridDim.x) / a.kv_heads - 1 - int(blockIdx.x) / a.kv_heads;

  if (threadIdx.x == 0) {
    for (int g = 0; g < kTiles; ++g) {
      bar_init(bar_q + 8 * g, 4);
      bar_init(bar_s_full + 8 * g, 1);
      bar_init(bar_p_ready + 16 * g, 4);
      bar_init(bar_p_ready + 16 * g + 8, 4);
      bar_init(bar_pv_done + 8 * g, 1);
    }
    for (int s = 0; s < kStages; ++s) {
      bar_init(bar_k_full + 8 * s, kDecWarps);
      bar_init(bar_k_empty + 8 * s, 1);
      bar_init(bar_v_full + 8 * s, kDecWarps);
      bar_init(bar_v_empty + 8 * s, 1);
    }
    for (int s = 0; s < kMetaStages; ++s) bar_init(bar_meta + 8 * s, 1);
    for (int s = 0; s < L::kRaw; ++s) {
      bar_init(bar_rk_full + 8 * s, 1);
      bar_init(bar_rk_empty + 8 * s, kDecWarps);
      bar_init(bar_rv_full + 8 * s, 1);
      bar_init(bar_rv_empty + 8 * s, kDecWarps);
    }
    bar_init(bar_o_full, 1);
    bar_init(bar_drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_ptr)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_ptr;
  pdl_wait();
  pdl_trigger();
  const Waiter waiter{a.wait_limit_ns, abort_flag, a.status};

  const Request rq = kv8::request(a, b, threadIdx.x == 0 && blockIdx.x == 0 && split == 0);
  const int rows = rq.nq * a.group, base = tile * kRows * kTiles;
  const int used = kv8::splits_of(a, rq.kv);
  // row tiles with rows, tokens of this range that any of them sees
  const int n_q = base >= rows || split >= used ? 0 : rows - base > kRows ? 2 : 1;
  const int t_begin = split * a.chunk;
  const int t_range = split == used - 1 ? rq.kv : min(rq.kv, t_begin + a.chunk);
  const int t_end =
      n_q ? min(t_range, kv8::sees(a, rq, min(base + kTiles * kRows, rows) - 1)) : t_begin;
  const int n_tiles = max(0, (t_end - t_begin + kKeys - 1) / kKeys);

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    more_regs<kSoftRegs>();
    const uint32_t g = uint32_t(warp) >> 2, quad = uint32_t(warp) & 3;
    const uint32_t row = quad * 32 + uint32_t(lane);
    const uint32_t o_addr = tmem + ((quad * 32) << 16) + kOCol0 + 128 * g;
    const uint32_t s_addr = tmem + ((quad * 32) << 16) + kSCol0 + 128 * g;
    const int rho = base + int(g) * kRows + int(row);
    const bool live = int(g) < n_q && rho < rows;
    // tokens of the range that this row sees (dead rows follow the last live one)
    const int vis = min(t_range, kv8::sees(a, rq, max(0, min(rho, rows - 1)))) - t_begin;
    const int vis_min = __reduce_min_sync(0xFFFFFFFFu, vis);
    bool ok = true;
    float m_run = -INFINITY, l_run = 0.0f;
    if (int(g) < n_q && n_tiles > 0) {
      // Q row -> shared memory in the dims' order of the decoders
      const uint4* src =
          reinterpret_cast<const uint4*>(live ? kv8::q_row(a, rq, h, rho, kD) : a.q);
      const uint32_t qs = sbase + L::kQ + g * L::kOp;
#pragma unroll 4
      for (uint32_t u = 0; u < kD / 8; ++u) {
        uint4 v = live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
        v = make_uint4(prmt(v.x, v.y, 0x5410), prmt(v.x, v.y, 0x7632), prmt(v.z, v.w, 0x5410),
                       prmt(v.z, v.w, 0x7632));
        st_shared_v4(qs + op_offset(row, u), v);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(bar_q + 8 * g);
      for (int j = 0; j < n_tiles; ++j) {
        ok = __all_sync(0xFFFFFFFFu, waiter.wait(bar_meta + 8 * (j % kMetaStages),
                                                 (j / kMetaStages) & 1));
        if (!ok) break;
        // per group: K scale times scale * log2 e; log2 of the V scale; 1 / V scale (0: no
        // page, left out)
        const float* ms = meta + (j % kMetaStages) * kMetaFloats;
        float sc[kGroups];
#pragma unroll
        for (int n = 0; n < kGroups; ++n) sc[n] = ms[n];
        ok = __all_sync(0xFFFFFFFFu, waiter.wait(bar_s_full + 8 * g, j & 1));
        if (!ok) break;
        tc_fence_after();
        uint32_t r[4][32];
        load_scores(s_addr, r);
        if (vis_min < (j + 1) * kKeys) {
          const int left = vis - j * kKeys;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= left) r[c][e] = 0xFF800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
          const uint32_t* s = &r[n >> 1][16 * (n & 1)];
          float t0 = __uint_as_float(s[0]), t1 = __uint_as_float(s[1]);
#pragma unroll
          for (int e = 2; e < 16; e += 4) {
            t0 = max3f(t0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
            if (e + 2 < 16)
              t1 = max3f(t1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
          }
          // (the scales are positive; a group of no page is left out)
          const float t = fmaxf(t0, t1) * sc[n];
          mx = fmaxf(mx, ms[2 * kGroups + n] == 0.0f ? -INFINITY : t);
        }
        float factor = 1.0f;
        if (mx > m_run + kLazyLog2) {
          factor = exp2_approx(m_run - mx);   // 0 on the first tokens
          m_run = mx;
          l_run *= factor;
        }
        if (__any_sync(0xFFFFFFFFu, factor != 1.0f) && j > 0) {
          // tile j - 1's P V is complete, since S of tile j is
          ok = __all_sync(0xFFFFFFFFu, waiter.wait(bar_pv_done + 8 * g, (j - 1) & 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (uint32_t c = 0; c < kD / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(o_addr + 16 * c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
            tmem_st16(o_addr + 16 * c, o);
          }
        }
        const float neg_m = m_run == -INFINITY ? 0.0f : -m_run;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float scn = sc[2 * c + n], off = ms[kGroups + 2 * c + n] + neg_m;
            const float2 sc2 = make_float2(scn, scn), of2 = make_float2(off, off);
            const float2 one2 = make_float2(1.0f, 1.0f);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[c][16 * n + 2 * e]),
                                                      __uint_as_float(r[c][16 * n + 2 * e + 1])),
                                          sc2, of2);
              const float2 p = make_float2(exp2_approx(x.x), exp2_approx(x.y));
              sum = __ffma2_rn(p, one2, sum);
              pk[8 * n + e] = kv8::bf16x2(p.x, p.y);
            }
            l_run = fmaf(sum.x + sum.y, ms[2 * kGroups + 2 * c + n], l_run);
          }
          tmem_st16(s_addr + 16 * c, pk);
          if (c & 1) {
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar_p_ready + 16 * g + 8 * (c >> 1));
          }
        }
      }
      if (ok) ok = __all_sync(0xFFFFFFFFu, waiter.wait(bar_o_full, 0));
      tc_fence_after();
    }
    // ---- O / l -> the output or the range's part; a row that saw nothing is zero
    if (ok && int(g) < n_q) {
      const float norm = l_run == 0.0f ? 0.0f : 1.0f / l_run;
      const float lse2 = l_run == 0.0f ? -INFINITY : m_run + log2f(l_run);
#pragma unroll 1
      for (uint32_t c = 0; c < kD / 16; ++c) {
        uint32_t o[16];
        if (n_tiles > 0) {
          tmem_ld16(o_addr + 16 * c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          // dims 1 and 2, 5 and 6 of every 8 change places
          const int from = (e & 3) == 1 ? e + 1 : (e & 3) == 2 ? e - 1 : e;
          v[e] = l_run == 0.0f ? 0.0f : __uint_as_float(o[from]) * norm;
        }
        if (live) kv8::store_row<16, kD>(a, rq, h, rho, split, used, 16 * c, v, lse2, c == 0);
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ decoders
    fewer_regs<kDecRegs>();
    constexpr int kUnits = kD / 16;                 // 16-byte units of a token
    constexpr int kPer = kDecWarps * 32 / kUnits;   // tokens of a pass
    constexpr int kMine = kKeys / kPer;             // units of a thread and plane
    const uint32_t t = threadIdx.x - kSoftWarps * 32, u = t % kUnits;
    // threads 0..7: the page scales of a tile's groups, read one tile ahead
    const int32_t* table = a.table + int64_t(b) * a.table_stride;
    auto group_page = [&](int j) {
      const int tok = t_begin + j * kKeys + 16 * int(t);
      return t < kGroups && tok < t_end ? __ldg(table + fast_div(a.page_div, uint32_t(tok))) : -1;
    };
    float ks = 0.0f, vs = -1.0f;   // vs < 0: no page
    auto load_scales = [&](int j, int id) {
      vs = -1.0f;
      if (id >= 0 && id < a.n_pages) {
        const int64_t ph = int64_t(id) * a.kv_heads + h;
        ks = __ldg(a.k_scale + ph);
        vs = __ldg(a.v_scale + ph);
      } else if (t < kGroups && t_begin + j * kKeys + 16 * int(t) < t_end) {
        record_status(a.status, NVFP4_ERR_INVALID_ARG);
      }
    };
    // one plane of a tile: codes of raw stage rs -> operand stage st
    auto decode = [&](uint32_t raw, uint32_t op) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "r"(raw + (t + kDecWarps * 32 * i) * 16));
        const uint32_t tok = t / kUnits + kPer * i;
        const uint2 w0 = decode4(w.x), w1 = decode4(w.y), w2 = decode4(w.z), w3 = decode4(w.w);
        const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y);
        const uint4 hi = make_uint4(w2.x, w2.y, w3.x, w3.y);
        // the upper half of the units starts with its second part: other banks
        const bool swap = u >= 4;
        st_shared_v4(op + op_offset(tok, 2 * u + swap), swap ? hi : lo);
        st_shared_v4(op + op_offset(tok, 2 * u + !swap), swap ? lo : hi);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    int next_page = -1;
    if (n_tiles > 0) {
      load_scales(0, group_page(0));
      next_page = group_page(1);
    }
    for (int j = 0; j < n_tiles; ++j) {
      const uint32_t st = j % kStages, empty = ((j / kStages) & 1) ^ 1;
      const uint32_t rs = j % L::kRaw, full = (j / L::kRaw) & 1;
      bool ok = waiter.wait(bar_k_empty + 8 * st, empty) && waiter.wait(bar_rk_full + 8 * rs, full);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      if (t < kGroups) {
        float* m = meta + (j % kMetaStages) * kMetaFloats + t;
        const bool none = vs < 0.0f;
        const float v = fmaxf(vs, 0x1p-60f);   // the smallest scale there is
        const uint32_t bits = __float_as_uint(v);
        m[0] = none ? 1.0f : ks * a.scale_log2;   // (not 0: a masked score is -inf)
        m[kGroups] = none ? -INFINITY
                          : float(int(bits >> 23) - 127) +
                                __log2f(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
        m[2 * kGroups] = none ? 0.0f : 1.0f / v;
      }
      if (warp == kSoftWarps) {
        __syncwarp();
        if (lane == 0) bar_arrive(bar_meta + 8 * (j % kMetaStages));
        if (j + 1 < n_tiles) {
          load_scales(j + 1, next_page);
          next_page = group_page(j + 2);
        }
      }
      decode(sbase + L::kRawK + rs * L::kRawBytes, sbase + L::kK + st * L::kOp);
      if (lane == 0) {
        bar_arrive(bar_rk_empty + 8 * rs);
        bar_arrive(bar_k_full + 8 * st);
      }
      ok = waiter.wait(bar_v_empty + 8 * st, empty) && waiter.wait(bar_rv_full + 8 * rs, full);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      decode(sbase + L::kRawV + rs * L::kRawBytes, sbase + L::kV + st * L::kOp);
      if (lane == 0) {
        bar_arrive(bar_rv_empty + 8 * rs);
        bar_arrive(bar_v_full + 8 * st);
      }
    }
  } else {
    // ------------------------------------------------------------ MMA issuer
    fewer_regs<kMmaRegs>();
    if (warp == kMmaWarp && n_tiles > 0) {
      // the whole warp, so that operands are uniform; one lane issues
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, waiter.wait(bar, parity));
      };
      bool ok = true;
      for (int g = 0; g < n_q && ok; ++g) ok = wait(bar_q + 8 * g, 0);
      // low descriptor words: K-major with LBO 1, MN-major with the chunk stride
      const uint32_t lo_k = ((sbase & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t lo_mn = ((sbase & 0x3FFFFu) >> 4) | (uint32_t(kChunkBytes >> 4) << 16);
      // S_g(j) = Q_g K_j^T: 16 dims a step, +32 bytes, the next chunk after 4
      auto issue_s = [&](uint32_t g, int j) {
        const uint32_t qd = lo_k + ((L::kQ + g * L::kOp) >> 4);
        const uint32_t kd = lo_k + ((L::kK + (j % kStages) * L::kOp) >> 4);
        unrolled(
            [&](auto k) {
              constexpr uint32_t at = (k.value >> 2) * (kChunkBytes >> 4) + 2 * (k.value & 3);
              warp_mma_ss<at, at>(tmem + kSCol0 + 128 * g, qd, kd, idesc(kKeys), k.value != 0);
            },
            std::make_integer_sequence<uint32_t, kD / 16>());
        warp_commit(bar_s_full + 8 * g);
      };
      // O_g += P_g(j) V_j, as the halves of P come: 16 keys a step, 8 columns of P
      auto issue_pv = [&](uint32_t g, int j) {
        const uint32_t vd = lo_mn + ((L::kV + (j % kStages) * L::kOp) >> 4);
        const uint32_t od = tmem + kOCol0 + 128 * g, pd = tmem + kSCol0 + 128 * g;
        if (!wait(bar_p_ready + 16 * g, j & 1)) return false;
        tc_fence_after();
        unrolled(
            [&](auto k) {
              warp_mma_ts<8 * k.value, k.value * (2048 >> 4)>(od, pd, vd, idesc(kD) | (1u << 16),
                                                              k.value != 0 || j != 0);
            },
            std::make_integer_sequence<uint32_t, 4>());
        if (!wait(bar_p_ready + 16 * g + 8, j & 1)) return false;
        tc_fence_after();
        unrolled(
            [&](auto k) {
              warp_mma_ts<32 + 8 * k.value, (4 + k.value) * (2048 >> 4)>(
                  od, pd, vd, idesc(kD) | (1u << 16), 1);
            },
            std::make_integer_sequence<uint32_t, 4>());
        warp_commit(bar_pv_done + 8 * g);
        return true;
      };
      auto ready = [&](uint32_t bar, int j) {
        if (!wait(bar + 8 * (j % kStages), (j / kStages) & 1)) return false;
        tc_fence_after();
        return true;
      };
      if (ok && (ok = ready(bar_k_full, 0))) {
        for (int g = 0; g < n_q; ++g) issue_s(g, 0);
        warp_commit(bar_k_empty);
      }
      for (int j = 0; j < n_tiles && ok; ++j) {
        const bool more = j + 1 < n_tiles;
#pragma unroll 1
        for (int g = 0; g < n_q; ++g) {
          const bool last = g == n_q - 1;
          if (g == 0 && !(ok = ready(bar_v_full, j))) break;
          if (!(ok = issue_pv(g, j))) break;
          if (last) warp_commit(bar_v_empty + 8 * (j % kStages));
          if (more) {
            if (g == 0 && !(ok = ready(bar_k_full, j + 1))) break;
            issue_s(g, j + 1);
            if (last) warp_commit(bar_k_empty + 8 * ((j + 1) % kStages));
          }
        }
      }
      if (ok) warp_commit(bar_o_full);
      // drain: every tcgen05 operation this warp issued has completed
      warp_commit(bar_drain);
      const uint64_t t0 = globaltimer();
      while (!bar_try_wait(bar_drain, 0)) {
        if (globaltimer() - t0 > 2000000000ull) {
          record_status(a.status, NVFP4_ERR_TIMEOUT);
          break;
        }
      }
    } else if (warp == kLoadWarp) {
      // ---------------------------------------------------------- codes, a tile ahead
      const int32_t* table = a.table + int64_t(b) * a.table_stride;
      auto page_of = [&](int j) {   // lanes 0..7: the groups' pages, -1 for none
        const int tok = t_begin + j * kKeys + 16 * lane;
        const int id = lane < kGroups && tok < t_end
                           ? __ldg(table + fast_div(a.page_div, uint32_t(tok)))
                           : -1;
        return id < a.n_pages ? id : -1;
      };
      constexpr uint32_t kBytes = 16 * kD;   // of a group
      int page = page_of(0), j = 0;
      for (; j < n_tiles; ++j) {
        const int next = page_of(j + 1);
        const uint32_t rs = j % L::kRaw, empty = ((j / L::kRaw) & 1) ^ 1;
        const int tok = t_begin + j * kKeys + 16 * lane;
        const int in_page = tok - int(fast_div(a.page_div, uint32_t(tok))) * a.page_tokens;
        const int64_t at = ((int64_t(max(page, 0)) * a.kv_heads + h) * a.page_tokens + in_page) * kD;
        const uint32_t live = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0));
        bool ok = true;
#pragma unroll
        for (int pl = 0; pl < 2 && ok; ++pl) {
          const uint32_t full = (pl ? bar_rv_full : bar_rk_full) + 8 * rs;
          ok = __all_sync(0xFFFFFFFFu,
                          waiter.wait((pl ? bar_rv_empty : bar_rk_empty) + 8 * rs, empty));
          if (!ok) break;
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                         "r"(live * kBytes)
                         : "memory");
          __syncwarp();
          if (page >= 0)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                "%2, [%3];" ::"r"(sbase + (pl ? L::kRawV : L::kRawK) + rs * L::kRawBytes +
                                  lane * kBytes),
                "l"((pl ? a.v_codes : a.k_codes) + at), "r"(kBytes), "r"(full)
                : "memory");
          __syncwarp();
        }
        if (!ok) break;
        page = next;
      }
      // drain: every copy issued has landed before the CTA may leave (an abort may have come
      // between a tile's K and V: its K is waited for, its V was not begun)
      for (int pl = 0; pl < 2; ++pl)
        for (int d = max(0, j - L::kRaw); d < (pl == 0 ? min(j + 1, n_tiles) : j); ++d) {
          const uint32_t full = (pl ? bar_rv_full : bar_rk_full) + 8 * (d % L::kRaw);
          const uint64_t t0 = globaltimer();
          while (!bar_try_wait(full, (d / L::kRaw) & 1)) {
            if (globaltimer() - t0 > 2000000000ull) break;
          }
        }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int kD>
cudaError_t launch(const Args& a, dim3 grid, cudaStream_t st) {
  cudaError_t e = allow_smem<chunk_kernel<kD>>(Layout<kD>::kBytes);
  if (e != cudaSuccess) return e;
  // the register split above adds up only with this launch allocation
  static const int regs = [] {
    cudaFuncAttributes f = {};
    return cudaFuncGetAttributes(&f, chunk_kernel<kD>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_pdl(chunk_kernel<kD>, grid, dim3(kThreads), size_t(Layout<kD>::kBytes), st, a);
}

}  // namespace kv8_chunk

cudaError_t launch_kv8_chunk(const kv8::Args& a, int32_t head_dim, int32_t row_tiles, int32_t batch,
                             cudaStream_t st) {
  const dim3 grid(unsigned(a.kv_heads) * unsigned(row_tiles), unsigned(batch),
                  unsigned(a.n_splits));
  return head_dim == 64 ? kv8_chunk::launch<64>(a, grid, st) : kv8_chunk::launch<128>(a, grid, st);
}

}  // namespace nvfp4
