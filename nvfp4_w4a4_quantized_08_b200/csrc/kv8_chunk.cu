// kv8_chunk.cu -- attention of many rows per request over the paged 8-bit cache, on the
// sm_100a tensor cores (chunks of new tokens, prompts).
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k[j]) v[j],  k = codes * page scale
//
// Bound by the softmax (one exponential for each row and token: 16 a clock and SM) and the
// tensor core (fp16 S = Q K^T and P V), which take about the same time per tile of 128 x
// 128; so both have to run all the time.  One CTA of 16 warps takes 256 packed rows (two
// tiles of 128) of one request and KV head and a range of its tokens:
//   warps 0..7   softmax: warpgroup g owns row tile g, one row a thread.  A row's 128
//                scores of a tile are read from tensor memory once, into registers
//                (200 a thread, moved over from the other warps by setmaxnreg); the
//                probabilities go back as fp16.
//   warps 8..11  decoders: E4M3 codes -> fp16 K and V operands in 128-byte-swizzled shared
//                memory (two stages each), one hardware conversion per two codes, exact.
//                (bf16 operands took 4.5 times the instructions, and set the pace.)
//   warp 12, 14  issue the MMAs, one S and one P V.
//   warp 13      copies the codes of a tile ahead (one bulk copy for the 16 tokens of a group,
//                which share a page).
// Tensor memory (512 columns): O0, O1, one S, P0, P1.  Both row tiles use the one S in turn:
// it is free again as soon as a softmax has read it, so the next S is there before the
// softmax that needs it is done with the last one, and no S waits for a P V.
//
// What a softmax warp executes sets the pace: two of them a scheduler, each alone with its
// latencies.  So it looks for no maximum: the weights of a tile are taken against the
// reference in use, and only where a sum of 16 of them shows that one might be too large for
// fp16 is the tile taken again, in a slower form that finds the maximum and raises the
// reference.  2640 rows over 10560 tokens and 24 heads: 429 us with the maximum taken every
// time, 375 without; 269 with no exponentials and no decoding at all.  On the way there: 624 us
// with S and P in one place and one MMA warp; 456 with rings of their own for K and V; what did
// not help: sixteen softmax warps of half a row each (517), a quarter of the exponentials as
// polynomials on the FMA pipe (478 against 458), and warps that take turns at the exponentials
// (493 against 458).  These are single short graphs, before the card is at its power limit; over a
// second of calls it is 390 us (879 TFLOP/s, 53% of the measured bf16 burst).
//
// The codes go into the products without their page scales.  Q is scaled by a power of two
// per row to fp16 (largest element in [2^8, 2^9): exact for elements within 2^-22 of it, an
// error of at most 2^-33 of it below).  Scores of a group of 16 tokens are multiplied by the
// page's K scale in fp32.  The page's V scale is an exponent added to the probability's:
// these weights 2^(x + log2 s_v) go into P relative to the reference, which follows their
// maximum (2^9 there; an error of at most 2^-34 of it where they become subnormal), and the
// normaliser takes a group's sum times 2^-exponent: exact, and one multiplication a group.
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
constexpr int kThreads = 512;              // four warpgroups; the last: MMA of S, loads, MMA of P V
constexpr int kLoadWarp = kMmaWarp + 1, kPvWarp = kMmaWarp + 2;
constexpr int kStages = 2;                 // decoded tiles of K, and of V
constexpr int kMetaStages = 4;             // page scales: read later than K
constexpr int kMetaFloats = 3 * kGroups + 1;   // and whether the tile is wide
// registers a thread at launch, and after the warpgroups have shared them out anew
constexpr int kLaunchRegs = 128, kSoftRegs = 200, kDecRegs = 56, kMmaRegs = 56;
static_assert(2 * kSoftRegs + kDecRegs + kMmaRegs == 4 * kLaunchRegs, "register split");
static_assert(kThreads * kLaunchRegs <= 65536, "registers of an SM");
constexpr uint32_t kTmemCols = 512;
// tensor memory columns: O_g at 128 g, S, P_g (fp16 pairs) at kPCol0 + 64 g
constexpr uint32_t kOCol0 = 0, kSCol0 = 256, kPCol0 = 384;
constexpr float kBias = 9.0f;     // the largest weight is 2^9 when it sets the reference,
constexpr float kLazy = 2.0f;     // and sets it where it would be more than 2^11
constexpr float kWide = 28.0f;    // |log2 s_v| above which a tile takes the slower exponentials

template <int kD>
struct Layout {
  static constexpr int kChunks = kD / 64;
  static constexpr int kOp = kChunks * kChunkBytes;        // 128 rows x kD fp16
  static constexpr int kQ = 0, kK = kTiles * kOp, kV = kK + kStages * kOp;
  static constexpr int kRaw = kD == 64 ? 3 : 1;            // tiles of codes ahead
  static constexpr int kRawBytes = kKeys * kD;             // of one plane
  static constexpr int kRawK = kV + kStages * kOp, kRawV = kRawK + kRaw * kRawBytes;
  static constexpr int kMeta = kRawV + kRaw * kRawBytes;
  static constexpr int kBar = (kMeta + kMetaStages * kMetaFloats * 4 + 7) / 8 * 8;
  // q[2], k_full, k_empty, v_full, v_empty [stage], s_full[2], s_free, p_ready[2],
  // pv_done[2], meta_full[4], raw K full, empty, raw V full, empty [raw stage], o_full, drain[2]
  static constexpr int kNumBars = 2 + 4 * kStages + 2 + 1 + 2 + 2 + kMetaStages + 4 * kRaw + 3;
  static constexpr int kTmemPtr = kBar + kNumBars * 8;
  static constexpr int kAbort = kTmemPtr + 4;
  static constexpr int kBytes = kAbort + 4 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

// kind::f16: fp32 D (bit 4), fp16 A and B, N >> 3 at 17, M >> 4 at 24; B MN-major: bit 16.
__host__ __device__ constexpr uint32_t idesc(uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | (uint32_t(kRows >> 4) << 24);
}

// Four E4M3 bytes -> two fp16 pairs, exact.
__device__ __forceinline__ uint2 decode4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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

template <int kD, bool kBrief>
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
  const uint32_t bar_s_free = bar_s_full + 8 * kTiles;
  const uint32_t bar_p_ready = bar_s_free + 8;                 // + 8 g
  const uint32_t bar_pv_done = bar_p_ready + 8 * kTiles;       // + 8 g
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
      bar_init(bar_p_ready + 8 * g, 4);
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
    bar_init(bar_s_free, 4);
    bar_init(bar_o_full, 1);
    bar_init(bar_drain, 1);
    bar_init(bar_drain + 8, 1);
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
  const WarpWaiter<kBrief> waiter{{a.wait_limit_ns, abort_flag, a.status}};

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
    const uint32_t lanes = tmem + ((quad * 32) << 16);
    const uint32_t o_addr = lanes + kOCol0 + 128 * g, p_addr = lanes + kPCol0 + 64 * g;
    const uint32_t s_addr = lanes + kSCol0;
    const int rho = base + int(g) * kRows + int(row);
    const bool live = int(g) < n_q && rho < rows;
    // tokens of the range that this row sees (dead rows follow the last live one)
    const int vis = min(t_range, kv8::sees(a, rq, max(0, min(rho, rows - 1)))) - t_begin;
    const int vis_min = __reduce_min_sync(0xFFFFFFFFu, vis);
    bool ok = true;
    // l and O are in units of 2^ref, ref the largest weight's logarithm less kBias (about: see
    // below); seen: a token has set it
    float ref = 0.0f, l_run = 0.0f;
    bool seen = false, all_seen = false;
    if (int(g) < n_q && n_tiles > 0) {
      // Q row -> fp16 in shared memory, its power of two into the scores' scale
      const uint4* src =
          reinterpret_cast<const uint4*>(live ? kv8::q_row(a, rq, h, rho, kD) : a.q);
      uint32_t top = 0;
#pragma unroll 4
      for (uint32_t u = 0; u < kD / 8; ++u) {
        const uint4 v = live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
      const uint32_t field = min(262u - (max(top & 0xFFFFu, top >> 16) >> 7), 253u);
      const float up = __uint_as_float(field << 23);
      const float q_scale = __uint_as_float((254u - field) << 23);
      const uint32_t qs = sbase + L::kQ + g * L::kOp;
      auto half2 = [&](uint32_t w) {
        return f16x2_rn(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
      };
#pragma unroll 4
      for (uint32_t u = 0; u < kD / 8; ++u) {
        const uint4 v = live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
        st_shared_v4(qs + op_offset(row, u),
                     make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w)));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(bar_q + 8 * g);
      for (int j = 0; j < n_tiles; ++j) {
        ok = waiter.wait(bar_meta + 8 * (j % kMetaStages), (j / kMetaStages) & 1);
        if (!ok) break;
        // per group: K scale times scale * log2 e; log2 of the V scale; 1 / V scale (0: no
        // page, left out, with a log2 of -inf)
        const float* ms = meta + (j % kMetaStages) * kMetaFloats;
        const bool slow = vis_min < (j + 1) * kKeys || ms[3 * kGroups] != 0.0f;
        ok = waiter.wait(bar_s_full + 8 * g, j & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[4][32];
        load_scores(s_addr, r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar_s_free);
        if (j > 0) {   // tile j - 1's P V has read P, and written O
          if (!(ok = waiter.wait(bar_pv_done + 8 * g, (j - 1) & 1))) break;
          tc_fence_after();
        }
        // Weights against the reference in use, without looking for a maximum first: a weight
        // cannot be too large for fp16 where no sum of 16 exceeds 2^15.
        bool again = slow || !all_seen;
        if (!again) {
          float l = 0.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float scn = ms[2 * c + n] * q_scale, off = ms[kGroups + 2 * c + n] - ref;
              const float2 sc2 = make_float2(scn, scn), of2 = make_float2(off, off);
              const float2 one2 = make_float2(1.0f, 1.0f);
              float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 x =
                    __ffma2_rn(make_float2(__uint_as_float(r[c][16 * n + 2 * e]),
                                           __uint_as_float(r[c][16 * n + 2 * e + 1])),
                               sc2, of2);
                const float2 w = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                sum = __ffma2_rn(w, one2, sum);
                pk[8 * n + e] = f16x2_rn(w.x, w.y);
              }
              const float both = sum.x + sum.y;
              l = fmaf(both, ms[2 * kGroups + 2 * c + n], l);
              again |= !(both <= 32768.0f);   // (true for NaN)
            }
            tmem_st16(p_addr + 16 * c, pk);
          }
          again = __any_sync(0xFFFFFFFFu, again);
          if (!again) l_run += l;
        }
        if (again) {
          // The slower form, until every row has seen a token, for masked tiles (exact zeros), V
          // scales far from 1, and a new maximum: the reference rises to it, l and O are
          // rescaled, and the V scale is multiplied in after the exponential, so that a token
          // counts for the normaliser even where its weight is lost against the largest.  A masked
          // score is -inf, so no factor may be 0: K scales are where a page was never written, and
          // small ones times the power of two of a row near 0 underflow.
          auto factor_of = [&](int n) { return fmaxf(ms[n] * q_scale, 0x1p-126f); };
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
            // (the scales are positive; a group of no page has a log2 of -inf)
            mx = fmaxf(mx, fmaf(fmaxf(t0, t1), factor_of(n), ms[kGroups + n]));
          }
          float factor = 1.0f;
          if (mx - kBias > ref + kLazy || !seen) {
            if (mx > -INFINITY) {
              // In two steps: the reference may rise by more than 2^126 through the pages' V
              // scales alone, after tokens that still are most of the normaliser (O in units of
              // the largest weight is lost then, the normaliser is not).
              const float half = seen ? exp2_approx(0.5f * (ref - (mx - kBias))) : 0.0f;
              factor = half * half;
              ref = mx - kBias;
              seen = true;
              l_run = l_run * half * half;
            }
          }
          all_seen = __all_sync(0xFFFFFFFFu, seen);
          if (j > 0 && __any_sync(0xFFFFFFFFu, factor != 1.0f)) {
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
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float scn = factor_of(2 * c + n);
              // a group of no page: 0 for the normaliser too
              const float lv = ms[kGroups + 2 * c + n];
              const float none = lv == -INFINITY ? -INFINITY : -ref, sv = exp2f(lv);
              float sum = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x0 =
                    exp2_approx(fmaf(__uint_as_float(r[c][16 * n + 2 * e]), scn, none));
                const float x1 =
                    exp2_approx(fmaf(__uint_as_float(r[c][16 * n + 2 * e + 1]), scn, none));
                sum += x0 + x1;
                pk[8 * n + e] = f16x2_rn(x0 * sv, x1 * sv);
              }
              l_run += sum;
            }
            tmem_st16(p_addr + 16 * c, pk);
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bar_p_ready + 8 * g);
      }
      if (ok) ok = waiter.wait(bar_o_full, 0);
      tc_fence_after();
    }
    // ---- O / l -> the output or the range's part; a row that saw nothing is zero
    if (ok && int(g) < n_q) {
      const float norm = l_run == 0.0f ? 0.0f : 1.0f / l_run;
      const float lse2 = l_run == 0.0f ? -INFINITY : ref + log2f(l_run);
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
          v[e] = l_run == 0.0f ? 0.0f : __uint_as_float(o[e]) * norm;
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
    int next_page = -1;
    if (n_tiles > 0) {
      load_scales(0, group_page(0));
      next_page = group_page(1);
    }
    for (int j = 0; j < n_tiles; ++j) {
      const uint32_t st = j % kStages, empty = ((j / kStages) & 1) ^ 1;
      const uint32_t rs = j % L::kRaw, full = (j / L::kRaw) & 1;
      const int left = t_end - t_begin - j * kKeys;
      if (warp == kSoftWarps) {
        float* m = meta + (j % kMetaStages) * kMetaFloats + t;
        const bool none = vs < 0.0f;
        const float v = fmaxf(vs, 0x1p-60f);   // the smallest scale there is
        const uint32_t bits = __float_as_uint(v);
        const float lv = float(int(bits >> 23) - 127) +
                         __log2f(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
        if (t < kGroups) {
          m[0] = none ? 1.0f : ks * a.scale_log2;
          m[kGroups] = none ? -INFINITY : lv;
          m[2 * kGroups] = none ? 0.0f : 1.0f / v;
        }
        const bool wide = __any_sync(0xFFFFFFFFu, t < kGroups && !none && fabsf(lv) > kWide);
        if (t == 0) m[3 * kGroups] = wide ? 1.0f : 0.0f;
        __syncwarp();
        if (lane == 0) bar_arrive(bar_meta + 8 * (j % kMetaStages));
        if (j + 1 < n_tiles) {
          load_scales(j + 1, next_page);
          next_page = group_page(j + 2);
        }
      }
      // K, then V: codes of raw stage rs -> operand stage st.  (Rolled loops: the softmax code
      // alone fills the instruction cache; unrolled decoders cost a quarter of the rate.)
      bool ok = true;
#pragma unroll 1
      for (int pl = 0; pl < 2; ++pl) {
        const uint32_t bar_empty = (pl ? bar_v_empty : bar_k_empty) + 8 * st;
        const uint32_t bar_full = (pl ? bar_v_full : bar_k_full) + 8 * st;
        const uint32_t bar_raw = (pl ? bar_rv_full : bar_rk_full) + 8 * rs;
        const uint32_t bar_raw_empty = (pl ? bar_rv_empty : bar_rk_empty) + 8 * rs;
        ok = waiter.wait(bar_empty, empty) && waiter.wait(bar_raw, full);
        if (!ok) break;
        const uint32_t raw = sbase + (pl ? L::kRawV : L::kRawK) + rs * L::kRawBytes + t * 16;
        const uint32_t op = sbase + (pl ? L::kV : L::kK) + st * L::kOp;
#pragma unroll 1
        for (int i0 = 0; i0 < kMine; i0 += 4) {   // four loads in flight
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "r"(raw + kDecWarps * 32 * 16 * (i0 + i)));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t tok = t / kUnits + kPer * (i0 + i);
            // past the range's end there may be anything, NaN codes included: 0
            if (int(tok) >= left) w[i] = make_uint4(0, 0, 0, 0);
            const uint2 w0 = decode4(w[i].x), w1 = decode4(w[i].y);
            const uint2 w2 = decode4(w[i].z), w3 = decode4(w[i].w);
            const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y);
            const uint4 hi = make_uint4(w2.x, w2.y, w3.x, w3.y);
            // the upper half of the units starts with its second part: other banks
            const bool swap = u >= 4;
            st_shared_v4(op + op_offset(tok, 2 * u + swap), swap ? hi : lo);
            st_shared_v4(op + op_offset(tok, 2 * u + !swap), swap ? lo : hi);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          bar_arrive(bar_raw_empty);
          bar_arrive(bar_full);
        }
      }
      if (!ok) break;
    }
  } else {
    // ------------------------------------------------------------ MMA issuer
    fewer_regs<kMmaRegs>();
    // Two warps issue the MMAs, one S and one P V, so that the waits of one overlap the products
    // of the other; a whole warp each, so that operands are uniform, one lane of which issues.
    if ((warp == kMmaWarp || warp == kPvWarp) && n_tiles > 0) {
      // low descriptor words: K-major with LBO 1, MN-major with the chunk stride
      const uint32_t lo_k = ((sbase & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t lo_mn = ((sbase & 0x3FFFFu) >> 4) | (uint32_t(kChunkBytes >> 4) << 16);
      bool ok = true;
      if (warp == kMmaWarp) {
        // S = Q_g K_j^T, once the softmax before has read S: 16 dims a step, +32 bytes, the
        // next chunk after 4
        uint32_t issued = 0;
        for (int g = 0; g < n_q && ok; ++g) ok = waiter.wait(bar_q + 8 * g, 0);
#pragma unroll 1
        for (int j = 0; j < n_tiles && ok; ++j) {
          const uint32_t st = j % kStages;
          if (!(ok = waiter.wait(bar_k_full + 8 * st, (j / kStages) & 1))) break;
          const uint32_t kd = lo_k + ((L::kK + st * L::kOp) >> 4);
#pragma unroll 1
          for (int g = 0; g < n_q; ++g) {
            if (issued > 0 && !(ok = waiter.wait(bar_s_free, (issued - 1) & 1))) break;
            ++issued;
            tc_fence_after();
            const uint32_t qd = lo_k + ((L::kQ + g * L::kOp) >> 4);
            unrolled(
                [&](auto k) {
                  constexpr uint32_t at = (k.value >> 2) * (kChunkBytes >> 4) + 2 * (k.value & 3);
                  warp_mma_ss<at, at>(tmem + kSCol0, qd, kd, idesc(kKeys), k.value != 0);
                },
                std::make_integer_sequence<uint32_t, kD / 16>());
            warp_commit(bar_s_full + 8 * g);
          }
          if (ok) warp_commit(bar_k_empty + 8 * st);
        }
      } else {
        // O_g += P_g(j) V_j: 16 keys a step, 8 columns of P
#pragma unroll 1
        for (int j = 0; j < n_tiles && ok; ++j) {
          const uint32_t st = j % kStages;
          if (!(ok = waiter.wait(bar_v_full + 8 * st, (j / kStages) & 1))) break;
          const uint32_t vd = lo_mn + ((L::kV + st * L::kOp) >> 4);
#pragma unroll 1
          for (int g = 0; g < n_q; ++g) {
            const uint32_t od = tmem + kOCol0 + 128 * g, pd = tmem + kPCol0 + 64 * g;
            if (!(ok = waiter.wait(bar_p_ready + 8 * g, j & 1))) break;
            tc_fence_after();
            unrolled(
                [&](auto k) {
                  warp_mma_ts<8 * k.value, k.value * (2048 >> 4)>(
                      od, pd, vd, idesc(kD) | (1u << 16), k.value != 0 || j != 0);
                },
                std::make_integer_sequence<uint32_t, 8>());
            warp_commit(bar_pv_done + 8 * g);
          }
          if (ok) warp_commit(bar_v_empty + 8 * st);
        }
        if (ok) warp_commit(bar_o_full);
      }
      // drain: every tcgen05 operation this warp issued has completed
      const uint32_t drain = bar_drain + (warp == kMmaWarp ? 0 : 8);
      warp_commit(drain);
      const uint64_t t0 = globaltimer();
      while (!bar_try_wait(drain, 0)) {
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
      int page = page_of(0), issued[2] = {0, 0};   // tiles whose K, V copies have begun
      for (int j = 0; j < n_tiles; ++j) {
        const int next = page_of(j + 1);
        const uint32_t rs = j % L::kRaw, empty = ((j / L::kRaw) & 1) ^ 1;
        const int tok = t_begin + j * kKeys + 16 * lane;
        const int in_page = tok - int(fast_div(a.page_div, uint32_t(tok))) * a.page_tokens;
        const int64_t at =
            ((int64_t(max(page, 0)) * a.kv_heads + h) * a.page_tokens + in_page) * kD;
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, page >= 0);
        bool ok = true;
#pragma unroll
        for (int pl = 0; pl < 2 && ok; ++pl) {
          const uint32_t full = (pl ? bar_rv_full : bar_rk_full) + 8 * rs;
          ok = waiter.wait((pl ? bar_rv_empty : bar_rk_empty) + 8 * rs, empty);
          if (!ok) break;
          const uint32_t to = sbase + (pl ? L::kRawV : L::kRawK) + rs * L::kRawBytes;
          // groups of no page are zero
          for (uint32_t none = 0xFFu & ~have; none != 0; none &= none - 1)
            for (uint32_t at = lane * 16; at < kBytes; at += 512)
              st_shared_v4(to + (__ffs(none) - 1) * kBytes + at, make_uint4(0, 0, 0, 0));
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full),
                         "r"(__popc(have) * kBytes)
                         : "memory");
          __syncwarp();
          if (page >= 0)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                "%2, [%3];" ::"r"(to + lane * kBytes),
                "l"((pl ? a.v_codes : a.k_codes) + at), "r"(kBytes), "r"(full)
                : "memory");
          __syncwarp();
          ++issued[pl];
        }
        if (!ok) break;
        page = next;
      }
      // drain: every copy issued has landed before the CTA may leave (a wait that ran out may have
      // come between a tile's K and V)
#pragma unroll
      for (int pl = 0; pl < 2; ++pl)
        for (int d = max(0, issued[pl] - L::kRaw); d < issued[pl]; ++d) {
          const uint32_t full = (pl ? bar_rv_full : bar_rk_full) + 8 * (d % L::kRaw);
          const uint64_t t0 = globaltimer();
          while (!bar_try_wait(full, (d / L::kRaw) & 1)) {
            if (globaltimer() - t0 > 2000000000ull) {
              record_status(a.status, NVFP4_ERR_TIMEOUT);
              break;
            }
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

template <int kD, bool kBrief>
cudaError_t launch(const Args& a, dim3 grid, cudaStream_t st) {
  cudaError_t e = allow_smem<chunk_kernel<kD, kBrief>>(Layout<kD>::kBytes);
  if (e != cudaSuccess) return e;
  // the register split above adds up only with this launch allocation (the build checks it too)
  static const int regs = [] {
    cudaFuncAttributes f = {};
    return cudaFuncGetAttributes(&f, chunk_kernel<kD, kBrief>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_pdl(chunk_kernel<kD, kBrief>, grid, dim3(kThreads), size_t(Layout<kD>::kBytes), st,
                    a);
}

template <int kD>
cudaError_t launch_dim(const Args& a, dim3 grid, cudaStream_t st) {
  return a.wait_limit_ns < kBriefNs ? launch<kD, true>(a, grid, st)
                                    : launch<kD, false>(a, grid, st);
}

}  // namespace kv8_chunk

cudaError_t launch_kv8_chunk(const kv8::Args& a, int32_t head_dim, int32_t row_tiles, int32_t batch,
                             cudaStream_t st) {
  const dim3 grid(unsigned(a.kv_heads) * unsigned(row_tiles), unsigned(batch),
                  unsigned(a.n_splits));
  return head_dim == 64 ? kv8_chunk::launch_dim<64>(a, grid, st)
                        : kv8_chunk::launch_dim<128>(a, grid, st);
}

}  // namespace nvfp4
