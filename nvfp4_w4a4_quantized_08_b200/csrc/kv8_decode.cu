// kv8_decode.cu -- attention of a few rows per request over the paged 8-bit cache
// (single tokens and short drafts), and the join of split ranges.
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . k[j]) v[j],  k = codes * page scale
//
// Bound by the cache: each K and V byte is read once for the rows of one request
// that share a KV head (G query heads times the request's queries, packed; tiles of
// 8 NT rows).  One CTA takes one tile of rows, one KV head and one range of tokens;
// its four warps take groups of 16 tokens in turn (2 KB of K and 2 KB of V for 128
// dims), each through a ring of its own in shared memory that asynchronous 16-byte
// copies fill kStages - 1 groups ahead: ~128 KB in flight an SM, where the latency of
// HBM at full rate needs ~40 KB and two groups a warp in registers gave 48 KB in
// theory and 62% of the rate.  Rings are private to a warp, so no barrier is waited on.
//
//   S^T = K Q^T    m16n8k16, A = 16 tokens of K, B = 8 rows of Q.  The order of the
//                  dims inside a product is free, so a lane's 32 contiguous bytes of a
//                  token are its A registers after one hardware conversion (E4M3 ->
//                  fp16, exact) per two elements (a table or shifts cost 2.5 times the
//                  issue slots: 10 against 25 words a clock and SM, measured).
//   O^T += V^T P^T m16n8k16, A = 16 dims by 16 tokens of V: a lane loads 16 contiguous
//                  dims of its four tokens and pairs tokens with byte permutes before
//                  the conversion.  P^T comes from S^T by an 8x8 transposition in
//                  registers (movmatrix).
//
// fp16 operands: Q is scaled by a power of two per row so that its largest element is
// in [2^8, 2^9) (exact for elements within 2^-22 of it, below that an error of at most
// 2^-33 of it); sums are fp32.  The page scale of K is multiplied into the fp32 scores.
// The page scale of V is an exponent added to the probability's, and the weights
// 2^(x + log2 s_v) are taken against their own running maximum, apart from the one of
// the normaliser: so fp16 holds them however far apart the pages' scales lie (2^7 at the
// maximum; an error of at most 2^-32 of it where they become subnormal).  Both maxima
// are raised lazily: only a group that exceeds one by 2^8 rescales (one warp vote a
// group decides).
//
// Ranges: with few requests and heads the tokens are split over CTAs; each leaves its
// normalised rows in fp32 and their log-sum-exp, and a second kernel joins them in
// order of the range, so results do not depend on timing.  Up to 8 ranges of one wave are
// a cluster, whose CTAs store their rows to the one that joins them (fetching them from one
// another instead: 0.6 us longer for 777 tokens).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv8_batch.cuh"

namespace nvfp4 {
namespace kv8 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kMaxCluster = 8;
constexpr float kLazy = 8.0f;
constexpr float kBias = 7.0f;   // weights are taken times 2^7: at most 2^15 in fp16
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 bytes -> two fp16 pairs (exact).
__device__ __forceinline__ void e4m3_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int kWords>
__device__ __forceinline__ void lds(uint32_t at, uint32_t* w) {
  if constexpr (kWords == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at));
  else
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
}

// Where byte `at` of a 16-token group's codes lies in its stage: 16-byte units of a token
// row exchanged by the token's place, so that the reads below meet no bank twice (128 dims)
// or at most twice (64).
template <int kDim>
__device__ __forceinline__ uint32_t place(uint32_t token, uint32_t unit) {
  if constexpr (kDim == 128)
    return token * 128 + ((unit ^ (token & 7)) << 4);
  else
    return token * 64 + ((unit ^ ((token >> 1) & 3)) << 4);
}

// Groups of 16 tokens that a warp takes at a time: two of 64 dims, so that the work that
// goes by tokens, not bytes, has two chains to overlap.
template <int kDim, int NT>
constexpr int kGroups = kDim == 64 && NT == 1 ? 2 : 1;

// Shared memory of a CTA by itself: the rings, or after them the warps' rows.
template <int kDim, int NT>
constexpr size_t kOwnBytes =
    std::max(size_t(kWarps) * kStages * kGroups<kDim, NT> * 2 * 16 * kDim,
             size_t(kWarps) * 8 * NT * (kDim + 4) * sizeof(float));

// CTAs of an SM: by registers.
template <int NT>
constexpr int kResident = NT == 1 ? 4 : 3;

template <int kDim, int NT>
__global__ void __launch_bounds__(kThreads, kResident<NT>) decode_kernel(const Args a) {
  constexpr int kSteps = kDim / 16;   // k16 steps of S
  constexpr int kTiles = kDim / 16;   // m16 tiles of O
  constexpr int kRows = 8 * NT;
  constexpr int kGroup = 16 * kDim;   // bytes of K (and of V) of a group
  constexpr int kG = kGroups<kDim, NT>, kStage = kG * 2 * kGroup;
  constexpr int kStepTokens = 16 * kG * kWarps;
  extern __shared__ __align__(128) uint8_t ring[];   // [warp][stage][group][K, V][kGroup]
  // after the last group: the warps' rows, in the rings' place
  float (*so)[kRows][kDim + 4] = reinterpret_cast<float (*)[kRows][kDim + 4]>(ring);
  __shared__ float sm[kWarps][3][kRows];   // maximum, weights' maximum, sum
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  // ranges are the slowest index: the later ones, which fewer requests have, come last
  const int h = blockIdx.x % a.kv_heads, tile = blockIdx.x / a.kv_heads;
  const int b = blockIdx.y, split = blockIdx.z;
  // This warp's steps: kG groups of 16 tokens, tokens first + kStepTokens i ..; a group is
  // inside one page.  The pages of 32 groups at a time, lane j's that of group j, whether the
  // request is as long or not: so the first ones are read along with the lengths.
  const int t_begin = split * a.chunk;
  const int first = t_begin + 16 * kG * warp;
  const int32_t* table = a.table + int64_t(b) * a.table_stride;
  auto group_token = [&](int n) { return first + (n / kG) * kStepTokens + (n % kG) * 16; };
  auto load_pages = [&](int n0) {
    const int tok = group_token(n0 + lane);
    return tok < a.max_tokens ? __ldg(table + fast_div(a.page_div, uint32_t(tok))) : 0;
  };
  if (a.cluster) cluster_arrive();   // waited for before the first store to another CTA
  pdl_wait();
  pdl_trigger();
  const int first_page = load_pages(0);
  int next_page = load_pages(32);
  const Request rq = request(a, b, tid == 0 && blockIdx.x == 0 && split == 0);
  const int rows = rq.nq * a.group;
  const int rho0 = tile * kRows;
  const int used = splits_of(a, rq.kv);
  if (rho0 >= rows || split >= used) {
    if (a.cluster) {  // the other CTAs count this one at both barriers
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
    return;
  }
  // this CTA's tokens: its range, up to what the tile's last row sees
  const int last_row = min(rho0 + kRows, rows) - 1;
  const int t_range = split == used - 1 ? rq.kv : min(rq.kv, t_begin + a.chunk);
  const int t_end = min(t_range, sees(a, rq, last_row));

  // Q: lane's rows r (one per tile), dims [kDim / 4 * c, ..), as B registers
  uint32_t qf[NT][kSteps][2];
  float qs[NT][2];   // softmax scale over Q's power of two, for rows 2c and 2c + 1
  int vis[NT][2];    // tokens those rows see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rho = rho0 + 8 * nt + r;
    uint32_t w[kDim / 8];
    const bool live = rho < rows;
    const uint16_t* src = live ? q_row(a, rq, h, rho, kDim) + c * (kDim / 4) : a.q;
#pragma unroll
    for (int i = 0; i < kDim / 32; ++i) {
      const uint4 v = live ? ld_nc_v4_l1(src + 8 * i) : make_uint4(0, 0, 0, 0);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kDim / 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t field = min(262u - (top >> 7), 253u);   // 2^e as an exponent field
    const float up = __uint_as_float(field << 23);
    const float down = __uint_as_float((254u - field) << 23) * a.scale_log2;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v = w[2 * ks + i];
        qf[nt][ks][i] =
            f16x2_rn(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      qs[nt][i] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * c + i));
      vis[nt][i] = sees(a, rq, min(rho0 + 8 * nt + 2 * c + i, rows - 1));
    }
  }
  // tokens every row of the tile sees (the first row sees the fewest)
  const int vis_all = sees(a, rq, rho0);

  // running maxima: base and basev (less kBias) are what the exponents are taken against, 0
  // before the first token; lim and limv what a score may reach without a rescale
  float o[NT][kTiles][4], l[NT][2], base[NT][2], basev[NT][2], lim[NT][2], limv[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[nt][t][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[nt][i] = base[nt][i] = basev[nt][i] = 0.0f;
      lim[nt][i] = limv[nt][i] = kNegInf;
    }
  }

  const int n_steps = t_end > first ? (t_end - first + kStepTokens - 1) / kStepTokens : 0;
  // place and page scales of 32 groups at a time; two windows, the second loaded while the
  // first is worked on
  struct Window {
    int64_t at;     // bytes from the start of the codes
    float ks, lv;   // scale of K, log2 of the scale of V
  };
  auto load_window = [&](int n0, int id) {
    Window w;
    const int tok = group_token(n0 + lane);
    const bool ok = id >= 0 && id < a.n_pages;
    const int64_t ph = int64_t(ok ? id : 0) * a.kv_heads + h;
    const int in_page = tok - int(fast_div(a.page_div, uint32_t(tok))) * a.page_tokens;
    w.at = (ph * a.page_tokens + in_page) * kDim;
    // a page that is not one of the pool's is left out, and recorded
    if (!ok && tok < t_end) record_status(a.status, NVFP4_ERR_INVALID_ARG);
    w.ks = ok ? __ldg(a.k_scale + ph) : kNegInf;
    // log2 of the V scale, exact for a power of two; -inf for 0 (a page never written)
    const uint32_t vb = __float_as_uint(__ldg(a.v_scale + ph));
    w.lv = vb < 0x00800000u ? kNegInf
                            : float(int(vb >> 23) - 127) +
                                  __log2f(__uint_as_float((vb & 0x7FFFFFu) | 0x3F800000u));
    return w;
  };
  const uint32_t my_ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) +
                           uint32_t(warp) * kStages * kStage;
  uint32_t copy_to[kGroup / 512];   // where this lane's units of a group go
#pragma unroll
  for (int j = 0; j < kGroup / 512; ++j) {
    const uint32_t n = lane + 32 * j;
    copy_to[j] = my_ring + place<kDim>(n / (kDim / 16), n % (kDim / 16));
  }
  const uint8_t* k_from = a.k_codes + lane * 16;
  const uint8_t* v_from = a.v_codes + lane * 16;
  // copies step i into its stage (nothing past the last; the group is committed all the same)
  auto issue = [&](int i, const Window& w) {
    const uint32_t st = uint32_t(i % kStages) * kStage;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int64_t at = __shfl_sync(0xFFFFFFFFu, w.at, (i * kG + g) & 31);
      if (first + i * kStepTokens + 16 * g < t_end) {
#pragma unroll
        for (int j = 0; j < kGroup / 512; ++j) {
          copy16(copy_to[j] + st + g * 2 * kGroup, k_from + at + 512 * j);
          copy16(copy_to[j] + st + (g * 2 + 1) * kGroup, v_from + at + 512 * j);
        }
      }
    }
    copies_commit();
  };

  auto compute = [&](int i, const Window& win) {
    const int tok = first + i * kStepTokens;
    float s[kG][NT][4], lv[kG];
    bool gone[kG];   // groups without tokens, or of no page
    bool masked = tok + 16 * kG > t_range || tok + 16 * kG > vis_all;
    bool cut = tok + 16 * kG > rq.kv;
    uint32_t st[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      st[g] = my_ring + uint32_t(i % kStages) * kStage + g * 2 * kGroup;
      // K: tokens r and r + 8, dims [kDim / 4 * c, ..)
      uint32_t kk[2][kDim / 16];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < kDim / 64; ++j)
          lds<4>(st[g] + place<kDim>(r + 8 * t, c * (kDim / 64) + j), &kk[t][4 * j]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[g][nt][j] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        uint32_t a0, a1, a2, a3;
        e4m3_f16(kk[0][ks], a0, a2);
        e4m3_f16(kk[1][ks], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(s[g][nt], a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
      }
    }
    bool raise = false;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const float ks_page = __shfl_sync(0xFFFFFFFFu, win.ks, (i * kG + g) & 31);
      lv[g] = __shfl_sync(0xFFFFFFFFu, win.lv, (i * kG + g) & 31);
      gone[g] = ks_page == kNegInf;
      masked |= gone[g];
      cut |= gone[g];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = qs[nt][j] * ks_page;
          s[g][nt][j] *= f;
          s[g][nt][2 + j] *= f;
        }
    }
    if (masked) {
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int left = (gone[g] ? 0 : min(vis[nt][j], t_range)) - tok - 16 * g - r;
            if (left <= 0) s[g][nt][j] = kNegInf;
            if (left <= 8) s[g][nt][2 + j] = kNegInf;
          }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int g = 0; g < kG; ++g)
          raise |= fmaxf(s[g][nt][j], s[g][nt][2 + j]) > fminf(lim[nt][j], limv[nt][j] - lv[g]);
      }
    if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = kNegInf, topv = kNegInf;
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const float x = fmaxf(s[g][nt][j], s[g][nt][2 + j]);
            top = fmaxf(top, x);
            topv = fmaxf(topv, x + lv[g]);
          }
#pragma unroll
          for (int m = 4; m <= 16; m <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
            topv = fmaxf(topv, __shfl_xor_sync(0xFFFFFFFFu, topv, m));
          }
          // (-inf stays: such a row has seen nothing)
          const float was = lim[nt][j] - kLazy, wasv = limv[nt][j] - kLazy;
          const float now = fmaxf(was, top), nowv = fmaxf(wasv, topv);
          float f = 1.0f;
          if (now > was) {
            l[nt][j] *= exp2_approx(was - now);
            base[nt][j] = now;
            lim[nt][j] = now + kLazy;
          }
          if (nowv > wasv) {
            f = exp2_approx(wasv - nowv);
            basev[nt][j] = nowv - kBias;
            limv[nt][j] = nowv + kLazy;
          }
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            o[nt][t][j] *= f;
            o[nt][t][2 + j] *= f;
          }
        }
    }
    uint32_t pb[kG][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          l[nt][j & 1] += exp2_approx(s[g][nt][j] - base[nt][j & 1]);
          // lv = -inf (a scale of 0) gives 0
          w[j] = exp2_approx(s[g][nt][j] + (lv[g] - basev[nt][j & 1]));
        }
        pb[g][nt][0] = transpose8x8(f16x2_rn(w[0], w[1]));
        pb[g][nt][1] = transpose8x8(f16x2_rn(w[2], w[3]));
      }
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      // V: tokens 2c, 2c + 1, 2c + 8, 2c + 9, dims [kDim / 8 * r, ..)
      uint32_t vv[4][kDim / 32];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int token = 2 * c + (t & 1) + 8 * (t >> 1);
        if constexpr (kDim == 128)
          lds<4>(st[g] + kGroup + place<kDim>(token, r), vv[t]);
        else
          lds<2>(st[g] + kGroup + place<kDim>(token, r >> 1) + 8 * (r & 1), vv[t]);
        // past the request's end (or in no page) it may be anything, NaN codes included: zero
        if (cut && (gone[g] || tok + 16 * g + token >= rq.kv)) {
#pragma unroll
          for (int j = 0; j < kDim / 32; ++j) vv[t][j] = 0;
        }
      }
#pragma unroll
      for (int j = 0; j < kDim / 32; ++j) {
        // words j of four tokens: dims 4 j .. 4 j + 3 of the lane's, two O tiles
        const uint32_t x0 = prmt(vv[0][j], vv[1][j], 0x5140);
        const uint32_t x1 = prmt(vv[0][j], vv[1][j], 0x7362);
        const uint32_t y0 = prmt(vv[2][j], vv[3][j], 0x5140);
        const uint32_t y1 = prmt(vv[2][j], vv[3][j], 0x7362);
        uint32_t a0, a1, a2, a3;
        e4m3_f16(x0, a0, a1);
        e4m3_f16(y0, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(o[nt][2 * j], a0, a1, a2, a3, pb[g][nt][0], pb[g][nt][1]);
        e4m3_f16(x1, a0, a1);
        e4m3_f16(y1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_f16(o[nt][2 * j + 1], a0, a1, a2, a3, pb[g][nt][0], pb[g][nt][1]);
      }
    }
  };

  constexpr int kWin = 32 / kG;   // steps of a window
  Window cur = load_window(0, first_page), nxt = cur;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i, cur);
  for (int i = 0; i < n_steps; ++i) {
    // the window of the steps that are copied runs kStages - 1 ahead of the computed ones'
    if (i % kWin == kWin / 2) nxt = load_window((i / kWin + 1) * 32, next_page);
    if (i % kWin == 0 && i > 0) {
      cur = nxt;
      next_page = load_pages((i / kWin + 1) * 32);
    }
    copies_wait<kStages - 2>();
    __syncwarp();   // step i is there for every lane, and stage i - 1 is read by every lane
    const int ahead = i + kStages - 1;
    issue(ahead, ahead / kWin == i / kWin ? cur : nxt);
    compute(i, cur);
  }
  copies_wait<0>();
  __syncthreads();   // the rings are free for the rows

  // join the four warps: sums of the lanes' tokens, then maxima and rows through
  // shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][i], 4);
      l[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][i], 8);
      l[nt][i] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][i], 16);
      const int row = 8 * nt + 2 * c + i;
      if (r == 0) {
        sm[warp][0][row] = lim[nt][i] == kNegInf ? kNegInf : base[nt][i];
        sm[warp][1][row] = limv[nt][i] == kNegInf ? kNegInf : basev[nt][i];
        sm[warp][2][row] = l[nt][i];
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        so[warp][row][kDim / 8 * r + 2 * t] = o[nt][t][i];
        so[warp][row][kDim / 8 * r + 2 * t + 1] = o[nt][t][2 + i];
      }
    }
  __syncthreads();
  constexpr int kPer = kDim / 16;   // 16 lanes a row
  // a cluster's rows of ranges: row `row` is joined by the CTA of range row % used; behind what
  // a CTA that is not as far still reads
  float (*joined)[kDim + 4] =
      reinterpret_cast<float (*)[kDim + 4]>(ring + kOwnBytes<kDim, NT>);
  const int share = (kRows + used - 1) / used;
  if (a.cluster) cluster_wait();   // the others have started
  const int d0 = (tid & 15) * kPer;
  for (int row = tid >> 4; row < kRows; row += kThreads / 16) {
    const int rho = rho0 + row;
    if (rho >= rows) break;
    float mt = kNegInf, mvt = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      mt = fmaxf(mt, sm[w][0][row]);
      mvt = fmaxf(mvt, sm[w][1][row]);
    }
    // (no weights: all V scales are 0; then 2^(topv - top) is kept from overflowing)
    const float top = mt == kNegInf ? 0.0f : mt, topv = mvt == kNegInf ? top : mvt;
    float sum = 0.0f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += sm[w][2][row] * exp2_approx(sm[w][0][row] - top);
      f[w] = exp2_approx(sm[w][1][row] - topv);
    }
    // 2^(weights' maximum - maximum) / sum; a row that sees nothing is zero
    const float norm = sum == 0.0f ? 0.0f : exp2f(topv - top) / sum;
    const float lse2 = sum == 0.0f ? kNegInf : top + log2f(sum);
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = d0 + i;
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x = fmaf(so[w][row][d], f[w], x);
      v[i] = x * norm;
    }
    if (used > 1 && a.cluster) {
      float* const to = &joined[split * share + row / used][0];
#pragma unroll
      for (int i = 0; i < kPer; i += 4)
        store_cluster4(to + d0 + i, row % used, v[i], v[i + 1], v[i + 2], v[i + 3]);
      if (d0 == 0) store_cluster(to + kDim, row % used, lse2);
    } else {
      store_row<kPer, kDim>(a, rq, h, rho, split, used, d0, v, lse2, d0 == 0);
    }
  }
  if (!a.cluster) return;
  // the ranges of a cluster, in order
  cluster_arrive();
  cluster_wait();
  if (used > 1) {
    for (int row = split + (tid >> 4) * used; row < kRows && rho0 + row < rows;
         row += kThreads / 16 * used) {
      const float* from[kMaxCluster];
      float lse[kMaxCluster], top = kNegInf, sum = 0.0f, v[kPer];
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) {
        lse[s] = kNegInf;
        if (s < used) {
          from[s] = joined[s * share + row / used];
          lse[s] = from[s][kDim];
          top = fmaxf(top, lse[s]);
        }
      }
      const float base = top == kNegInf ? 0.0f : top;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
#pragma unroll
      for (int s = 0; s < kMaxCluster; ++s) {
        if (s < used) {
          const float w = exp2f(lse[s] - base);
          sum += w;
#pragma unroll
          for (int i = 0; i < kPer; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(from[s] + d0 + i);
            v[i] = fmaf(w, x.x, v[i]);
            v[i + 1] = fmaf(w, x.y, v[i + 1]);
            v[i + 2] = fmaf(w, x.z, v[i + 2]);
            v[i + 3] = fmaf(w, x.w, v[i + 3]);
          }
        }
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] *= inv;
      store_row<kPer, kDim>(a, rq, h, rho0 + row, 0, 1, d0, v,
                            sum == 0.0f ? kNegInf : base + log2f(sum), d0 == 0);
    }
  }
}

// Joins the ranges of requests that were split.  WPR warps a row take its ranges in turn,
// eight loads in flight each; their sums are added in order.
template <int kDim, int WPR>
__global__ void __launch_bounds__(kThreads) join_kernel(const Args a) {
  constexpr int kPer = kDim / 32, kJoined = kWarps / WPR;   // rows of a CTA
  __shared__ float rows_of[WPR][kJoined][kDim + 1];
  const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = warp / kJoined;
  pdl_wait();
  pdl_trigger();
  const Request rq = request(a, b, false);
  const int used = splits_of(a, rq.kv);
  if (used <= 1) return;
  const int n = int(blockIdx.x) * kJoined + warp % kJoined;   // (token, head) of the request
  const bool live = n < rq.nq * a.q_heads;
  const int64_t row = int64_t(rq.q0) * a.q_heads + n;
  const int64_t plane = int64_t(a.tq) * a.q_heads;
  float top = kNegInf, sum = 0.0f, v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
  if (live)
    for (int s = lane; s < used; s += 32) top = fmaxf(top, a.part_lse[s * plane + row]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const float base = top == kNegInf ? 0.0f : top;
  if (live) {
    for (int s0 = g; s0 < used; s0 += 8 * WPR) {
      float w[8], x[8][kPer];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int s = s0 + j * WPR;
        w[j] = s < used ? a.part_lse[s * plane + row] : kNegInf;
        const float* p = a.part_o + (min(s, used - 1) * plane + row) * kDim + lane * kPer;
        if constexpr (kPer == 4) {
          const float4 q = *reinterpret_cast<const float4*>(p);
          x[j][0] = q.x, x[j][1] = q.y, x[j][2] = q.z, x[j][3] = q.w;
        } else {
          const float2 q = *reinterpret_cast<const float2*>(p);
          x[j][0] = q.x, x[j][1] = q.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = exp2f(w[j] - base);
        sum += f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = fmaf(f, x[j][i], v[i]);
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) rows_of[g][warp % kJoined][lane * kPer + i] = v[i];
    if (lane == 0) rows_of[g][warp % kJoined][kDim] = sum;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int j = 1; j < WPR; ++j) {
      sum += rows_of[j][warp % kJoined][kDim];
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] += rows_of[j][warp % kJoined][lane * kPer + i];
    }
  }
  if (!live) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t tok = rq.q0 + n / a.q_heads;
  uint16_t* dst = a.out + tok * a.out_stride + int64_t(n % a.q_heads) * kDim + lane * kPer;
  uint32_t w[kPer / 2];
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) w[i] = bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (a.lse && lane == 0)
    a.lse[row] = sum == 0.0f ? kNegInf : (base + log2f(sum)) * 0.6931471805599453f;
}

template <int kDim, int NT>
cudaError_t launch_decode(const Args& a, dim3 grid, cudaStream_t st) {
  constexpr size_t kOwn = kOwnBytes<kDim, NT>;
  constexpr size_t kJoin = size_t(8 * NT + kMaxCluster) * (kDim + 4) * sizeof(float);
  constexpr size_t kForThree = size_t(72) << 10;
  static_assert(kOwn + kJoin <= kForThree, "a cluster's rows");
  // Clusters get shared memory for three CTAs an SM, as the number of ranges assumes: where a
  // fourth fits, they are packed onto some SMs and leave others idle (16 x 8500 tokens, 4
  // heads: 34 us against 30).
  const size_t smem = a.cluster ? kForThree : kOwn;
  const cudaError_t e = allow_smem<decode_kernel<kDim, NT>>(std::max(kOwn, kForThree));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(decode_kernel<kDim, NT>, grid, dim3(1, 1, a.cluster ? a.n_splits : 1),
                            dim3(kThreads), smem, st, a);
}

template <int kDim>
cudaError_t launch_join(const Args& a, int32_t batch, int32_t max_q, cudaStream_t st) {
  // a warp a row for up to 8 ranges, a CTA a row beyond
  const int64_t rows = int64_t(max_q) * a.q_heads;
  if (a.n_splits <= 8)
    return launch_pdl(join_kernel<kDim, 1>,
                      dim3(unsigned((rows + kWarps - 1) / kWarps), unsigned(batch)),
                      dim3(kThreads), 0, st, a);
  return launch_pdl(join_kernel<kDim, kWarps>, dim3(unsigned(rows), unsigned(batch)),
                    dim3(kThreads), 0, st, a);
}

template <int kDim>
cudaError_t launch_dim(const Args& a, const Kv8Plan& p, int32_t batch, int32_t max_q,
                       cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (p.chunked) {
    e = launch_kv8_chunk(a, kDim, p.row_tiles, batch, st);
  } else {
    const dim3 grid(unsigned(a.kv_heads) * unsigned(p.row_tiles), unsigned(batch),
                    unsigned(p.n_splits));
    e = p.rows == 8 ? launch_decode<kDim, 1>(a, grid, st) : launch_decode<kDim, 2>(a, grid, st);
  }
  if (e != cudaSuccess || p.n_splits == 1 || a.cluster) return e;
  return launch_join<kDim>(a, batch, max_q, st);
}

}  // namespace kv8

// How a call is laid out; goes by sizes alone, so that the scratch size and the launch agree.
Kv8Plan kv8_plan(const LaunchKv8Attn& d) {
  Kv8Plan p;
  const int32_t group = d.q_heads / d.kv_heads;
  const int64_t rows = int64_t(d.max_q) * group;
  // The tensor-core kernel from 33 packed rows on: its tiles have 128.  (8 x 5 queries of 4 heads
  // over 3000 tokens, 20 rows: 33 us here, in two tiles of 16 rows, 40 there; 4 x 16 queries, 64
  // rows: 33 and 29.)
  p.chunked = rows > 32;
  p.rows = p.chunked ? 256 : rows <= 8 ? 8 : 16;
  p.row_tiles = int32_t((rows + p.rows - 1) / p.rows);
  // Ranges, none shorter than 128 tokens.  Few units: as many as fill one wave of three CTAs
  // an SM (2 x 131072 tokens, 8 heads: 86 us; 93 for four an SM, 107 in 2.7 waves; short graphs:
  // over a second of calls the 86 are 97, at the card's power limit), or the 8
  // of a cluster where that keeps a range below 512 tokens (1500 tokens, 24 heads: 6.3 us
  // against 8.3).  Many units: enough ranges for three waves of four CTAs an SM, because
  // lengths differ (64 ragged requests, 8 heads: 90 us in four ranges, 96 in two, 105 in one),
  // until there are two waves of units (200 requests: 76 us whole, 80 in two ranges).
  const int64_t units = int64_t(d.batch) * d.kv_heads * p.row_tiles;
  const int64_t sms = d.sm_count, wave = sms * 3;
  int64_t n = units * 2 <= wave  ? wave / units
              : units < sms * 8 ? (sms * 12 + units - 1) / units
                                : 1;
  n = std::min(n, (int64_t(d.max_kv) + 127) / 128);
  if (n > kv8::kMaxCluster && d.max_kv <= kv8::kMaxCluster * 512) n = kv8::kMaxCluster;
  // Chunks: ranges only where the row tiles leave half of the SMs without a CTA.
  if (p.chunked)
    n = units * 2 <= sms ? std::min(sms / units, (int64_t(d.max_kv) + 511) / 512) : 1;
  n = std::max<int64_t>(1, std::min<int64_t>(n, NVFP4_KV8_MAX_SPLITS));
  const int64_t whole = p.chunked ? 128 : 64;   // a range is whole tiles of tokens
  const int64_t chunk = ((int64_t(d.max_kv) + n - 1) / n + whole - 1) / whole * whole;
  p.chunk = int32_t(std::max(chunk, whole));
  p.n_splits = int32_t((int64_t(d.max_kv) + p.chunk - 1) / p.chunk);
  if (p.n_splits < 1) p.n_splits = 1;
  // In one wave the ranges of a unit can be a cluster, which joins them without a second
  // kernel (777 tokens, 24 heads: 5.4 us against 7.6); in several, CTAs that wait for their
  // cluster hold up others (64 ragged requests: 121 us against 94).
  p.cluster = !p.chunked && p.n_splits > 1 && p.n_splits <= kv8::kMaxCluster &&
              units * p.n_splits <= wave;
  p.scratch = p.n_splits == 1 || p.cluster
                  ? 0
                  : size_t(p.n_splits) * size_t(d.tq) * size_t(d.q_heads) *
                        size_t(d.head_dim + 1) * sizeof(float);
  return p;
}

cudaError_t launch_kv8_attention(const LaunchKv8Attn& d, cudaStream_t st) {
  const Kv8Plan p = kv8_plan(d);
  kv8::Args a;
  a.q = static_cast<const uint16_t*>(d.q);
  a.q_stride = d.q_stride;
  a.out = static_cast<uint16_t*>(d.out);
  a.out_stride = d.out_stride;
  a.lse = d.lse;
  a.cu_q = d.cu_q;
  a.kv_lens = d.kv_lens;
  a.table = d.table;
  a.table_stride = d.table_stride;
  a.k_codes = d.k_codes;
  a.v_codes = d.v_codes;
  a.k_scale = d.k_scale;
  a.v_scale = d.v_scale;
  a.tq = int32_t(d.tq);
  a.q_heads = d.q_heads;
  a.kv_heads = d.kv_heads;
  a.group = d.q_heads / d.kv_heads;
  a.group_div = make_fastdiv(uint32_t(a.group));
  a.max_q = d.max_q;
  a.max_tokens = int32_t(int64_t(d.max_pages) * d.page_tokens);
  a.n_pages = d.n_pages;
  a.page_tokens = d.page_tokens;
  a.page_div = make_fastdiv(uint32_t(d.page_tokens));
  a.causal = d.causal;
  a.scale_log2 = d.scale_log2;
  a.chunk = p.chunk;
  a.n_splits = p.n_splits;
  a.cluster = p.cluster;
  a.part_o = static_cast<float*>(d.scratch);
  a.part_lse = a.part_o + int64_t(p.n_splits) * d.tq * d.q_heads * d.head_dim;
  a.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(d.ws) + kWsStatus);
  a.wait_limit_ns = d.wait_limit_ns;
  return d.head_dim == 64 ? kv8::launch_dim<64>(a, p, d.batch, d.max_q, st)
                          : kv8::launch_dim<128>(a, p, d.batch, d.max_q, st);
}

}  // namespace nvfp4
