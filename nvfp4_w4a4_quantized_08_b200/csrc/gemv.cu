// gemv.cu -- matrix-vector products with NVFP4 weights: the linear layer of a
// few rows (up to 16) whose activations stay bf16 or fp32.
//
//   y[m][n] = act(s_t sum_k x[m][k] v(q[n][k]) s_b[n][k / 16])
//
// Bound by the weights: N K 9/16 bytes are read once, everything else is small.
// What the arithmetic has to keep up with is ~42 codes a clock and SM at the
// measured HBM rate, which rules out scalar fp32 products (two instructions a
// code and row); so the codes go through the tensor cores as fp16:
//   - v(q) s_b is exact in fp16: a 2-bit times a 4-bit significand, magnitudes
//     2^-10 .. 2688.  One hardware conversion per two codes, one packed multiply.
//   - x is scaled by a power of two per row and 256 columns to magnitudes below
//     2^9 and converted to fp16: exact for bf16 values within 2^-22 of the
//     largest of the 256, below that an error of at most 2^-33 of the largest.
//     fp32 x takes two fp16 parts (the second is the remainder times 2^11) in
//     two columns of the product, 22 bits together.
//   - m16n8k16 with fp32 accumulation: 16 weight rows by 8 columns, the columns
//     being the rows of x (or their parts).  The 16 products of a 256-column step
//     start from zero and are joined to the fp32 sum by one FMA with the step's
//     power of two, which also bounds the tensor core's truncation to 16 sums.
// The order of the 16 columns inside one product is free as long as both
// operands use the same one, so a thread's 32 bytes of codes (64 columns, four
// scale blocks) feed 16 products without any exchange between threads.
//
// A warp takes steps of 32 weight rows by 256 columns (16 rows for the widest x): 128 bytes, a
// whole line, of each row, copied asynchronously into a ring of its own two steps deep.  (Loads
// straight into registers, 64 bytes of a row at a time and 16 rows a warp, took 17.4 us for
// 14336 x 4096 and one row, 13.7 with 32 rows; the rings took 11.5 at first.  Three steps deep
// leaves one CTA an SM: 17 us.)  A CTA has 8 warps: KW of them split the columns (steps dealt out
// in turn), the other factor 8 / KW takes further rows, which then share the converted x; KW falls
// with the rows of x, so that the conversion stays a small part of the work.  For one or two rows
// a warp converts what it reads itself, and no barrier is needed (14336 x 4096: 10.5 us against
// 11.3).  (Converting all of x first, in a prologue, cost 0.7 us at 1024 x 1024.)  The 16 weight
// rows of a product are 4 i-values by 4 rows 32 apart: the scale tile of the tensor-core layout
// keeps their scales in 64 contiguous bytes.  Where rows alone leave SMs idle, a cluster of up to
// 8 CTAs splits the columns again; each CTA stores its sums to the one that finishes them, which
// adds them in rank order: no workspace, no atomics, the same result every time.  (Fetching the
// others' sums instead took 2 us a CTA of the cluster: 7 x 5000 x 14336 in clusters of 6 37 us
// against 23.)
//
// 1 x 1024 x 1024 2.1 us (the launch, one step, the join of the warps); 1 x 14336 x 4096 with its
// GELU 10.7 us, 47% of the copy rate: 224 CTAs, so that half of the SMs have two and half one, and
// 12 to 16 warps an SM (issue slots 47% in use); 7 x 5000 x 14336 in fp32 21.5 us, 29%, the
// conversions' and products' latency with 16 warps an SM.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace gemv {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 256;         // columns a warp takes at a time
constexpr int kStages = 2;         // steps of weights in a warp's ring
constexpr int kXRow = 576;         // bytes of one converted row-step: 512 and a bank offset
constexpr int kMaxCluster = 8;

struct Args {
  const void* x;          // bf16 or fp32 [M][ldx]
  int64_t ldx;
  const uint8_t* codes;   // [N][K / 2]
  const uint8_t* sf;
  const float* s_t;
  void* y;                // bf16 or fp32 [M][ldy]
  int64_t ldy;
  int32_t M, N, K;
  int32_t sf_tiled;       // tensor-core layout of the scales (else row-major)
  int32_t y_bf16, act;
  FastDiv m_div;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 codes -> four fp16 pairs (codes 2i, 2i + 1), exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 16 bytes to shared memory, zeros where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float gelu_tanh(float y) {
  // y (1 + tanh u) / 2 = y / (1 + exp(-2u)), without the cancellation for y below 0 (there
  // 1 + tanh u has no more than the last bits of 1); exp overflows to inf where the result is -0
  const float u = 0.7978845608028654f * (y + 0.044715f * y * y * y);
  return y / (1.0f + expf(-2.0f * u));
}

// Products of 16 weight rows per warp (one where four tiles of columns fill the registers).
template <int NT>
constexpr int kRowTiles = NT < 4 ? 2 : 1;

// Shared memory: the rings, or after the last step the warps' sums; then KW M <= 16 row-steps
// of x, twice.
template <int NT>
constexpr int kRingBytes = std::max(kWarps * kStages * kRowTiles<NT> * 16 * (kStep / 2),
                                    kWarps * kRowTiles<NT> * 16 * (NT * 8 + 1) * 4);
template <bool FP32>
constexpr int kXBytes = 2 * 16 * (FP32 ? 2 : 1) * kXRow;

// Sums of a cluster's CTAs: KW M <= 16.
template <int KW, int NT>
constexpr int kJoinBytes = (kWarps / KW * kRowTiles<NT> * 16 * (16 / KW) + kMaxCluster) * 4;

// KW warps split the columns; NT tiles of 8 product columns; FP32 x in two parts.
// SELF: every warp converts its own x (M <= 2), which needs no barrier.
template <int KW, int NT, bool FP32, bool SELF>
__global__ void __launch_bounds__(kThreads, 2) gemv_kernel(const Args a) {
  constexpr int kTiles = kRowTiles<NT>;
  constexpr int RG = kWarps / KW;          // groups of 16 kTiles weight rows
  constexpr int kOf128 = 8 / kTiles;       // groups of a 128-row tile
  constexpr int kPairs = 16;               // row-steps converted at a time (KW M <= 16)
  constexpr int kPasses = kPairs / kWarps; // of them by one warp
  constexpr int kParts = FP32 ? 2 : 1;
  constexpr int kCols = NT * 8;
  constexpr int kStage = kTiles * 16 * (kStep / 2);   // bytes of weights
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float xe[2][kPairs];          // power of two of each row-step
  // the rings, and after the last step the warps' sums in their place; then converted x
  float (*red)[kTiles * 16][kCols + 1] = reinterpret_cast<float (*)[kTiles * 16][kCols + 1]>(smem);
  uint8_t* xs = smem + (kRingBytes<NT> + 15) / 16 * 16;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kw = warp % KW, rg = warp / KW;
  const int r = lane >> 2, c = lane & 3;
  const int cs = int(cluster_size()), rank = int(cluster_rank());
  if (cs > 1) cluster_arrive();   // waited for before the first store to another CTA
  const int group0 = int(blockIdx.x) / cs * RG;
  const int n_steps = (a.K + kStep - 1) / kStep;
  const int stride = KW * cs;                          // steps between a warp's own
  const int iters = (n_steps + stride - 1) / stride;   // the same for every CTA of a cluster
  const int first = rank * KW + kw;
  const int group = group0 + rg;

  // weight row of row rho of product t: 4 (kTiles g + t) + rho % 4 + 32 (rho / 4) of a
  // 128-row tile
  auto row_of = [&](int t, int rho) {
    return min(group / kOf128 * 128 + (kTiles * (group % kOf128) + t) * 4 + (rho & 3) +
                   32 * (rho >> 2),
               a.N - 1);
  };
  // copies: lane l takes 16-byte unit l % 8 of rows l / 8 + 4 i; units exchanged by the row's
  // place, so that the reads below meet no bank twice
  uint32_t from[kTiles * 4];   // in units of 16 bytes: below 2^30
  uint32_t to[4];
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                        uint32_t(warp) * kStages * kStage;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rho = lane / 8 + 4 * i;
    to[i] = ring + rho * 128 + (((lane & 7) ^ (rho & 7)) << 4);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
      from[4 * t + i] = uint32_t(row_of(t, rho)) * uint32_t(a.K / 32) + (lane & 7);
  }
  auto issue = [&](int i) {   // step i of this warp
    const int st = first + i * stride;
    if (i < iters && st < n_steps) {
      const uint32_t in = st * kStep + 32 * (lane & 7) < a.K ? 16 : 0;
      const uint32_t stage = uint32_t(i % kStages) * kStage;
      const uint32_t at = in ? uint32_t(st) * (kStep / 32) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          copy16(to[j] + stage + t * 16 * (kStep / 2),
                 a.codes + 16 * int64_t(from[4 * t + j] + at), in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // scales: the four of blocks 4 c .. 4 c + 3 of rows r and r + 8, two steps ahead
  int32_t s_at[kTiles][2];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = row_of(t, r + 8 * i);
      s_at[t][i] = a.sf_tiled ? ((row >> 7) * ((a.K / 16 + 3) / 4) + c) * 512 + (row & 31) * 16 +
                                    ((row >> 5) & 3) * 4
                              : row * (a.K / 16) + 4 * c;
    }
  auto load_s = [&](int i, uint32_t (&sc)[kTiles][2]) {
    const int st = first + i * stride;
    const int left = i < iters ? a.K / 16 - st * (kStep / 16) - 4 * c : 0;   // blocks (even)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[t][j] = 0;
        if (left > 0) {
          if (a.sf_tiled) {   // (padded to whole tiles with zeros)
            sc[t][j] = __ldg(reinterpret_cast<const uint32_t*>(a.sf + s_at[t][j] + st * 2048));
          } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(a.sf + s_at[t][j] + st * 16);
            sc[t][j] = __ldg(p);
            if (left > 2) sc[t][j] |= uint32_t(__ldg(p + 1)) << 16;
          }
        }
      }
  };

  // conversion: a warp takes a row-step, 8 columns a lane.  With KW = 8 its own step's rows, else
  // row-steps `warp` and `warp + 8` of the CTA's.
  struct Eight {
    uint4 v[kParts];
  };
  Eight xv[kPasses];
  auto pair_of = [&](int p, int& step_of, int& m) {
    const int pair = warp + kWarps * p;
    step_of = SELF ? kw : int(fast_div(a.m_div, uint32_t(pair)));
    m = SELF ? p : pair - step_of * a.M;
    return SELF ? p < a.M : step_of < KW;
  };
  auto load_x = [&](int i) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      int step_of, m;
      const bool on = pair_of(p, step_of, m);
      const int col = (rank * KW + step_of + i * stride) * kStep + 8 * lane;
#pragma unroll
      for (int e = 0; e < kParts; ++e) xv[p].v[e] = make_uint4(0, 0, 0, 0);
      if (on && i < iters && col < a.K) {
        if constexpr (FP32) {
          const float* x = static_cast<const float*>(a.x) + m * a.ldx + col;
          xv[p].v[0] = ld_nc_v4_l1(x);
          xv[p].v[1] = ld_nc_v4_l1(x + 4);
        } else {
          xv[p].v[0] = ld_nc_v4_l1(static_cast<const uint16_t*>(a.x) + m * a.ldx + col);
        }
      }
    }
  };
  auto convert_x = [&](int buf) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      int step_of, m;
      if (!pair_of(p, step_of, m)) continue;   // the same for the whole warp
      float f[8];
      const uint4 v0 = xv[p].v[0];
      if constexpr (FP32) {
        const uint4 v1 = xv[p].v[1];
        f[0] = __uint_as_float(v0.x); f[1] = __uint_as_float(v0.y);
        f[2] = __uint_as_float(v0.z); f[3] = __uint_as_float(v0.w);
        f[4] = __uint_as_float(v1.x); f[5] = __uint_as_float(v1.y);
        f[6] = __uint_as_float(v1.z); f[7] = __uint_as_float(v1.w);
      } else {
        const uint32_t w[4] = {v0.x, v0.y, v0.z, v0.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = __uint_as_float(w[i] << 16);
          f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      // 2^e with max |x| 2^e in [2^8, 2^9), kept where its inverse is normal too
      const uint32_t field = min(262u - (top >> 23), 253u);
      const float scale = __uint_as_float(field << 23);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = f[2 * i] * scale, v = f[2 * i + 1] * scale;
        hi[i] = f16x2_rn(u, v);
        if constexpr (FP32) {
          const __half2 h = *reinterpret_cast<const __half2*>(&hi[i]);
          lo[i] = f16x2_rn((u - __low2float(h)) * 2048.0f, (v - __high2float(h)) * 2048.0f);
          // an infinity is whole in its first part (inf - inf is not)
          if (top >= 0x7F800000u) lo[i] = 0;
        }
      }
      // columns 64 c + 8 q .. of a step (lane 8 c + q): unit 4 q + c of its row, so that the
      // reads below, lanes c of one q, are 64 contiguous bytes
      const int pair = (SELF ? warp : step_of) * a.M + m;
      uint8_t* d = xs + (buf * kPairs + pair) * kParts * kXRow +
                   ((lane & 7) * 4 + (lane >> 3)) * 16;
      *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (FP32)
        *reinterpret_cast<uint4*>(d + kXRow) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (lane == 0) xe[buf][pair] = __uint_as_float((254u - field) << 23);
    }
  };

  float acc[kTiles][NT][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][n][i] = 0.0f;
  const int cols = a.M * kParts;   // product column n: row n / kParts, part n % kParts

  auto step = [&](int i, int buf, const uint32_t (&sc)[kTiles][2]) {
    float d[kTiles][NT][4];
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[t][n][j] = 0.0f;
    const uint32_t stage = ring + uint32_t(i % kStages) * kStage;
    const uint8_t* xb = xs + (buf * kPairs + (SELF ? warp : kw) * a.M) * kParts * kXRow + c * 16;
    // halves of a lane's 32 bytes: two scale blocks, 8 products each
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 w[kTiles][2];
      uint32_t s2[kTiles][2][2];   // the block scales of rows r and r + 8, both halves of a pair
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t rho = r + 8 * j;
          w[t][j] = lds16(stage + t * 16 * (kStep / 2) + rho * 128 +
                          (((2 * c + half) ^ (rho & 7)) << 4));
          uint32_t h;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
              : "=r"(h)
              : "h"((unsigned short)(sc[t][j] >> (16 * half))));
          s2[t][j][0] = prmt(h, h, 0x1010);
          s2[t][j][1] = prmt(h, h, 0x3232);
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n] = make_uint4(0, 0, 0, 0);
          if (8 * n + r < cols)
            b[n] = *reinterpret_cast<const uint4*>(xb + (8 * n + r) * kXRow + (4 * half + k) * 64);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          uint32_t h[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4& q = w[t][j];
            codes_f16(k == 0 ? q.x : k == 1 ? q.y : k == 2 ? q.z : q.w, h[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[j][e] = mul_f16x2(h[j][e], s2[t][j][k >> 1]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(d[t][n], h[0][0], h[1][0], h[0][1], h[1][1], b[n].x, b[n].y);
            mma_f16(d[t][n], h[0][2], h[1][2], h[0][3], h[1][3], b[n].z, b[n].w);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int n0 = 8 * n + 2 * c;
      const float* e = xe[buf] + (SELF ? warp : kw) * a.M;
      const float e0 = n0 < cols ? e[n0 / kParts] : 0.0f;
      const float e1 = n0 + 1 < cols ? e[(n0 + 1) / kParts] : 0.0f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        acc[t][n][0] = fmaf(d[t][n][0], e0, acc[t][n][0]);
        acc[t][n][1] = fmaf(d[t][n][1], e1, acc[t][n][1]);
        acc[t][n][2] = fmaf(d[t][n][2], e0, acc[t][n][2]);
        acc[t][n][3] = fmaf(d[t][n][3], e1, acc[t][n][3]);
      }
    }
  };

  pdl_wait();
  pdl_trigger();
  load_x(0);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  uint32_t sc[2][kTiles][2];
  load_s(0, sc[0]);
  load_s(1, sc[1]);
  for (int i0 = 0; i0 < iters; i0 += 2) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = i0 + j;
      if (i < iters) {
        convert_x(j);
        load_x(i + 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        // the step's weights and x are there; x's buffer j is written again two steps on, after
        // the next barrier, which every reader of this step has then passed
        if constexpr (SELF) __syncwarp(); else __syncthreads();
        issue(i + kStages - 1);
        if (first + i * stride < n_steps) step(i, j, sc[j]);
        load_s(i + 2, sc[j]);
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();   // the rings are free for the sums

  // sums of the warps that split the columns, then of the cluster's CTAs
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      red[warp][16 * t + r][8 * n + 2 * c] = acc[t][n][0];
      red[warp][16 * t + r][8 * n + 2 * c + 1] = acc[t][n][1];
      red[warp][16 * t + r + 8][8 * n + 2 * c] = acc[t][n][2];
      red[warp][16 * t + r + 8][8 * n + 2 * c + 1] = acc[t][n][3];
    }
  __syncthreads();
  const float st = __ldg(a.s_t);
  constexpr int kRun = 4 * kTiles * RG;   // consecutive weight rows of each 32
  auto finish = [&](int o, float sum) {
    const int i4 = o % kRun, q = (o / kRun) & 3, m = o / (4 * kRun);
    const int grp = group0 + i4 / (4 * kTiles);
    const int n = grp / kOf128 * 128 + grp % kOf128 * (4 * kTiles) + i4 % (4 * kTiles) + 32 * q;
    if (n >= a.N) return;
    float y = sum * st;
    if (a.y_bf16) {
      if (a.act == NVFP4_ACT_GELU_TANH) y = gelu_tanh(__bfloat162float(__float2bfloat16_rn(y)));
      static_cast<__nv_bfloat16*>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(y);
    } else {
      if (a.act == NVFP4_ACT_GELU_TANH) y = gelu_tanh(y);
      static_cast<float*>(a.y)[m * a.ldy + n] = y;
    }
  };
  // a rank finishes `share` of the outputs; the others store their sums of them to it
  const int total = RG * kTiles * 16 * a.M;
  const int share = (total + cs - 1) / cs;
  float* const joined = reinterpret_cast<float*>(xs + kXBytes<FP32>);   // [cs][share]
  if (cs > 1) cluster_wait();   // the others have started
  for (int o = tid; o < total; o += kThreads) {
    const int i4 = o % kRun, q = (o / kRun) & 3, m = o / (4 * kRun);
    const int g = i4 / (4 * kTiles), rho = 16 * ((i4 >> 2) % kTiles) + (i4 & 3) + 4 * q;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const float* p = &red[g * KW + w][rho][m * kParts];
      float v = p[0];
      if constexpr (FP32) v = fmaf(p[1], 0x1p-11f, v);
      sum += v;
    }
    if (cs == 1) {
      finish(o, sum);
    } else {
      const int owner = o / share;
      store_cluster(joined + rank * share + (o - owner * share), owner, sum);
    }
  }
  if (cs == 1) return;
  cluster_arrive();
  cluster_wait();
  for (int i = tid; i < share && rank * share + i < total; i += kThreads) {
    float sum = 0.0f;
    for (int k = 0; k < cs; ++k) sum += joined[k * share + i];
    finish(rank * share + i, sum);
  }
}

template <int KW, int NT>
int ctas_of(const Args& a) {
  constexpr int RG = kWarps / KW;
  const int groups = (a.N + 127) / 128 * (8 / kRowTiles<NT>);
  return (groups + RG - 1) / RG;
}

// How many CTAs split the columns, and what that costs in quarters of a step: a CTA's steps,
// 5/4 as long where SMs have two CTAs, in as many waves as it takes (2 CTAs an SM, of clusters
// 7/4); the join.  7 x 5000 x 14336, fp32: 73 us in 40 CTAs, 29.5 in 120, 29.3 in 160, 23.1 in
// 240, 30.4 in 280 (two waves); 16 x 9216 x 5120: 52 in 36, 23.1 in 144, 17.3 in 252, 27 in 288;
// 1 x 1024 x 12800: 9.5 in 32, 5.1 in 128, 6.5 in 160, 4.6 in 224.
template <int KW>
int split_of(int ctas, int n_steps, int sm_count, int& cost) {
  int best = 1;
  cost = INT32_MAX;
  for (int cs = 1; cs <= kMaxCluster; ++cs) {
    const int64_t n = int64_t(ctas) * cs, room = cs == 1 ? 2 * sm_count : sm_count * 7 / 4;
    const int64_t waves = (n + room - 1) / room, iters = (n_steps + KW * cs - 1) / (KW * cs);
    const int64_t c = waves * iters * (n > sm_count ? 5 : 4) + (waves - 1) + (cs > 1);
    if (c < cost) {
      cost = int(c);
      best = cs;
    }
  }
  return best;
}

template <int KW, int NT, bool FP32, bool SELF = false>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t st) {
  const int ctas = ctas_of<KW, NT>(a);
  int cost;
  const int cs = split_of<KW>(ctas, (a.K + kStep - 1) / kStep, sm_count, cost);
  constexpr size_t kSmem = (kRingBytes<NT> + 15) / 16 * 16 + kXBytes<FP32> + kJoinBytes<KW, NT>;
  const cudaError_t e = allow_smem<gemv_kernel<KW, NT, FP32, SELF>>(kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(gemv_kernel<KW, NT, FP32, SELF>, dim3(unsigned(ctas * cs)),
                            dim3(unsigned(cs)), dim3(kThreads), kSmem, st, a);
}

// One or two rows: all warps on one group of weight rows, or, where that fills the SMs worse,
// four (1 x 14336 x 4096: 10.6 us with four against 11.8; 1 x 9216 x 5120 13.5 against 7.5).
bool all_on_one(const Args& a, int sm_count) {
  const int n_steps = (a.K + kStep - 1) / kStep;
  int eight, four;
  split_of<8>(ctas_of<8, 1>(a), n_steps, sm_count, eight);
  split_of<4>(ctas_of<4, 1>(a), n_steps, sm_count, four);
  return eight <= four;
}

}  // namespace gemv

cudaError_t launch_gemv(const LaunchGemv& g, cudaStream_t st) {
  gemv::Args a;
  a.x = g.x;
  a.ldx = g.ldx;
  a.codes = g.w_codes;
  a.sf = g.w_sf;
  a.s_t = g.w_st;
  a.y = g.y;
  a.ldy = g.ldy;
  a.M = int32_t(g.M);
  a.N = int32_t(g.N);
  a.K = int32_t(g.K);
  a.sf_tiled = g.sf_layout == NVFP4_SF_MMA128x4;
  a.y_bf16 = g.y_dtype == NVFP4_BF16;
  a.act = g.act;
  a.m_div = make_fastdiv(uint32_t(a.M));
  // KW M <= 16 row-steps are converted at a time; 8 NT >= product columns
  const bool one = g.M <= 2 && gemv::all_on_one(a, g.sm_count);
  if (g.x_dtype == NVFP4_BF16) {
    if (one) return gemv::launch<8, 1, false, true>(a, g.sm_count, st);
    if (g.M <= 2) return gemv::launch<4, 1, false, true>(a, g.sm_count, st);
    if (g.M <= 4) return gemv::launch<4, 1, false>(a, g.sm_count, st);
    if (g.M <= 8) return gemv::launch<2, 1, false>(a, g.sm_count, st);
    return gemv::launch<1, 2, false>(a, g.sm_count, st);
  }
  if (one) return gemv::launch<8, 1, true, true>(a, g.sm_count, st);
  if (g.M <= 2) return gemv::launch<4, 1, true, true>(a, g.sm_count, st);
  if (g.M <= 4) return gemv::launch<4, 1, true>(a, g.sm_count, st);
  if (g.M <= 8) return gemv::launch<2, 2, true>(a, g.sm_count, st);
  return gemv::launch<1, 4, true>(a, g.sm_count, st);
}

}  // namespace nvfp4
