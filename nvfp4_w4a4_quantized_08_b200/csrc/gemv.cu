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
//   - x is scaled by a power of two per row and 128 columns to magnitudes below
//     2^9 and converted to fp16: exact for bf16 values within 2^-22 of the
//     largest of the 128, below that an error of at most 2^-33 of the largest.
//     fp32 x takes two fp16 parts (the second is the remainder times 2^11) in
//     two columns of the product, 22 bits together.
//   - m16n8k16 with fp32 accumulation: 16 weight rows by 8 columns, the columns
//     being the rows of x (or their parts).  The 8 products of a 128-column step
//     start from zero and are joined to the fp32 sum by one FMA with the step's
//     power of two, which also bounds the tensor core's truncation to 8 sums.
// The order of the 16 columns inside one product is free as long as both
// operands use the same one, so a thread's 16-byte load of codes (32 columns,
// two scale blocks) feeds 8 products without any exchange between threads.
//
// A CTA has 8 warps: KW of them split the columns (steps dealt out in turn),
// the other factor 8 / KW takes further rows, which then share the converted x.
// KW falls with the rows of x (8 warps convert at most 16 row-steps at a time),
// so the conversion stays a small part of the work.  The 16 weight rows of a
// warp are 4 i-values by 4 rows 32 apart: the scale tile of the tensor-core
// layout keeps exactly their scales in 64 contiguous bytes.  Where rows alone
// leave SMs idle, a cluster of up to 8 CTAs splits the columns again and joins
// the sums through distributed shared memory in rank order: no workspace, no
// atomics, the same result every time.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {
namespace gemv {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 128;         // columns a warp takes at a time
constexpr int kDepth = 4;          // steps of weight loads in flight per warp
constexpr int kXRow = 320;         // bytes of one converted row-step: 256 and a bank offset
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
  const float u = 0.7978845608028654f * (y + 0.044715f * y * y * y);
  return 0.5f * y * (1.0f + tanhf(u));
}

// KW warps split the columns; NT tiles of 8 product columns; FP32 x in two parts.
template <int KW, int NT, bool FP32>
__global__ void __launch_bounds__(kThreads, 2) gemv_kernel(const Args a) {
  namespace cg = cooperative_groups;
  constexpr int RG = kWarps / KW;          // row groups of 16 weight rows
  constexpr int kPairs = 16;               // row-steps converted at a time (KW M <= 16)
  constexpr int kParts = FP32 ? 2 : 1;
  constexpr int kCols = NT * 8;
  __shared__ alignas(16) uint8_t xs[2][kPairs * kParts * kXRow];
  __shared__ float xe[2][kPairs];          // power of two of each row-step
  __shared__ float red[kWarps][16][kCols + 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kw = warp % KW, rg = warp / KW;
  const int r = lane >> 2, c = lane & 3;
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int group0 = int(blockIdx.x) / cs * RG;
  const int n_steps = (a.K + kStep - 1) / kStep;
  const int stride = KW * cs;                          // steps between a warp's own
  const int iters = (n_steps + stride - 1) / stride;   // the same for every CTA of a cluster

  // weight row of tensor-core row rho: 4 g + rho % 4 + 32 (rho / 4) of its 128-row tile
  const int group = group0 + rg;
  const int row0 = (group >> 3) * 128 + (group & 7) * 4 + (r & 3) + 32 * (r >> 2);
  const int ra = min(row0, a.N - 1), rb = min(row0 + 64, a.N - 1);
  const int64_t pitch = a.K / 2;
  const uint8_t* wa = a.codes + ra * pitch + 16 * c;
  const uint8_t* wb = a.codes + rb * pitch + 16 * c;
  const uint8_t *sa, *sb;
  int64_t s_step;
  if (a.sf_tiled) {
    const int64_t tiles = (a.K / 16 + 3) / 4;
    auto at = [&](int row) {
      return a.sf + (int64_t(row >> 7) * tiles + (c >> 1)) * 512 + (row & 31) * 16 +
             ((row >> 5) & 3) * 4 + (c & 1) * 2;
    };
    sa = at(ra);
    sb = at(rb);
    s_step = 1024;
  } else {
    sa = a.sf + int64_t(ra) * (a.K / 16) + 2 * c;
    sb = a.sf + int64_t(rb) * (a.K / 16) + 2 * c;
    s_step = 8;
  }
  const int first = rank * KW + kw;

  pdl_wait();
  pdl_trigger();

  uint4 wq[kDepth][2];
  uint32_t sq[kDepth][2];
  // step i of this warp: columns [128 s + 32 c, + 32) are all inside K or all outside
  auto load_w = [&](int i, uint4 (&w)[2], uint32_t (&s)[2]) {
    const int st = first + i * stride;
    if (st * kStep + 32 * c < a.K) {
      w[0] = ld_nc_v4(wa + int64_t(st) * (kStep / 2));
      w[1] = ld_nc_v4(wb + int64_t(st) * (kStep / 2));
      s[0] = __ldg(reinterpret_cast<const uint16_t*>(sa + st * s_step));
      s[1] = __ldg(reinterpret_cast<const uint16_t*>(sb + st * s_step));
    } else {
      w[0] = w[1] = make_uint4(0, 0, 0, 0);
      s[0] = s[1] = 0;
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load_w(i, wq[i], sq[i]);

  // conversion: half warp p takes row-step p = kw' * M + m, thread u its columns 8 u ..
  const int pair = tid >> 4, u = tid & 15;
  const int cv_kw = pair / a.M, cv_m = pair % a.M;
  const bool cv = cv_kw < KW;
  uint4 xv[kParts];
  auto load_x = [&](int i) {
    const int col = (rank * KW + cv_kw + i * stride) * kStep + 8 * u;
    xv[0] = make_uint4(0, 0, 0, 0);
    if constexpr (FP32) xv[1] = xv[0];
    if (cv && i < iters && col < a.K) {
      if constexpr (FP32) {
        const float* p = static_cast<const float*>(a.x) + cv_m * a.ldx + col;
        xv[0] = ld_nc_v4_l1(p);
        xv[1] = ld_nc_v4_l1(p + 4);
      } else {
        xv[0] = ld_nc_v4_l1(static_cast<const uint16_t*>(a.x) + cv_m * a.ldx + col);
      }
    }
  };
  auto convert_x = [&](int buf) {
    float f[8];
    if constexpr (FP32) {
      f[0] = __uint_as_float(xv[0].x); f[1] = __uint_as_float(xv[0].y);
      f[2] = __uint_as_float(xv[0].z); f[3] = __uint_as_float(xv[0].w);
      f[4] = __uint_as_float(xv[1].x); f[5] = __uint_as_float(xv[1].y);
      f[6] = __uint_as_float(xv[1].z); f[7] = __uint_as_float(xv[1].w);
    } else {
      const uint32_t w[4] = {xv[0].x, xv[0].y, xv[0].z, xv[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    // 2^e with max |x| 2^e in [2^8, 2^9), kept where its inverse is normal too
    const uint32_t field = min(262u - (top >> 23), 253u);
    const float scale = __uint_as_float(field << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = f[2 * i] * scale, q = f[2 * i + 1] * scale;
      hi[i] = f16x2_rn(p, q);
      if constexpr (FP32) {
        const __half2 h = *reinterpret_cast<const __half2*>(&hi[i]);
        lo[i] = f16x2_rn((p - __low2float(h)) * 2048.0f, (q - __high2float(h)) * 2048.0f);
      }
    }
    if (cv) {
      const uint32_t at = ((u & 3) * 4 + (u >> 2)) * 16;
      uint8_t* d = xs[buf] + (cv_kw * a.M + cv_m) * kParts * kXRow + at;
      *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if constexpr (FP32)
        *reinterpret_cast<uint4*>(d + kXRow) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (u == 0) xe[buf][cv_kw * a.M + cv_m] = __uint_as_float((254u - field) << 23);
    }
  };

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.0f;
  const int cols = a.M * kParts;   // product column n: row n / kParts, part n % kParts

  auto step = [&](int buf, const uint4 (&w)[2], const uint32_t (&s)[2]) {
    float d[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) d[t][i] = 0.0f;
    // the two block scales of each weight row, both halves of a pair
    uint32_t s2[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)s[i]));
      s2[i][0] = prmt(h, h, 0x1010);
      s2[i][1] = prmt(h, h, 0x3232);
    }
    const uint32_t wa4[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    const uint32_t wb4[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
    const uint8_t* xb = xs[buf] + kw * cols * kXRow + c * 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t ha[4], hb[4];
      codes_f16(wa4[q], ha);
      codes_f16(wb4[q], hb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ha[i] = mul_f16x2(ha[i], s2[0][q >> 1]);
        hb[i] = mul_f16x2(hb[i], s2[1][q >> 1]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint4 b = make_uint4(0, 0, 0, 0);
        if (8 * t + r < cols)
          b = *reinterpret_cast<const uint4*>(xb + (8 * t + r) * kXRow + q * 64);
        mma_f16(d[t], ha[0], hb[0], ha[1], hb[1], b.x, b.y);
        mma_f16(d[t], ha[2], hb[2], ha[3], hb[3], b.z, b.w);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int n0 = 8 * t + 2 * c;
      const float* e = xe[buf] + kw * a.M;
      const float e0 = n0 < cols ? e[n0 / kParts] : 0.0f;
      const float e1 = n0 + 1 < cols ? e[(n0 + 1) / kParts] : 0.0f;
      acc[t][0] = fmaf(d[t][0], e0, acc[t][0]);
      acc[t][1] = fmaf(d[t][1], e1, acc[t][1]);
      acc[t][2] = fmaf(d[t][2], e0, acc[t][2]);
      acc[t][3] = fmaf(d[t][3], e1, acc[t][3]);
    }
  };

  load_x(0);
  for (int i0 = 0; i0 < iters; i0 += kDepth) {
#pragma unroll
    for (int j = 0; j < kDepth; ++j) {
      const int i = i0 + j;
      if (i < iters) {
        convert_x(j & 1);
        load_x(i + 1);
        // one barrier a step: buffer j & 1 is written again two steps on, after
        // the next barrier, which every reader of this step has then passed
        __syncthreads();
        step(j & 1, wq[j], sq[j]);
        load_w(i + kDepth, wq[j], sq[j]);
      }
    }
  }

  // sums of the warps that split the columns, then of the cluster's CTAs
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    red[warp][r][8 * t + 2 * c] = acc[t][0];
    red[warp][r][8 * t + 2 * c + 1] = acc[t][1];
    red[warp][r + 8][8 * t + 2 * c] = acc[t][2];
    red[warp][r + 8][8 * t + 2 * c + 1] = acc[t][3];
  }
  if (cs > 1) cluster.sync(); else __syncthreads();
  const float st = __ldg(a.s_t);
  for (int o = rank * kThreads + tid; o < RG * 16 * a.M; o += kThreads * cs) {
    // consecutive threads: the 4 RG consecutive weight rows of each 32
    const int i4 = o % (4 * RG), q = (o / (4 * RG)) & 3, m = o / (16 * RG);
    const int g = i4 >> 2, rho = (i4 & 3) + 4 * q;
    const int grp = group0 + g;
    const int n = (grp >> 3) * 128 + (grp & 7) * 4 + (i4 & 3) + 32 * q;
    float sum = 0.0f;
    for (int k = 0; k < cs; ++k) {
      const float* base =
          cs > 1 ? cluster.map_shared_rank(&red[0][0][0], k) : &red[0][0][0];
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float* p = base + ((g * KW + w) * 16 + rho) * (kCols + 1) + m * kParts;
        float v = p[0];
        if constexpr (FP32) v = fmaf(p[1], 0x1p-11f, v);
        sum += v;
      }
    }
    if (n < a.N) {
      float y = sum * st;
      if (a.y_bf16) {
        if (a.act == NVFP4_ACT_GELU_TANH) y = gelu_tanh(__bfloat162float(__float2bfloat16_rn(y)));
        static_cast<__nv_bfloat16*>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(y);
      } else {
        if (a.act == NVFP4_ACT_GELU_TANH) y = gelu_tanh(y);
        static_cast<float*>(a.y)[m * a.ldy + n] = y;
      }
    }
  }
  if (cs > 1) cluster.sync();   // peers read this CTA's shared memory until here
}

template <int KW, int NT, bool FP32>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t st) {
  constexpr int RG = kWarps / KW;
  const int groups = (a.N + 127) / 128 * 8;
  const int ctas = groups / RG;
  const int n_steps = (a.K + kStep - 1) / kStep;
  // split the columns over a cluster while that leaves every CTA two steps a warp and
  // the grid within two CTAs an SM
  int cs = 1;
  while (cs < kMaxCluster && ctas * cs * 2 <= 2 * sm_count && n_steps >= KW * cs * 4) cs *= 2;
  return launch_pdl_cluster(gemv_kernel<KW, NT, FP32>, dim3(unsigned(ctas * cs)),
                            dim3(unsigned(cs)), dim3(kThreads), 0, st, a);
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
  // KW M <= 16 row-steps are converted at a time; 8 NT >= product columns
  if (g.x_dtype == NVFP4_BF16) {
    if (g.M <= 2) return gemv::launch<8, 1, false>(a, g.sm_count, st);
    if (g.M <= 4) return gemv::launch<4, 1, false>(a, g.sm_count, st);
    if (g.M <= 8) return gemv::launch<2, 1, false>(a, g.sm_count, st);
    return gemv::launch<1, 2, false>(a, g.sm_count, st);
  }
  if (g.M <= 2) return gemv::launch<8, 1, true>(a, g.sm_count, st);
  if (g.M <= 4) return gemv::launch<4, 1, true>(a, g.sm_count, st);
  if (g.M <= 8) return gemv::launch<2, 2, true>(a, g.sm_count, st);
  return gemv::launch<1, 4, true>(a, g.sm_count, st);
}

}  // namespace nvfp4
