// kv8_batch.cuh -- what the attention kernels over the paged 8-bit cache share:
// their arguments, the requests of a batch, which tokens a row sees, and where a
// row's result goes.
//
// Rows: the query heads of one KV head and the queries of a request are packed, row
// rho = query * group + (head of the group).
#pragma once
#include "common.cuh"

namespace nvfp4 {
namespace kv8 {

struct Args {
  const uint16_t* q;       // bf16, token t, head h at t * q_stride + h * dim
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  float* lse;              // [tq][q_heads] natural log-sum-exp, or NULL
  const int32_t* cu_q;     // [batch + 1]
  const int32_t* kv_lens;  // [batch]
  const int32_t* table;    // [batch][table_stride]
  int64_t table_stride;
  const uint8_t *k_codes, *v_codes;  // [page][kv head][token][dim]
  const float *k_scale, *v_scale;    // [page][kv head]
  int32_t tq, q_heads, kv_heads, group, max_q, max_tokens, n_pages, page_tokens, causal;
  FastDiv group_div, page_div;
  float scale_log2;        // softmax scale * log2(e)
  int32_t chunk, n_splits; // tokens of a range, most ranges
  int32_t cluster;         // the ranges of a unit are a cluster, which joins them itself
  float* part_o;           // [n_splits][tq][q_heads][dim]
  float* part_lse;         // [n_splits][tq][q_heads], base 2
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct Request {
  int32_t q0, nq, kv;  // first query, queries, cached tokens
};

// Request b, held inside the buffers whatever the device arrays say (a length or an
// offset outside them is recorded by the thread that has `record` set).
__device__ __forceinline__ Request request(const Args& a, int b, bool record) {
  const int32_t lo = __ldg(a.cu_q + b), hi = __ldg(a.cu_q + b + 1), kv = __ldg(a.kv_lens + b);
  Request r;
  r.q0 = max(0, min(lo, a.tq));
  r.nq = max(0, min(max(0, min(hi, a.tq)) - r.q0, a.max_q));
  r.kv = max(0, min(kv, a.max_tokens));
  if (record && (r.q0 != lo || int64_t(lo) + r.nq != hi || r.kv != kv))
    record_status(a.status, NVFP4_ERR_INVALID_ARG);
  return r;
}

// Tokens that row rho sees: all, or (causal) those up to its own place, the queries
// being the request's last tokens.
__device__ __forceinline__ int sees(const Args& a, const Request& r, int rho) {
  if (!a.causal) return r.kv;
  return max(0, r.kv - r.nq + 1 + int(fast_div(a.group_div, uint32_t(rho))));
}

// Ranges of a request of kv tokens (at least one; the last takes what is left).
__device__ __forceinline__ int splits_of(const Args& a, int kv) {
  return max(1, min(a.n_splits, int((uint32_t(kv) + a.chunk - 1) / uint32_t(a.chunk))));
}

__device__ __forceinline__ const uint16_t* q_row(const Args& a, const Request& r, int h, int rho,
                                                 int dim) {
  const int i = int(fast_div(a.group_div, uint32_t(rho))), g = rho - i * a.group;
  return a.q + int64_t(r.q0 + i) * a.q_stride + int64_t(h * a.group + g) * dim;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Stores kPer consecutive dims from d0 on of a finished row: to the output where the
// request has one range, else to the range's partial result.
template <int kPer, int kDim>
__device__ __forceinline__ void store_row(const Args& a, const Request& r, int h, int rho,
                                          int split, int used, int d0, const float (&v)[kPer],
                                          float lse2, bool first) {
  const int i = int(fast_div(a.group_div, uint32_t(rho))), g = rho - i * a.group;
  const int64_t tok = r.q0 + i, row = tok * a.q_heads + h * a.group + g;
  if (used == 1) {
    uint16_t* dst = a.out + tok * a.out_stride + int64_t(h * a.group + g) * kDim + d0;
#pragma unroll
    for (int j = 0; j < kPer; j += 4)
      *reinterpret_cast<uint2*>(dst + j) =
          make_uint2(bf16x2(v[j], v[j + 1]), bf16x2(v[j + 2], v[j + 3]));
    if (a.lse && first) a.lse[row] = lse2 * 0.6931471805599453f;
  } else {
    const int64_t at = int64_t(split) * a.tq * a.q_heads + row;
    float* dst = a.part_o + at * kDim + d0;
#pragma unroll
    for (int j = 0; j < kPer; j += 4)
      *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    if (first) a.part_lse[at] = lse2;
  }
}

}  // namespace kv8

cudaError_t launch_kv8_chunk(const kv8::Args& a, int32_t head_dim, int32_t row_tiles, int32_t batch,
                             cudaStream_t st);

}  // namespace nvfp4
