// kv8.cu -- the paged 8-bit KV cache: page plans from request lengths, and the
// quantizing write of new tokens.
//
// Page: page_tokens consecutive tokens of one request; codes of one (page, head)
// are contiguous, [page][head][token][dim] E4M3 bytes, with one scale for each
// page and head.  Scales are powers of two: an E4M3 value keeps its 4-bit
// significand under them, so nothing is lost against a scale of any other form,
// and a page whose scale has to grow recodes its older tokens exactly except
// where they become subnormal.
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

// ---------------------------------------------------------------- plan
namespace plan {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct Args {
  const int32_t *cached, *fresh;  // [batch]
  int32_t* table;                 // [batch][table_stride]
  int64_t table_stride;
  const int32_t* free_pages;      // [n_free]
  const int32_t* free_head;       // [1]
  int32_t *seq_lens, *cu_new, *slot_map, *free_head_out;
  int32_t batch, max_pages, n_free, n_pages, page_tokens, max_new;
  FastDiv page_div;
  uint32_t* status;
};

// Pages that n tokens fill, the last one perhaps in part.
__device__ __forceinline__ int32_t pages_of(const Args& a, uint32_t n) {
  return int32_t(fast_div(a.page_div, n + uint32_t(a.page_tokens) - 1));
}

// Latency is all of it (a few hundred KB at most), so it is one launch: every CTA
// computes the two prefix sums over the requests for itself (they are read from
// L2; one request a thread up to 512) and then fills its share of the slot map
// and the tables.  No CTA waits for another.
__global__ void __launch_bounds__(kThreads) plan_kernel(const Args a) {
  extern __shared__ int32_t smem[];
  int32_t* cu = smem;                   // [batch + 1] tokens before each request
  int32_t* first = smem + a.batch + 1;  // [batch] pages taken before each request
  __shared__ unsigned long long warp_sum[kWarps];
  __shared__ unsigned long long totals[2];
  __shared__ int32_t bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bad = 0, totals[0] = 0, totals[1] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();

  // totals in 64 bits, and the checks that let the sums below be 32-bit
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  const int64_t room = int64_t(a.max_pages) * a.page_tokens;
  unsigned long long need = 0, tokens = 0;
  bool over = false, negative = false;
  for (int b = b0; b < b1; ++b) {
    const int64_t c = a.cached[b], t = a.fresh[b];
    if (c < 0 || t < 0) {
      negative = true;
    } else if (c + t > room) {
      over = true;
    } else {
      need += unsigned(pages_of(a, uint32_t(c + t)) - pages_of(a, uint32_t(c)));
      tokens += uint64_t(t);
    }
  }
  const int32_t head = *a.free_head;
  if (head < 0 || head > a.n_free) negative = true;
  unsigned long long rn = need, rt = tokens;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    rn += __shfl_xor_sync(0xFFFFFFFFu, rn, o);
    rt += __shfl_xor_sync(0xFFFFFFFFu, rt, o);
  }
  if (lane == 0) {
    if (rn) atomicAdd(&totals[0], rn);
    if (rt) atomicAdd(&totals[1], rt);
  }
  if (negative) atomicOr(&bad, 1);
  if (over) atomicOr(&bad, 2);
  // exclusive prefix sums, pages in the high word, tokens in the low one (wrong where
  // a sum does not fit, and then not used)
  unsigned long long mine = (need << 32) + (tokens & 0xFFFFFFFFull), inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long before = inc - mine;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  const unsigned long long all_pages = totals[0], all_tokens = totals[1];
  const int fault = bad;
  const bool full = all_tokens > uint64_t(a.max_new) ||
                    (fault == 0 && all_pages > uint64_t(a.n_free - head));
  if (fault != 0 || full) {
    // all or nothing: no page is taken, no slot is given
    if (blockIdx.x == 0 && tid == 0) {
      record_status(a.status, (fault & 1) ? NVFP4_ERR_INVALID_ARG : NVFP4_ERR_CAPACITY);
      *a.free_head_out = head;
    }
    const int step = gridDim.x * kThreads, g = blockIdx.x * kThreads + tid;
    for (int i = g; i < a.batch; i += step) a.seq_lens[i] = a.cached[i];
    for (int i = g; i <= a.batch; i += step) a.cu_new[i] = 0;
    for (int i = g; i < a.max_new; i += step) a.slot_map[i] = -1;
    return;
  }
  for (int b = b0; b < b1; ++b) {
    const uint32_t c = uint32_t(a.cached[b]), t = uint32_t(a.fresh[b]);
    cu[b] = int32_t(before & 0xFFFFFFFFull);
    first[b] = head + int32_t(before >> 32);
    before += (static_cast<unsigned long long>(pages_of(a, c + t) - pages_of(a, c)) << 32) + t;
  }
  if (tid == 0) cu[a.batch] = int32_t(all_tokens);
  __syncthreads();

  // lengths and offsets
  const int step = gridDim.x * kThreads, g = blockIdx.x * kThreads + tid;
  for (int i = g; i <= a.batch; i += step) {
    a.cu_new[i] = cu[i];
    if (i < a.batch) a.seq_lens[i] = a.cached[i] + a.fresh[i];
  }
  if (g == 0) *a.free_head_out = head + int32_t(all_pages);
  // new table entries, a warp for each request in turn
  for (int b = blockIdx.x * kWarps + warp; b < a.batch; b += gridDim.x * kWarps) {
    const uint32_t c = uint32_t(a.cached[b]);
    const int held = pages_of(a, c), total = pages_of(a, c + uint32_t(a.fresh[b]));
    for (int i = held + lane; i < total; i += 32)
      a.table[b * a.table_stride + i] = a.free_pages[first[b] + i - held];
  }
  // slots: the request by bisection of cu, its page from the free list or the table
  for (int t = g; t < a.max_new; t += step) {
    int32_t slot = -1;
    if (t < int(all_tokens)) {
      int lo = 0, hi = a.batch;  // the last b with cu[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid;
      }
      const uint32_t c = uint32_t(a.cached[lo]), pos = c + uint32_t(t - cu[lo]);
      const int held = pages_of(a, c), idx = int(fast_div(a.page_div, pos));
      const int32_t id = idx < held ? a.table[lo * a.table_stride + idx]
                                    : a.free_pages[first[lo] + idx - held];
      if (id >= 0 && id < a.n_pages)
        slot = id * a.page_tokens + int32_t(pos - uint32_t(idx) * uint32_t(a.page_tokens));
      else
        record_status(a.status, NVFP4_ERR_INVALID_ARG);
    }
    a.slot_map[t] = slot;
  }
}

}  // namespace plan

cudaError_t launch_plan(const LaunchPlan& p, cudaStream_t st) {
  plan::Args a;
  a.cached = p.cached;
  a.fresh = p.fresh;
  a.table = p.table;
  a.table_stride = p.table_stride;
  a.free_pages = p.free_pages;
  a.free_head = p.free_head;
  a.seq_lens = p.seq_lens;
  a.cu_new = p.cu_new;
  a.slot_map = p.slot_map;
  a.free_head_out = p.free_head_out;
  a.batch = p.batch;
  a.max_pages = p.max_pages;
  a.n_free = p.n_free;
  a.n_pages = p.n_pages;
  a.page_tokens = p.page_tokens;
  a.max_new = p.max_new;
  a.page_div = make_fastdiv(uint32_t(p.page_tokens));
  a.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.ws) + kWsStatus);
  const size_t smem = (2 * size_t(p.batch) + 1) * sizeof(int32_t);
  const cudaError_t e = allow_smem<plan::plan_kernel>(
      (2 * size_t(NVFP4_PLAN_MAX_BATCH) + 1) * sizeof(int32_t));
  if (e != cudaSuccess) return e;
  const int64_t work = p.max_new > p.batch ? p.max_new : p.batch;
  int64_t ctas = (work + plan::kThreads - 1) / plan::kThreads;
  if (ctas > p.sm_count) ctas = p.sm_count;
  return launch_pdl(plan::plan_kernel, dim3(unsigned(ctas < 1 ? 1 : ctas)), dim3(plan::kThreads),
                    smem, st, a);
}

// ---------------------------------------------------------------- append
namespace append {

constexpr int kThreads = 128;
constexpr int kHeld = 8;  // rows of a thread kept in registers between the two passes

struct Args {
  const uint16_t* x[2];    // K, V: bf16, token t, head h at t * stride + h * dim
  int64_t stride;
  uint8_t* codes[2];       // [page][head][token][dim]
  float* scale[2];         // [page][head]
  const int32_t* slots;    // [tokens]
  int32_t tokens, heads, page_tokens, per_cta;
  int64_t n_slots;         // n_pages * page_tokens
  FastDiv page_div;
  uint32_t* status;
};

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// The smallest e in [-60, 60] with amax <= 448 2^e, from amax's bf16 bits:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int fit_exponent(uint32_t bits) {
  const int e = int(bits >> 7) - 127 - 8 + ((bits & 0x7F) > 0x60 ? 1 : 0);
  return max(NVFP4_KV8_MIN_EXP, min(NVFP4_KV8_MAX_EXP, e));
}

// Largest magnitude of 8 bf16 values as bf16 bits, non-finite ones left out.
__device__ __forceinline__ uint32_t amax8(uint4 v, bool& nonfinite) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                        __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= 0x7F80u) {
    nonfinite = true;
    m = 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
      if (b < 0x7F80u) m = max(m, b);
    }
  }
  return m;
}

// 8 bf16 values times inv -> 8 E4M3 bytes (nearest even, saturating; NaN -> 0).
__device__ __forceinline__ uint2 encode8(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo = __uint_as_float(w[i] << 16) * inv, hi = __uint_as_float(w[i] & 0xFFFF0000u) * inv;
    lo = lo == lo ? lo : 0.0f;
    hi = hi == hi ? hi : 0.0f;
    h[i] = e4m3x2(hi, lo);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Four E4M3 bytes times a power of two <= 1, rounded again.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    h[i] = e4m3x2(e4m3_to_f32(w >> (16 * i + 8)) * ratio, e4m3_to_f32(w >> (16 * i)) * ratio);
  return h[0] | (h[1] << 16);
}

// Largest value over the CTA.
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* buf) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return max(max(buf[0], buf[1]), max(buf[2], buf[3]));
}

// One CTA takes the runs (tokens in a row whose slots follow one another inside a
// page) that begin among its per_cta tokens, for one head and one of K and V: the
// scale of a page is set by one CTA, which sees all of the page's new tokens.
// HBM-bound when there are many tokens (4 bytes read and 2 written for each K and
// V element pair): a run is read once, up to kHeld rows a thread in registers.
template <int kDim>
__global__ void __launch_bounds__(kThreads) append_kernel(const Args a) {
  constexpr int kLanes = kDim / 8;              // threads of a token row
  constexpr int kRows = kThreads / kLanes;      // token rows of a pass
  __shared__ uint32_t buf[kThreads / 32];
  const int tid = threadIdx.x, u = tid % kLanes, row = tid / kLanes;
  const int h = blockIdx.y, plane = blockIdx.z;
  const int page_tokens = a.page_tokens;
  pdl_wait();
  pdl_trigger();
  const uint16_t* x = a.x[plane] + int64_t(h) * kDim + 8 * u;
  const int t_end = min(a.tokens, (int(blockIdx.x) + 1) * a.per_cta);
  bool nonfinite = false;
  for (int t = int(blockIdx.x) * a.per_cta; t < t_end;) {
    const int64_t s = a.slots[t];
    if (s < 0 || s >= a.n_slots) {
      if (s != -1 && tid == 0) record_status(a.status, NVFP4_ERR_INVALID_ARG);
      ++t;
      continue;
    }
    const int page = int(fast_div(a.page_div, uint32_t(s)));
    const int off = int(s) - page * page_tokens;
    // length of the run: the first place where the slots do not go on
    const int most = min(page_tokens - off, a.tokens - t);
    uint32_t stop = 0;  // most - index of the break, so that the largest is the first
    for (int i = 1 + tid; i < most && stop == 0; i += kThreads)
      if (a.slots[t + i] != int(s) + i) stop = uint32_t(most - i);
    const int len = most > 1 ? most - int(cta_max(stop, buf)) : 1;
    if (off > 0 && t > 0 && t == int(blockIdx.x) * a.per_cta && a.slots[t - 1] == int(s) - 1) {
      t += len;  // the rest of a run that the previous CTA has
      continue;
    }
    const uint16_t* src = x + int64_t(t) * a.stride;
    const int64_t ph = int64_t(page) * a.heads + h;
    uint8_t* dst = a.codes[plane] + ph * page_tokens * kDim;
    float* scale = a.scale[plane] + ph;
    const float was = off > 0 ? *scale : 0.0f;
    uint4 v[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = row + j * kRows;
      v[j] = i < len ? ld_nc_v4(src + i * a.stride) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) top = max(top, amax8(v[j], nonfinite));
    for (int i = row + kHeld * kRows; i < len; i += kRows)
      top = max(top, amax8(ld_nc_v4_l1(src + i * a.stride), nonfinite));
    const float fit = pow2(fit_exponent(cta_max(top, buf)));
    const float now = fmaxf(was, fit);
    const float inv = 1.0f / now;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = row + j * kRows;
      if (i < len) *reinterpret_cast<uint2*>(dst + (off + i) * kDim + 8 * u) = encode8(v[j], inv);
    }
    for (int i = row + kHeld * kRows; i < len; i += kRows)
      *reinterpret_cast<uint2*>(dst + (off + i) * kDim + 8 * u) =
          encode8(ld_nc_v4_l1(src + i * a.stride), inv);
    if (off > 0 && now > was) {
      const float ratio = was * inv;
      for (int i = tid; i < off * kDim / 16; i += kThreads) {
        uint4 w = reinterpret_cast<uint4*>(dst)[i];
        w.x = recode4(w.x, ratio);
        w.y = recode4(w.y, ratio);
        w.z = recode4(w.z, ratio);
        w.w = recode4(w.w, ratio);
        reinterpret_cast<uint4*>(dst)[i] = w;
      }
    }
    if (tid == 0) *scale = now;
    t += len;
  }
  if (nonfinite) record_status(a.status, NVFP4_ERR_DOMAIN);
}

}  // namespace append

cudaError_t launch_kv8_append(const LaunchKv8Append& p, cudaStream_t st) {
  append::Args a;
  a.x[0] = static_cast<const uint16_t*>(p.k);
  a.x[1] = static_cast<const uint16_t*>(p.v);
  a.stride = p.token_stride;
  a.codes[0] = p.k_codes;
  a.codes[1] = p.v_codes;
  a.scale[0] = p.k_scale;
  a.scale[1] = p.v_scale;
  a.slots = p.slot_map;
  a.tokens = int32_t(p.tokens);
  a.heads = p.heads;
  a.page_tokens = p.page_tokens;
  a.n_slots = int64_t(p.n_pages) * p.page_tokens;
  a.page_div = make_fastdiv(uint32_t(p.page_tokens));
  a.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.ws) + kWsStatus);
  // few tokens: one a CTA (each may be a run of its own); many: up to a page's worth, so
  // that CTAs without a run's beginning stay few
  int64_t per = p.tokens * p.heads * 2 / (int64_t(p.sm_count) * 16);
  per = per < 1 ? 1 : per > p.page_tokens ? p.page_tokens : per;
  a.per_cta = int32_t(per);
  const dim3 grid(unsigned((p.tokens + per - 1) / per), unsigned(p.heads), 2);
  return p.head_dim == 64
             ? launch_pdl(append::append_kernel<64>, grid, dim3(append::kThreads), 0, st, a)
             : launch_pdl(append::append_kernel<128>, grid, dim3(append::kThreads), 0, st, a);
}

}  // namespace nvfp4
