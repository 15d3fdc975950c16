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
// and the tables.  No CTA waits for another.  One request 2.3 us, 512 requests with 66
// thousand new tokens 4.2 us: the launch, three loads in a row and the sums' barriers.
__global__ void __launch_bounds__(kThreads) plan_kernel(const Args a) {
  extern __shared__ int32_t smem[];
  int32_t* cu = smem;                   // [batch + 1] tokens before each request
  int32_t* first = smem + a.batch + 1;  // [batch] pages taken before each request
  __shared__ unsigned long long warp_sum[kWarps];
  __shared__ unsigned long long totals[2];
  __shared__ int32_t bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int step = gridDim.x * kThreads, g = blockIdx.x * kThreads + tid;
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
    for (int i = g; i < a.batch; i += step) a.seq_lens[i] = a.cached[i];
    for (int i = g; i <= a.batch; i += step) a.cu_new[i] = 0;
    for (uint32_t i = g; i < uint32_t(a.max_new); i += step) a.slot_map[i] = -1;
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
  // slots: the request by bisection of cu, its page from the free list or the table (unsigned: the
  // last t + step may be past 2^31)
  for (uint32_t i = g; i < uint32_t(a.max_new); i += step) {
    const int t = int(i);
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
    a.slot_map[i] = slot;
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
constexpr int kOld = 4;   // 16-byte loads of a thread in flight while it codes old tokens again
constexpr int kMaxCluster = 8;
constexpr int kResident = 5;  // CTAs of an SM: six (80 registers) spill

struct Args {
  const uint16_t* x[2];    // K, V: bf16, token t, head h at t * stride + h * dim
  int64_t stride;
  uint8_t* codes[2];       // [page][head][token][dim]
  float* scale[2];         // [page][head]
  const int32_t* slots;    // [tokens]
  int32_t tokens, heads, page_tokens, per_tile;
  int32_t parts, per_part;  // of a tile's 2 * heads heads of K and V
  int64_t n_slots;         // n_pages * page_tokens
  FastDiv page_div, part_div;
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

// The larger of m and the magnitudes of 8 bf16 values, as bf16 bits, in each half.
__device__ __forceinline__ uint32_t amax8(uint4 v, uint32_t m) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(m, __vmaxu2(v.x & kAbs, v.y & kAbs)),
                  __vmaxu2(v.z & kAbs, v.w & kAbs));
}

// 8 bf16 values with the non-finite ones zero.
__device__ __forceinline__ uint4 finite8(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
    if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 bf16 values with the NaN zero.
__device__ __forceinline__ uint4 no_nan8(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFF0000u;
    if ((w[i] & 0x7FFFFFFFu) > 0x7F80FFFFu) w[i] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 bf16 values (none a NaN) times inv, a power of two twice in bf16 -> 8 E4M3 bytes
// (nearest even, saturating).  The product is exact, or so small (bf16 subnormal) that its
// code is zero either way: one rounding.
__device__ __forceinline__ uint2 encode8(uint4 v, uint32_t inv) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(inv));
    h[i] = e4m3x2(__uint_as_float(w[i] & 0xFFFF0000u), __uint_as_float(w[i] << 16));
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

// n times 16 old codes, by `set` threads of which this is `id`.  Not inlined: the loads in
// flight would cost the caller the registers of its rows.
__device__ __noinline__ void recode(uint4* old, int n, float ratio, int id, int set) {
  for (int i = id; i < n; i += kOld * set) {
    uint4 q[kOld];
#pragma unroll
    for (int j = 0; j < kOld; ++j) q[j] = old[min(i + j * set, n - 1)];
#pragma unroll
    for (int j = 0; j < kOld; ++j)
      if (i + j * set < n)
        old[i + j * set] = make_uint4(recode4(q[j].x, ratio), recode4(q[j].y, ratio),
                                      recode4(q[j].z, ratio), recode4(q[j].w, ratio));
  }
}

// Largest value over the CTA.  The callers alternate between two buffers: one barrier.
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* buf) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return max(max(buf[0], buf[1]), max(buf[2], buf[3]));
}

// Largest value over a cluster of n CTAs; buf is this CTA's, 4 words for each rank.
__device__ __forceinline__ uint32_t cluster_max(uint32_t v, uint32_t* buf, uint32_t rank, int n) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  const int lane = threadIdx.x & 31;
  if (lane < n) store_cluster(buf + 4 * rank + (threadIdx.x >> 5), lane, v);
  cluster_arrive();
  cluster_wait();
  return __reduce_max_sync(0xFFFFFFFFu, lane < 4 * n ? buf[lane] : 0);
}

// A run is a row of tokens whose slots follow one another inside a page; the scale of a
// page is set by whoever has its run, from all of the run's tokens.  A tile of per_tile
// tokens belongs to one CTA, or where pages are longer than a CTA holds in registers
// (kHeld rows a thread) to a cluster, for per_part of the heads of K and V: it takes the
// runs that begin in the tile, one head after another.  A run that a warp holds is a
// warp's, the warps taking turns; one that a CTA holds a CTA's; a longer one is divided
// among the cluster, and its largest value found over distributed shared memory.
//
// HBM-bound when there are many tokens (2 bytes read and 1 written per element).  A chunk
// of slots is read at once and gives the beginnings and lengths of all its runs, for all
// heads of the part, so that each head's rows are one load latency and are read once.
//
// 18 thousand tokens of 8 heads of 128 in 64-token pages (113 MB): 26 us, 66% of the copy rate
// (one head a CTA 30 us: the latency of the slots in front of every 16 KB; 16-token pages of
// 64 elements 21 us).  512 single tokens 11 us, 33 of them 3.1 us: two load latencies and
// the launch.  Pages of 880 tokens 69 us, 115 without the clusters.
template <int kDim>
__global__ void __launch_bounds__(kThreads, kResident) append_kernel(const Args a) {
  constexpr int kLanes = kDim / 8;  // threads of a token row
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps == 4, "cta_max and cluster_max");
  __shared__ uint32_t begins[kWarps], stops[kWarps], shorts[kWarps];
  __shared__ int32_t slot_of[kThreads], len_of[kThreads];
  __shared__ uint32_t own_buf[2][kWarps], all_buf[2][kWarps * kMaxCluster];
  const int tid = threadIdx.x, u = tid % kLanes;
  const int page_tokens = a.page_tokens;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  // the parts of a tile next to one another: CTAs that run together read whole rows of x
  const uint32_t cta = blockIdx.x / ranks, tile = fast_div(a.part_div, cta);
  const int item0 = int(cta - tile * uint32_t(a.parts)) * a.per_part;
  const int item_end = min(item0 + a.per_part, 2 * a.heads);
  if (ranks > 1) cluster_arrive();  // waited for before the first store to another CTA
  bool started = ranks == 1;
  pdl_wait();
  pdl_trigger();
  const int t0 = int(tile) * a.per_tile;
  const int t_end = min(a.tokens, t0 + a.per_tile);
  bool nonfinite = false;
  uint32_t warp_turn = 0, cta_turn = 0, own_uses = 0, all_uses = 0;

  // the run of len tokens from token t at slot s, by `set` threads (a warp, a CTA or the
  // cluster) of which this is `id`
  auto take = [&](int t, int s, int len, int id, int set) {
    const int page = int(fast_div(a.page_div, uint32_t(s)));
    const int off = s - page * page_tokens;
    const int r0 = id / kLanes, step = set / kLanes;
    for (int item = item0; item < item_end; ++item) {
      const bool is_v = item >= a.heads;
      const int h = is_v ? item - a.heads : item;
      const uint16_t* src = (is_v ? a.x[1] : a.x[0]) + int64_t(t) * a.stride + h * kDim + 8 * u;
      const int64_t ph = int64_t(page) * a.heads + h;
      uint8_t* dst = (is_v ? a.codes[1] : a.codes[0]) + ph * page_tokens * kDim;
      float* scale = (is_v ? a.scale[1] : a.scale[0]) + ph;
      const float was = off > 0 ? *scale : 0.0f;
      uint4 v[kHeld];
      const uint16_t* in = src + r0 * a.stride;
#pragma unroll
      for (int j = 0; j < kHeld; ++j, in += step * a.stride)
        v[j] = r0 + j * step < len ? ld_nc_v4(in) : make_uint4(0, 0, 0, 0);
      uint32_t tops = 0;  // even and odd elements
#pragma unroll
      for (int j = 0; j < kHeld; ++j) tops = amax8(v[j], tops);
      for (int i = r0 + kHeld * step; i < len; i += step, in += step * a.stride)
        tops = amax8(ld_nc_v4_l1(in), tops);
      uint32_t top = max(tops & 0xFFFFu, tops >> 16);
      const bool odd = top >= 0x7F80u;  // the thread's part has infinities or NaN
      if (odd) {
        nonfinite = true;
        tops = 0;
        for (int i = r0; i < len; i += step)
          tops = amax8(finite8(ld_nc_v4_l1(src + i * a.stride)), tops);
        top = max(tops & 0xFFFFu, tops >> 16);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) v[j] = no_nan8(v[j]);
      }
      if (set == 32) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
      } else if (set == kThreads) {
        top = cta_max(top, own_buf[own_uses++ & 1]);
      } else {
        if (!started) cluster_wait();
        started = true;
        top = cluster_max(top, all_buf[all_uses++ & 1], rank, int(ranks));
      }
      const float now = fmaxf(was, pow2(fit_exponent(top)));
      const uint32_t inv = 0x7F00u - (__float_as_uint(now) >> 16);  // 1 / now in bf16
      const uint32_t inv2 = inv | (inv << 16);
      uint8_t* const to = dst + (off + r0) * kDim + 8 * u;
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const uint2 c = encode8(v[j], inv2);
        if (r0 + j * step < len) *reinterpret_cast<uint2*>(to + j * step * kDim) = c;
      }
      for (int i = r0 + kHeld * step; i < len; i += step) {
        uint4 x8 = ld_nc_v4_l1(src + i * a.stride);
        if (odd) x8 = no_nan8(x8);
        *reinterpret_cast<uint2*>(dst + (off + i) * kDim + 8 * u) = encode8(x8, inv2);
      }
      if (off > 0 && now > was) {
        const float ratio = was * __uint_as_float(inv << 16);
        recode(reinterpret_cast<uint4*>(dst), off * kDim / 16, ratio, id, set);
      }
      if (id == 0) *scale = now;
    }
  };

  for (int base = t0; base < t_end; base += kThreads) {
    if (base != t0) __syncthreads();
    const int mine = base + tid;
    bool begin = false, stop = true;  // of a run; not the continuation of one
    int most = 0;                     // tokens of a run that begins here, by page and tokens
    if (mine < a.tokens) {
      const int32_t s = a.slots[mine], before = mine > 0 ? a.slots[mine - 1] : -1;
      slot_of[tid] = s;
      if (s >= 0 && s < a.n_slots) {
        const int off = s - int(fast_div(a.page_div, uint32_t(s))) * page_tokens;
        stop = off == 0 || before != s - 1;
        begin = stop && mine < t_end;
        most = min(page_tokens - off, a.tokens - mine);
      } else if (s != -1 && mine < t_end) {
        record_status(a.status, NVFP4_ERR_INVALID_ARG);
      }
    }
    const uint32_t bw = __ballot_sync(0xFFFFFFFFu, begin), sw = __ballot_sync(0xFFFFFFFFu, stop);
    if ((tid & 31) == 0) {
      begins[tid >> 5] = bw;
      stops[tid >> 5] = sw;
    }
    __syncthreads();
    int len = kThreads - tid;  // to the next stop, or to the chunk's end and maybe on (open)
    bool open = true;
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      const uint32_t later = w < (tid >> 5)   ? 0
                             : w > (tid >> 5) ? stops[w]
                                              : stops[w] & (0xFFFFFFFEu << (tid & 31));
      if (later) {
        len = 32 * w + __ffs(later) - 1 - tid;
        open = false;
      }
    }
    open = open && len < most;
    len_of[tid] = open ? -len : len;
    const uint32_t few = __ballot_sync(0xFFFFFFFFu, begin && !open && len <= kHeld * 32 / kLanes);
    if ((tid & 31) == 0) shorts[tid >> 5] = few;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      for (uint32_t bits = begins[w] & ~shorts[w]; bits != 0; bits &= bits - 1) {
        const int at = 32 * w + __ffs(bits) - 1, t = base + at, s = slot_of[at];
        int n = len_of[at];
        if (n < 0) {
          // most - the place of the break behind the chunk, the largest the first
          const int off = s - int(fast_div(a.page_div, uint32_t(s))) * page_tokens;
          const int limit = min(page_tokens - off, a.tokens - t);
          uint32_t left = 0;
          for (int i = tid - n; i < limit && left == 0; i += kThreads)
            if (a.slots[t + i] != s + i) left = uint32_t(limit - i);
          n = limit - int(cta_max(left, own_buf[own_uses++ & 1]));
        }
        if (n <= kHeld * kThreads / kLanes || ranks == 1) {
          if ((cta_turn++ & (ranks - 1)) == rank) take(t, s, n, tid, kThreads);
        } else {
          take(t, s, n, int(rank) * kThreads + tid, kThreads * int(ranks));
        }
      }
    }
    const uint32_t warp = rank * kWarps + (tid >> 5);
    for (int w = 0; w < kWarps; ++w)
      for (uint32_t bits = shorts[w]; bits != 0; bits &= bits - 1)
        if ((warp_turn++ & (kWarps * ranks - 1)) == warp) {
          const int at = 32 * w + __ffs(bits) - 1;
          take(base + at, slot_of[at], len_of[at], tid & 31, 32);
        }
  }
  if (!started) cluster_wait();
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
  // as many CTAs as hold a page's rows in registers, if there are that many tokens
  const int64_t held = append::kHeld * append::kThreads / (p.head_dim / 8);
  const int64_t longest = p.tokens < p.page_tokens ? p.tokens : p.page_tokens;
  int64_t ranks = 1;
  while (ranks < append::kMaxCluster && ranks * held < longest) ranks *= 2;
  // About 8 CTAs an SM.  Few tokens: short tiles, as every token may be a run of its own;
  // many: as long as a page or four warps' runs, so that few tiles have no beginning.
  const int64_t ctas = int64_t(p.sm_count) * 8;
  const int64_t widest = p.page_tokens > 64 ? p.page_tokens : 64;
  int64_t per = p.tokens * p.heads * 2 * ranks / ctas;
  per = per < 1 ? 1 : per > widest ? widest : per;
  a.per_tile = int32_t(per);
  // ... and then several heads a CTA, for which the slots are looked at once
  const int64_t tiles = (p.tokens + per - 1) / per;
  int64_t part = tiles * p.heads * 2 * ranks / ctas;
  part = part < 1 ? 1 : part > 2 * p.heads ? 2 * p.heads : part;
  a.per_part = int32_t(part);
  a.parts = int32_t((2 * p.heads + part - 1) / part);
  a.part_div = make_fastdiv(uint32_t(a.parts));
  const dim3 grid(unsigned(tiles * a.parts * ranks));
  const dim3 cluster(static_cast<unsigned>(ranks), 1, 1), block(append::kThreads);
  if (ranks == 1)
    return p.head_dim == 64
               ? launch_pdl(append::append_kernel<64>, grid, block, 0, st, a)
               : launch_pdl(append::append_kernel<128>, grid, block, 0, st, a);
  return p.head_dim == 64
             ? launch_pdl_cluster(append::append_kernel<64>, grid, cluster, block, 0, st, a)
             : launch_pdl_cluster(append::append_kernel<128>, grid, cluster, block, 0, st, a);
}

}  // namespace nvfp4
