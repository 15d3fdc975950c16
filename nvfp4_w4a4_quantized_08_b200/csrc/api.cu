// api.cu -- the C ABI of libnvfp4 (declared in include/nvfp4.h): host-side
// argument checks, then one or two kernel launches on the caller's stream.
#include <cmath>
#include <atomic>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

using namespace nvfp4;

namespace {

std::atomic<uint64_t> g_wait_limit_ns{2000000000ull};

struct DeviceInfo {
  bool ok;
  int sm_count;
};

// Compute capability and SM count of the current device, cached per device.
// Host threads may call in concurrently: an entry is published through its
// atomic word (0 = not yet queried, else 1 + sm_count, negated when the
// device is not sm_100), so a reader sees either nothing or a whole entry.
DeviceInfo current_device() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return {false, 0};
  int word = cache[dev].load(std::memory_order_acquire);
  if (word == 0) {
    int major = 0, minor = 0, sms = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    word = (major == 10 && minor == 0) ? 1 + sms : -(1 + sms);
    cache[dev].store(word, std::memory_order_release);
  }
  return {word > 0, (word > 0 ? word : -word) - 1};
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// n rows of `width` bytes, `stride` bytes apart (at least width).
struct Rows {
  const void* p;
  int64_t n, width, stride;
};
Rows block(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }

// Whether two sets of rows share a byte.  Rows of one stride may lie beside each other (parts of a
// fused projection); where the strides differ, sets whose spans meet count as sharing.
bool overlap(Rows a, Rows b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0 || a.width <= 0 || b.width <= 0) return false;
  const int64_t a0 = int64_t(reinterpret_cast<uintptr_t>(a.p));
  const int64_t b0 = int64_t(reinterpret_cast<uintptr_t>(b.p));
  if (a0 + (a.n - 1) * a.stride + a.width <= b0 || b0 + (b.n - 1) * b.stride + b.width <= a0)
    return false;
  if (a.n == 1) a.stride = b.stride;
  if (b.n == 1) b.stride = a.stride;
  const int64_t s = a.stride;
  if (b.stride != s || a.width > s || b.width > s) return true;
  // row j of b begins in row j + r of a, `at` bytes behind its start, and may run into the next
  const int64_t d = b0 - a0, at = (d % s + s) % s, r = (d - at) / s;
  auto meet = [&](int64_t shift) { return shift < a.n && shift + b.n > 0; };
  return (at < a.width && meet(r)) || (at + b.width > s && meet(r + 1));
}

nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

bool valid_layout(int32_t l) { return l == NVFP4_SF_ROWMAJOR || l == NVFP4_SF_MMA128x4; }

// Checks shared by every NVFP4 tensor argument.
nvfp4_status check_tensor(const nvfp4_tensor* t) {
  if (!t || !t->codes || !t->sf || !t->s_t) return NVFP4_ERR_INVALID_ARG;
  if (t->rows <= 0 || t->cols <= 0 || !valid_layout(t->sf_layout)) return NVFP4_ERR_INVALID_ARG;
  if (t->cols % 16 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (t->rows * (t->cols / 8) >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(t->codes, 16) || !aligned(t->sf, 16) || !aligned(t->s_t, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

nvfp4_status check_cache(const nvfp4_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_sf || !c->v_sf || !c->k_st || !c->v_st)
    return NVFP4_ERR_INVALID_ARG;
  if (c->n_slots <= 0 || c->tokens_per_frame <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return NVFP4_ERR_INVALID_ARG;
  if (c->scale_rule != NVFP4_SCALE_ONTO_6 && c->scale_rule != NVFP4_SCALE_FOUR_OVER_SIX)
    return NVFP4_ERR_INVALID_ARG;
  if (c->head_dim % 16 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t per_frame = int64_t(c->tokens_per_frame) * c->heads * c->head_dim;
  if (per_frame * c->n_slots / 8 >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_sf, 16) ||
      !aligned(c->v_sf, 16) || !aligned(c->k_st, 4) || !aligned(c->v_st, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

bool valid_pages(int64_t n_pages, int64_t page_tokens) {
  return page_tokens % 16 == 0 && page_tokens <= NVFP4_KV8_MAX_PAGE_TOKENS &&
         n_pages * page_tokens < (int64_t(1) << 31);
}

nvfp4_status check_kv8(const nvfp4_kv8_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return NVFP4_ERR_INVALID_ARG;
  if (c->n_pages <= 0 || c->page_tokens <= 0 || c->kv_heads <= 0 || c->head_dim <= 0)
    return NVFP4_ERR_INVALID_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->kv_heads > 65535 ||
      !valid_pages(c->n_pages, c->page_tokens))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// The batch, and the sizes every kernel of the attention relies on.
nvfp4_status check_kv8_batch(const nvfp4_kv8_cache* c, const nvfp4_kv8_batch* b, int64_t tq,
                             int32_t q_heads, int32_t causal) {
  if (!b || !b->cu_q || !b->kv_lens || !b->block_table) return NVFP4_ERR_INVALID_ARG;
  if (b->batch < 1 || b->max_pages < 1 || b->max_q < 1 || b->max_kv < 1 ||
      b->table_stride < b->max_pages || tq < 0 || q_heads < 1 || (causal != 0 && causal != 1))
    return NVFP4_ERR_INVALID_ARG;
  if (q_heads % c->kv_heads != 0) return NVFP4_ERR_INVALID_ARG;
  if (b->batch > 65535 || tq * q_heads >= (int64_t(1) << 31) ||
      int64_t(b->max_q) * q_heads >= (int64_t(1) << 31) ||
      int64_t(b->max_pages) * c->page_tokens > NVFP4_KV8_MAX_TOKENS)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(b->cu_q, 4) || !aligned(b->kv_lens, 4) || !aligned(b->block_table, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

LaunchKv8Attn kv8_args(const nvfp4_kv8_cache* c, const nvfp4_kv8_batch* b, int64_t tq,
                       int32_t q_heads, int32_t causal, int sm_count) {
  LaunchKv8Attn d = {};
  d.k_codes = c->k_codes;
  d.v_codes = c->v_codes;
  d.k_scale = c->k_scale;
  d.v_scale = c->v_scale;
  d.n_pages = c->n_pages;
  d.page_tokens = c->page_tokens;
  d.kv_heads = c->kv_heads;
  d.head_dim = c->head_dim;
  d.tq = tq;
  d.q_heads = q_heads;
  d.cu_q = b->cu_q;
  d.kv_lens = b->kv_lens;
  d.table = b->block_table;
  d.table_stride = b->table_stride;
  d.batch = b->batch;
  d.max_pages = b->max_pages;
  // bounds beyond what the buffers hold would only make the grid larger
  d.max_q = int32_t(b->max_q < tq ? b->max_q : tq);
  if (d.max_q < 1) d.max_q = 1;
  const int64_t room = int64_t(b->max_pages) * c->page_tokens;
  d.max_kv = int32_t(b->max_kv < room ? b->max_kv : room);
  d.causal = causal;
  d.sm_count = sm_count;
  return d;
}

}  // namespace

extern "C" {

size_t nvfp4_codes_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols % 16 != 0) return 0;
  return size_t(rows) * size_t(cols / 2);
}

size_t nvfp4_sf_bytes(int64_t rows, int64_t cols, int32_t sf_layout) {
  if (rows < 0 || cols < 0 || cols % 16 != 0 || !valid_layout(sf_layout)) return 0;
  if (sf_layout == NVFP4_SF_ROWMAJOR) return size_t(rows) * size_t(cols / 16);
  const size_t rows_pad = size_t((rows + 127) / 128) * 128;
  const size_t blocks_pad = size_t((cols / 16 + 3) / 4) * 4;
  return rows_pad * blocks_pad;
}

size_t nvfp4_workspace_bytes(void) { return kWsBytes; }

void nvfp4_set_wait_limit_ns(uint64_t ns) { g_wait_limit_ns.store(ns); }

const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case NVFP4_ERR_MISALIGNED: return "misaligned pointer or stride";
    case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
    case NVFP4_ERR_ARCH: return "device is not sm_100 (B200)";
    case NVFP4_ERR_CUDA: return "CUDA error";
    case NVFP4_ERR_TIMEOUT: return "device wait timed out";
    case NVFP4_ERR_DOMAIN: return "tensor scale outside the recipe's domain";
    case NVFP4_ERR_CAPACITY: return "page pool, block table or slot map too small";
  }
  return "unknown status";
}

nvfp4_status nvfp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                            const nvfp4_tensor* out, const float* s_t_in, float* amax_in, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!x || (dtype != NVFP4_BF16 && dtype != NVFP4_FP32)) return NVFP4_ERR_INVALID_ARG;
  if (s_t_in && amax_in) return NVFP4_ERR_INVALID_ARG;
  nvfp4_status st = check_tensor(out);
  if (st != NVFP4_OK) return st;
  if (rows != out->rows || cols != out->cols || ld < cols) return NVFP4_ERR_INVALID_ARG;
  const int64_t esz = dtype == NVFP4_BF16 ? 2 : 4;
  if (!aligned(x, 16) || (ld * esz) % 16 != 0) return NVFP4_ERR_MISALIGNED;
  if ((s_t_in && !aligned(s_t_in, 4)) || (amax_in && !aligned(amax_in, 4)))
    return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchQuant q;
  q.x = x;
  q.dtype = dtype;
  q.rows = rows;
  q.cols = cols;
  q.ld = ld;
  q.codes = out->codes;
  q.sf = out->sf;
  q.sf_layout = out->sf_layout;
  q.s_t_out = out->s_t;
  q.s_t_in = s_t_in;
  q.amax_in = amax_in;
  q.ws = ws;
  q.sm_count = dev.sm_count;
  q.wait_limit_ns = g_wait_limit_ns.load();
  return cuda_status(launch_quantize(q, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_dequantize(const nvfp4_tensor* in, void* out, int64_t ld, void* stream) {
  nvfp4_status st = check_tensor(in);
  if (st != NVFP4_OK) return st;
  if (!out || ld < in->cols) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(out, 16) || ld % 8 != 0) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchDequant d;
  d.codes = in->codes;
  d.sf = in->sf;
  d.s_t = in->s_t;
  d.sf_layout = in->sf_layout;
  d.rows = in->rows;
  d.cols = in->cols;
  d.ld = ld;
  d.out = out;
  d.sm_count = dev.sm_count;
  return cuda_status(launch_dequantize(d, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* W, void* C, int32_t c_dtype,
                        int64_t ldc, int32_t act, float* c_amax, int64_t c_amax_cols, void* ws,
                        size_t ws_bytes, void* stream) {
  nvfp4_status st = check_tensor(A);
  if (st != NVFP4_OK) return st;
  st = check_tensor(W);
  if (st != NVFP4_OK) return st;
  if (!C || (c_dtype != NVFP4_BF16 && c_dtype != NVFP4_FP32)) return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_INVALID_ARG;
  if (A->sf_layout != NVFP4_SF_MMA128x4 || W->sf_layout != NVFP4_SF_MMA128x4)
    return NVFP4_ERR_INVALID_ARG;
  if (A->cols != W->cols) return NVFP4_ERR_INVALID_ARG;
  // K: whole 16-byte code rows (TMA); a K step past K reads TMA zero fill and the
  // scale layout's zero padding
  if (A->cols % 32 != 0 || W->rows < 1) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (A->rows >= (int64_t(1) << 31) || W->rows >= (int64_t(1) << 31))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ldc < W->rows) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(C, 16) || ldc % 8 != 0) return NVFP4_ERR_MISALIGNED;
  if (c_amax_cols < 0 || (c_amax_cols > 0 && (c_amax_cols % 256 != 0 || W->rows % c_amax_cols != 0)))
    return NVFP4_ERR_INVALID_ARG;
  if (c_amax && !aligned(c_amax, 4)) return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchGemm g;
  g.a_codes = A->codes;
  g.a_sf = A->sf;
  g.a_st = A->s_t;
  g.w_codes = W->codes;
  g.w_sf = W->sf;
  g.w_st = W->s_t;
  g.M = A->rows;
  g.N = W->rows;
  g.K = A->cols;
  g.c = C;
  g.c_dtype = c_dtype;
  g.ldc = ldc;
  g.act = act;
  g.c_amax = c_amax;
  g.c_amax_cols = c_amax_cols;
  g.ws = ws;
  g.wait_limit_ns = g_wait_limit_ns.load();
  g.sm_count = dev.sm_count;
  return cuda_status(launch_gemm(g, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_quant_chunk(const nvfp4_kv_cache* cache, const void* k, const void* v,
                                  int64_t token_stride, const int32_t* dst_slots, int32_t n_frames,
                                  float* k_amax_in, float* v_amax_in, void* ws, size_t ws_bytes,
                                  void* stream) {
  nvfp4_status st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (!k || !v || !dst_slots) return NVFP4_ERR_INVALID_ARG;
  if ((k_amax_in == nullptr) != (v_amax_in == nullptr)) return NVFP4_ERR_INVALID_ARG;
  if (n_frames < 1 || n_frames > NVFP4_KV_MAX_CHUNK_FRAMES) return NVFP4_ERR_INVALID_ARG;
  const int64_t row_elems = int64_t(cache->heads) * cache->head_dim;
  if (token_stride < row_elems) return NVFP4_ERR_INVALID_ARG;
  for (int f = 0; f < n_frames; ++f) {
    if (dst_slots[f] < 0 || dst_slots[f] >= cache->n_slots) return NVFP4_ERR_INVALID_ARG;
    for (int g = 0; g < f; ++g)
      if (dst_slots[g] == dst_slots[f]) return NVFP4_ERR_INVALID_ARG;
  }
  if (!aligned(k, 16) || !aligned(v, 16) || token_stride % 8 != 0) return NVFP4_ERR_MISALIGNED;
  if ((k_amax_in && !aligned(k_amax_in, 4)) || (v_amax_in && !aligned(v_amax_in, 4)))
    return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchKvQuant q;
  q.k = k;
  q.v = v;
  q.token_stride = token_stride;
  q.n_frames = n_frames;
  q.tpf = cache->tokens_per_frame;
  q.heads = cache->heads;
  q.head_dim = cache->head_dim;
  q.slots = dst_slots;
  q.k_codes = cache->k_codes;
  q.v_codes = cache->v_codes;
  q.k_sf = cache->k_sf;
  q.v_sf = cache->v_sf;
  q.k_st = cache->k_st;
  q.v_st = cache->v_st;
  q.k_amax_in = k_amax_in;
  q.v_amax_in = v_amax_in;
  q.scale_rule = cache->scale_rule;
  q.ws = ws;
  q.sm_count = dev.sm_count;
  q.wait_limit_ns = g_wait_limit_ns.load();
  return cuda_status(launch_kv_quant(q, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_dequant_window(const nvfp4_kv_cache* cache, const int32_t* slot_ids,
                                     int32_t n, void* k_out, void* v_out, void* stream) {
  nvfp4_status st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (!slot_ids || !k_out || !v_out || n < 1 || n > NVFP4_KV_MAX_WINDOW_SLOTS)
    return NVFP4_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (slot_ids[i] < 0 || slot_ids[i] >= cache->n_slots) return NVFP4_ERR_INVALID_ARG;
  const int64_t per_frame = int64_t(cache->tokens_per_frame) * cache->heads * cache->head_dim;
  if (per_frame * n / 8 >= (int64_t(1) << 32)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchKvDequant d;
  d.k_codes = cache->k_codes;
  d.v_codes = cache->v_codes;
  d.k_sf = cache->k_sf;
  d.v_sf = cache->v_sf;
  d.k_st = cache->k_st;
  d.v_st = cache->v_st;
  d.slots = slot_ids;
  d.n = n;
  d.tpf = cache->tokens_per_frame;
  d.heads = cache->heads;
  d.head_dim = cache->head_dim;
  d.k_out = k_out;
  d.v_out = v_out;
  d.sm_count = dev.sm_count;
  return cuda_status(launch_kv_dequant(d, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_window_attention(const nvfp4_kv_cache* cache, const int32_t* slot_ids,
                                    int32_t n, const void* q, int64_t q_token_stride, int64_t tq,
                                    float softmax_scale, void* out, int64_t out_token_stride,
                                    void* ws, size_t ws_bytes, void* stream) {
  nvfp4_status st = check_cache(cache);
  if (st != NVFP4_OK) return st;
  if (!slot_ids || !q || !out || n < 1 || n > NVFP4_KV_MAX_WINDOW_SLOTS)
    return NVFP4_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (slot_ids[i] < 0 || slot_ids[i] >= cache->n_slots) return NVFP4_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return NVFP4_ERR_INVALID_ARG;
  const int64_t row = int64_t(cache->heads) * cache->head_dim;
  if (q_token_stride < row || out_token_stride < row) return NVFP4_ERR_INVALID_ARG;
  if (cache->head_dim != 128 || tq < 1 || tq > (int64_t(1) << 30) || cache->heads > 65535 ||
      int64_t(n) * cache->tokens_per_frame >= (int64_t(1) << 31))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(q, 16) || !aligned(out, 16) || q_token_stride % 8 != 0 ||
      out_token_stride % 8 != 0)
    return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchAttn d;
  d.k_codes = cache->k_codes;
  d.v_codes = cache->v_codes;
  d.k_sf = cache->k_sf;
  d.v_sf = cache->v_sf;
  d.k_st = cache->k_st;
  d.v_st = cache->v_st;
  d.slot_ids = slot_ids;
  d.n = n;
  d.tpf = cache->tokens_per_frame;
  d.heads = cache->heads;
  d.q = q;
  d.out = out;
  d.q_stride = q_token_stride;
  d.out_stride = out_token_stride;
  d.tq = tq;
  d.scale_log2 = float(double(softmax_scale) * 1.4426950408889634);
  d.ws = ws;
  d.wait_limit_ns = g_wait_limit_ns.load();
  return cuda_status(launch_window_attention(d, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_gemv(const void* x, int32_t x_dtype, int64_t m, int64_t ldx,
                        const nvfp4_tensor* W, void* y, int32_t y_dtype, int64_t ldy, int32_t act,
                        void* stream) {
  nvfp4_status st = check_tensor(W);
  if (st != NVFP4_OK) return st;
  if (!x || !y || (x_dtype != NVFP4_BF16 && x_dtype != NVFP4_FP32) ||
      (y_dtype != NVFP4_BF16 && y_dtype != NVFP4_FP32))
    return NVFP4_ERR_INVALID_ARG;
  if (act != NVFP4_ACT_NONE && act != NVFP4_ACT_GELU_TANH) return NVFP4_ERR_INVALID_ARG;
  if (m < 1 || ldx < W->cols || ldy < W->rows) return NVFP4_ERR_INVALID_ARG;
  if (m > NVFP4_GEMV_MAX_ROWS || W->cols % 32 != 0 || W->rows >= (int64_t(1) << 30) ||
      W->cols >= (int64_t(1) << 30) ||
      nvfp4_sf_bytes(W->rows, W->cols, W->sf_layout) >= (size_t(1) << 31))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t xsz = x_dtype == NVFP4_BF16 ? 2 : 4, ysz = y_dtype == NVFP4_BF16 ? 2 : 4;
  if (!aligned(x, 16) || (ldx * xsz) % 16 != 0 || !aligned(y, uintptr_t(ysz)))
    return NVFP4_ERR_MISALIGNED;
  // y is written while other blocks still read x and W
  const Rows out = {y, m, W->rows * ysz, ldy * ysz};
  if (overlap(out, {x, m, W->cols * xsz, ldx * xsz}) ||
      overlap(out, block(W->codes, int64_t(nvfp4_codes_bytes(W->rows, W->cols)))) ||
      overlap(out, block(W->sf, int64_t(nvfp4_sf_bytes(W->rows, W->cols, W->sf_layout)))) ||
      overlap(out, block(W->s_t, 4)))
    return NVFP4_ERR_INVALID_ARG;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchGemv g;
  g.x = x;
  g.x_dtype = x_dtype;
  g.M = m;
  g.N = W->rows;
  g.K = W->cols;
  g.ldx = ldx;
  g.w_codes = W->codes;
  g.w_sf = W->sf;
  g.w_st = W->s_t;
  g.sf_layout = W->sf_layout;
  g.y = y;
  g.y_dtype = y_dtype;
  g.ldy = ldy;
  g.act = act;
  g.sm_count = dev.sm_count;
  return cuda_status(launch_gemv(g, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_plan_pages(const int32_t* cached_lens, const int32_t* new_lens, int32_t batch,
                              int32_t* block_table, int64_t table_stride, int32_t max_pages,
                              const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                              int32_t page_tokens, int32_t n_pages, int32_t* seq_lens,
                              int32_t* cu_new, int32_t* slot_map, int32_t max_new,
                              int32_t* free_head_out, void* ws, size_t ws_bytes, void* stream) {
  if (batch < 0 || max_pages < 0 || table_stride < max_pages || n_free < 0 || n_pages < 1 ||
      page_tokens < 1 || max_new < 0)
    return NVFP4_ERR_INVALID_ARG;
  if (!free_head || !free_head_out || !cu_new || (n_free > 0 && !free_pages) ||
      (max_new > 0 && !slot_map))
    return NVFP4_ERR_INVALID_ARG;
  if (batch > 0 && (!cached_lens || !new_lens || !seq_lens || (max_pages > 0 && !block_table)))
    return NVFP4_ERR_INVALID_ARG;
  if (batch > NVFP4_PLAN_MAX_BATCH || !valid_pages(n_pages, page_tokens) ||
      int64_t(max_pages) * page_tokens >= (int64_t(1) << 31))
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const void* ptrs[] = {cached_lens, new_lens, block_table, free_pages, free_head,
                        seq_lens,    cu_new,   slot_map,    free_head_out};
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return NVFP4_ERR_MISALIGNED;
  // an output that is also read (or written twice) would race between the CTAs
  struct Span {
    const int32_t* p;
    int64_t n;
  };
  const int64_t table = batch > 0 && max_pages > 0 ? (batch - 1) * table_stride + max_pages : 0;
  const Span spans[] = {{cached_lens, batch}, {new_lens, batch},      {free_pages, n_free},
                        {free_head, 1},       {block_table, table},   {seq_lens, batch},
                        {cu_new, batch + 1},  {slot_map, max_new},    {free_head_out, 1}};
  for (int i = 4; i < 9; ++i)
    for (int j = 0; j < i; ++j)
      if (spans[i].n > 0 && spans[j].n > 0 && spans[i].p < spans[j].p + spans[j].n &&
          spans[j].p < spans[i].p + spans[i].n)
        return NVFP4_ERR_INVALID_ARG;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  LaunchPlan p;
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.table = block_table;
  p.table_stride = table_stride;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.seq_lens = seq_lens;
  p.cu_new = cu_new;
  p.slot_map = slot_map;
  p.free_head_out = free_head_out;
  p.batch = batch;
  p.max_pages = max_pages;
  p.n_free = n_free;
  p.n_pages = n_pages;
  p.page_tokens = page_tokens;
  p.max_new = max_new;
  p.ws = ws;
  p.sm_count = dev.sm_count;
  return cuda_status(launch_plan(p, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv8_append(const nvfp4_kv8_cache* cache, const void* k, const void* v,
                              int64_t token_stride, int64_t tokens, const int32_t* slot_map,
                              void* ws, size_t ws_bytes, void* stream) {
  nvfp4_status st = check_kv8(cache);
  if (st != NVFP4_OK) return st;
  if (tokens < 0) return NVFP4_ERR_INVALID_ARG;
  if (tokens > 0 && (!k || !v || !slot_map)) return NVFP4_ERR_INVALID_ARG;
  if (token_stride < int64_t(cache->kv_heads) * cache->head_dim) return NVFP4_ERR_INVALID_ARG;
  if (tokens >= (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(k, 16) || !aligned(v, 16) || token_stride % 8 != 0 || !aligned(slot_map, 4))
    return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  if (tokens == 0) return NVFP4_OK;
  LaunchKv8Append p;
  p.k = k;
  p.v = v;
  p.token_stride = token_stride;
  p.tokens = tokens;
  p.slot_map = slot_map;
  p.k_codes = cache->k_codes;
  p.v_codes = cache->v_codes;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.n_pages = cache->n_pages;
  p.page_tokens = cache->page_tokens;
  p.heads = cache->kv_heads;
  p.head_dim = cache->head_dim;
  p.ws = ws;
  p.sm_count = dev.sm_count;
  return cuda_status(launch_kv8_append(p, static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_kv8_attention_scratch_bytes(const nvfp4_kv8_cache* cache,
                                         const nvfp4_kv8_batch* batch, int64_t tq, int32_t q_heads,
                                         int32_t causal) {
  if (check_kv8(cache) != NVFP4_OK || check_kv8_batch(cache, batch, tq, q_heads, causal) != NVFP4_OK)
    return 0;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return 0;
  return kv8_plan(kv8_args(cache, batch, tq, q_heads, causal, dev.sm_count)).scratch;
}

nvfp4_status nvfp4_kv8_attention(const nvfp4_kv8_cache* cache, const nvfp4_kv8_batch* batch,
                                 const void* q, int64_t q_token_stride, int64_t tq,
                                 int32_t q_heads, int32_t causal, float softmax_scale, void* out,
                                 int64_t out_token_stride, float* lse, void* scratch,
                                 size_t scratch_bytes, void* ws, size_t ws_bytes, void* stream) {
  nvfp4_status st = check_kv8(cache);
  if (st != NVFP4_OK) return st;
  st = check_kv8_batch(cache, batch, tq, q_heads, causal);
  if (st != NVFP4_OK) return st;
  if (tq > 0 && (!q || !out)) return NVFP4_ERR_INVALID_ARG;
  const float scale_log2 = float(double(softmax_scale) * 1.4426950408889634);
  if (!(softmax_scale > 0.0f) || !std::isfinite(scale_log2)) return NVFP4_ERR_INVALID_ARG;
  const int64_t row = int64_t(q_heads) * cache->head_dim;
  if (q_token_stride < row || out_token_stride < row) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || q_token_stride % 8 != 0 ||
      out_token_stride % 8 != 0 || !aligned(lse, 4) || !aligned(scratch, 16))
    return NVFP4_ERR_MISALIGNED;
  if (!ws || ws_bytes < kWsBytes) return NVFP4_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return NVFP4_ERR_MISALIGNED;
  // what is written has to be apart from what other blocks still read
  const Rows rows_out = {out, tq, row * 2, out_token_stride * 2};
  const Rows rows_lse = block(lse, tq * q_heads * 4);
  const int64_t scales = int64_t(cache->n_pages) * cache->kv_heads;
  const int64_t codes = scales * cache->page_tokens * cache->head_dim;
  const Rows read[] = {
      {q, tq, row * 2, q_token_stride * 2}, block(cache->k_codes, codes),
      block(cache->v_codes, codes), block(cache->k_scale, scales * 4),
      block(cache->v_scale, scales * 4), block(batch->cu_q, (int64_t(batch->batch) + 1) * 4),
      block(batch->kv_lens, int64_t(batch->batch) * 4),
      {batch->block_table, batch->batch, int64_t(batch->max_pages) * 4, batch->table_stride * 4}};
  for (const Rows& r : read)
    if (overlap(rows_out, r) || overlap(rows_lse, r)) return NVFP4_ERR_INVALID_ARG;
  if (overlap(rows_out, rows_lse)) return NVFP4_ERR_INVALID_ARG;
  const DeviceInfo dev = current_device();
  if (!dev.ok) return NVFP4_ERR_ARCH;
  if (tq == 0) return NVFP4_OK;
  LaunchKv8Attn d = kv8_args(cache, batch, tq, q_heads, causal, dev.sm_count);
  const size_t need = kv8_plan(d).scratch;
  if (need > 0 && (!scratch || scratch_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (overlap(block(scratch, int64_t(need)), rows_out) ||
      overlap(block(scratch, int64_t(need)), rows_lse) ||
      overlap(block(scratch, int64_t(need)), read[0]))
    return NVFP4_ERR_INVALID_ARG;
  d.q = q;
  d.q_stride = q_token_stride;
  d.out = out;
  d.out_stride = out_token_stride;
  d.lse = lse;
  d.scale_log2 = scale_log2;
  d.scratch = scratch;
  d.ws = ws;
  d.wait_limit_ns = g_wait_limit_ns.load();
  return cuda_status(launch_kv8_attention(d, static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_get_device_status(void* ws, void* stream) {
  if (!ws) return NVFP4_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  uint32_t* dev_word = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kWsStatus);
  if (cudaMemcpyAsync(&word, dev_word, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return NVFP4_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return NVFP4_ERR_CUDA;
  // cleared only where it is set: what another stream records in between is not lost
  if (word != 0) {
    if (cudaMemsetAsync(dev_word, 0, sizeof(word), s) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return NVFP4_ERR_CUDA;
  }
  return static_cast<nvfp4_status>(word);
}

}  // extern "C"
