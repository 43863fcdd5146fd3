// pkv_api.cu -- the extern "C" boundary of the library: argument checks,
// per-device facts, the device status word, launch tracing.
//
// Ownership and error rules follow the native-runtime contract of TensorRT
// Edge-LLM "HTTP Inference Server Architecture" ("Request Lifecycle",
// "Extension Rules": the native side owns retained pages and keeps a single
// writer; unsupported options are rejected up front) and the tensor-lifetime
// rule of the vLLM notes "EngineCoreClient ..." ("Flujo de datos": buffers
// stay alive until the asynchronous consumer is done with them).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <limits>
#include <mutex>
#include <vector>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

// One status word per device (each device that loads the library gets its
// own copy of this variable).
__device__ unsigned g_status_word;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_dev_mu;
DeviceInfo g_dev[kMaxDevices];
unsigned* g_status_addr[kMaxDevices];
std::atomic<uint64_t> g_launches{0};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_desc(const pkv_desc* d) {
  if (!d) return PKV_ERR_NULL;
  if (d->head_dim != kHeadDim || d->page_size != kPage) return PKV_ERR_SHAPE;
  if (d->num_kv_heads <= 0 || d->num_q_heads <= 0 || d->num_q_heads % d->num_kv_heads)
    return PKV_ERR_SHAPE;
  const int G = d->num_q_heads / d->num_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16) return PKV_ERR_SHAPE;
  if (d->num_blocks <= 0 || d->max_blocks_per_seq <= 0) return PKV_ERR_RANGE;
  // page byte offsets are computed in 64 bits; bound the pool to int32 pages
  return PKV_OK;
}

// Latent pages: one shared row a token, any number of query heads.
int check_latent_desc(const pkv_desc* d) {
  if (!d) return PKV_ERR_NULL;
  if (d->head_dim != kLatentRow || d->page_size != kPage || d->num_kv_heads != 1) return PKV_ERR_SHAPE;
  if (d->num_q_heads <= 0 || d->num_q_heads > PKV_LATENT_MAX_HEADS) return PKV_ERR_SHAPE;
  if (d->num_blocks <= 0 || d->max_blocks_per_seq <= 0) return PKV_ERR_RANGE;
  return PKV_OK;
}

// Rows, groups of eight cache rows and positions are int32 on the device (with
// a tile of rows or keys on top), and the work split adds its weights, heads x
// keys for each tile of 16 rows at the finest, up in 64 bits.
int check_latent_range(const pkv_desc* d, int32_t num_seqs, int32_t num_tokens) {
  constexpr int64_t top = int64_t(1) << 31;
  if (int64_t(num_tokens) * d->num_q_heads >= top - 1024 || int64_t(d->num_blocks) * 2 >= top ||
      int64_t(d->max_blocks_per_seq) * kPage >= top - 1024)
    return PKV_ERR_RANGE;
  const double heaviest = 2.0 * d->num_q_heads * (double(kPage) * d->max_blocks_per_seq + 1024);
  const double tiles = double(num_tokens) * d->num_q_heads / 16.0 + num_seqs;
  return heaviest * tiles < 9.0e18 ? PKV_OK : PKV_ERR_RANGE;
}

// Positions in a sequence are int32 on the device, with a tile of them on top.
int check_positions(const pkv_desc* d) {
  return int64_t(d->max_blocks_per_seq) * kPage >= (int64_t(1) << 31) - 1024 ? PKV_ERR_RANGE : PKV_OK;
}

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// A token stride in elements: rows of `row` elements, 16-byte aligned.
bool bad_stride(int64_t stride, int64_t row) { return stride < row || stride % 8; }

int check_rope(const pkv_rope* r, int max_dim) {
  if (!r || !r->cos_sin) return PKV_ERR_NULL;
  if (!aligned(r->cos_sin, 16)) return PKV_ERR_ALIGN;
  if (r->rotary_dim <= 0 || r->rotary_dim > max_dim || r->rotary_dim % 16) return PKV_ERR_SHAPE;
  if (r->max_position <= 0) return PKV_ERR_RANGE;
  return PKV_OK;
}

}  // namespace

const DeviceInfo* current_device(int* err) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    *err = PKV_ERR_DEVICE;
    return nullptr;
  }
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& info = g_dev[dev];
  if (info.device == dev) return &info;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) {
    *err = PKV_ERR_DEVICE;
    return nullptr;
  }
  if (prop.major != 10 || prop.minor != 3) {  // built for sm_103a only
    *err = PKV_ERR_DEVICE;
    return nullptr;
  }
  DeviceInfo fresh;
  fresh.device = dev;
  fresh.sm_count = prop.multiProcessorCount;
  fresh.cc_major = prop.major;
  fresh.cc_minor = prop.minor;
  fresh.smem_optin = prop.sharedMemPerBlockOptin;
  // A variant that cannot be resident gets 0 warps; pkv_attend then rejects
  // the head ratios that need it instead of failing here.
  for (int v = 0; v < 3; ++v) {
    fresh.dec_warps[v] = fresh.sm_count * decode_ctas_per_sm(v, false) * kDecWarps;
    fresh.dec_warps_f8[v] = fresh.sm_count * decode_ctas_per_sm(v, true) * kDecWarpsF8;
  }
  void* addr = nullptr;
  if (cudaGetSymbolAddress(&addr, g_status_word) != cudaSuccess) {
    *err = PKV_ERR_LAUNCH;
    return nullptr;
  }
  g_status_addr[dev] = static_cast<unsigned*>(addr);
  info = fresh;
  return &info;
}

unsigned* status_word(int device) {
  return device >= 0 && device < kMaxDevices ? g_status_addr[device] : nullptr;
}

static int make_ctx(pkv_stream_t stream, LaunchCtx* ctx) {
  int err = PKV_OK;
  const DeviceInfo* dev = current_device(&err);
  if (!dev) return err != PKV_OK ? err : PKV_ERR_DEVICE;
  ctx->stream = reinterpret_cast<cudaStream_t>(stream);
  ctx->dev = dev;
  ctx->status = g_status_addr[dev->device];
  return PKV_OK;
}

// ---------------------------------------------------------------------------
// tracing
// ---------------------------------------------------------------------------
}  // namespace pkv

struct pkv_trace {
  int device = -1;
  int capacity = 0;
  std::vector<cudaEvent_t> events;  // 2 per record
  std::vector<int> kernel;          // kernel id per record
  int used = 0;
  int64_t untimed[PKV_K_COUNT] = {};
};

namespace pkv {
namespace {
thread_local pkv_trace* t_trace = nullptr;
}

TraceScope::TraceScope(cudaStream_t s, int kernel_id) : stream_(s), kernel_(kernel_id), slot_(-1) {
  pkv_trace* tr = t_trace;
  if (tr) {
    if (tr->used < tr->capacity) {
      slot_ = tr->used++;
      tr->kernel[slot_] = kernel_id;
      cudaEventRecord(tr->events[2 * slot_], s);
    } else {
      tr->untimed[kernel_id]++;
    }
  }
}

int TraceScope::done() {
  const cudaError_t e = cudaGetLastError();
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (slot_ >= 0 && t_trace) cudaEventRecord(t_trace->events[2 * slot_ + 1], stream_);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

}  // namespace pkv

using namespace pkv;

static_assert(kMaxSeqs == PKV_MAX_SEQS, "the plan's shared-memory arrays hold PKV_MAX_SEQS sequences");

extern "C" {

int pkv_write(const pkv_bf16* k_new, const pkv_bf16* v_new, const int64_t* slot_mapping,
              int64_t num_tokens, pkv_bf16* k_cache, pkv_bf16* v_cache, const pkv_desc* desc,
              pkv_stream_t stream) {
  if (int e = check_desc(desc)) return e;
  if (num_tokens < 0) return PKV_ERR_RANGE;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_NULL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
    return PKV_ERR_ALIGN;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  return launch_write(ctx, k_new, v_new, slot_mapping, num_tokens, k_cache, v_cache,
                      desc->num_blocks, desc->num_kv_heads);
}

int pkv_attend_workspace_size(const pkv_desc* desc, int32_t num_seqs, int32_t num_tokens,
                              int32_t shared_prefix_pages, size_t* bytes) {
  if (int e = check_desc(desc)) return e;
  if (!bytes) return PKV_ERR_NULL;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0 || shared_prefix_pages < 0 ||
      shared_prefix_pages > desc->max_blocks_per_seq)
    return PKV_ERR_RANGE;
  int err = PKV_OK;
  const DeviceInfo* dev = current_device(&err);
  if (!dev) return err;
  *bytes = attend_workspace_bytes(*dev, *desc, num_seqs, num_tokens, shared_prefix_pages);
  return PKV_OK;
}

int pkv_attend_fp8_workspace_size(const pkv_desc* desc, int32_t num_seqs, int32_t num_tokens,
                                  int32_t shared_prefix_pages, size_t* bytes) {
  if (int e = check_desc(desc)) return e;
  if (!bytes) return PKV_ERR_NULL;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0 || shared_prefix_pages < 0 ||
      shared_prefix_pages > desc->max_blocks_per_seq)
    return PKV_ERR_RANGE;
  int err = PKV_OK;
  const DeviceInfo* dev = current_device(&err);
  if (!dev) return err;
  *bytes = attend_workspace_bytes(*dev, *desc, num_seqs, num_tokens, shared_prefix_pages, true);
  return PKV_OK;
}

int pkv_attend(const pkv_bf16* q, const pkv_bf16* k_cache, const pkv_bf16* v_cache,
               const int32_t* block_tables, const int32_t* seq_lens,
               const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens,
               int32_t max_query_len, int32_t shared_prefix_pages, float scale, pkv_bf16* out,
               void* workspace, size_t workspace_bytes, const pkv_desc* desc,
               pkv_stream_t stream) {
  if (int e = check_desc(desc)) return e;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0 || shared_prefix_pages < 0 ||
      shared_prefix_pages > desc->max_blocks_per_seq)
    return PKV_ERR_RANGE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc || !out ||
      !workspace)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
      !aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  AttendArgs a{q,          k_cache,    v_cache,    block_tables,  seq_lens,
               query_start_loc, num_seqs, num_tokens, max_query_len, shared_prefix_pages,
               scale,      out,        workspace,  workspace_bytes, *desc};
  return launch_attend(ctx, a);
}

int pkv_write_fp8(const pkv_bf16* k_new, const pkv_bf16* v_new, const int64_t* slot_mapping,
                  int64_t num_tokens, pkv_fp8* k_cache, pkv_fp8* v_cache, uint8_t* k_scale,
                  uint8_t* v_scale, const pkv_desc* desc, pkv_stream_t stream) {
  if (int e = check_desc(desc)) return e;
  if (num_tokens < 0) return PKV_ERR_RANGE;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale)
    return PKV_ERR_NULL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
    return PKV_ERR_ALIGN;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  return launch_write_fp8(ctx, k_new, v_new, slot_mapping, num_tokens, k_cache, v_cache, k_scale,
                          v_scale, desc->num_blocks, desc->num_kv_heads);
}

int pkv_attend_fp8(const pkv_bf16* q, const pkv_fp8* k_cache, const pkv_fp8* v_cache,
                   const uint8_t* k_scale, const uint8_t* v_scale, const int32_t* block_tables,
                   const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs,
                   int32_t num_tokens, int32_t max_query_len, int32_t shared_prefix_pages,
                   float scale, pkv_bf16* out,
                   void* workspace, size_t workspace_bytes, const pkv_desc* desc,
                   pkv_stream_t stream) {
  if (int e = check_desc(desc)) return e;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0 || shared_prefix_pages < 0 ||
      shared_prefix_pages > desc->max_blocks_per_seq)
    return PKV_ERR_RANGE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !seq_lens ||
      !query_start_loc || !out || !workspace)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) ||
      !aligned(v_scale, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  AttendArgs a{q,     k_cache, v_cache,   block_tables,    seq_lens, query_start_loc,
               num_seqs, num_tokens, max_query_len, shared_prefix_pages, scale, out, workspace,
               workspace_bytes, *desc};
  a.fp8 = true;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return launch_attend(ctx, a);
}

static pkv_rope one_axis(const pkv_rope_axes* r) {
  return r ? pkv_rope{r->cos_sin, r->max_position, r->rotary_dim, r->interleaved} : pkv_rope{};
}

static int write_rope(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, int64_t q_stride,
                      int64_t k_stride, int64_t v_stride, const int64_t* positions,
                      const int64_t* slot_mapping, int64_t num_tokens, const pkv_rope* rope,
                      pkv_bf16* q_out, void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale,
                      const pkv_desc* desc, pkv_stream_t stream, bool fp8, const pkv_rope_axes* axes = nullptr,
                      int64_t position_stride = 0) {
  if (int e = check_desc(desc)) return e;
  if (num_tokens < 0) return PKV_ERR_RANGE;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !positions || !slot_mapping || !k_cache || !v_cache || !q != !q_out ||
      (fp8 && (!k_scale || !v_scale)))
    return PKV_ERR_NULL;
  if (int e = check_rope(rope, kHeadDim)) return e;
  if (axes) {
    if (!axes->axis_of_pair) return PKV_ERR_NULL;
    if (axes->num_axes < 1 || axes->num_axes > PKV_MAX_AXES || position_stride < 0) return PKV_ERR_RANGE;
    for (int i = 0; i < rope->rotary_dim / 2; ++i)
      if (axes->axis_of_pair[i] >= axes->num_axes) return PKV_ERR_RANGE;
  }
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(q, 16) || !aligned(q_out, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) ||
      !aligned(positions, 8) || !aligned(slot_mapping, 8))
    return PKV_ERR_ALIGN;
  const int64_t kv_row = int64_t(desc->num_kv_heads) * kHeadDim;
  if (bad_stride(k_stride, kv_row) || bad_stride(v_stride, kv_row) ||
      (q && bad_stride(q_stride, int64_t(desc->num_q_heads) * kHeadDim)))
    return PKV_ERR_SHAPE;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  RopeWriteArgs a{};
  a.q = q, a.k = k_new, a.v = v_new;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.positions = positions, a.slots = slot_mapping, a.num_tokens = num_tokens;
  a.cos_sin = rope->cos_sin;
  a.max_position = rope->max_position, a.rotary_dim = rope->rotary_dim, a.interleaved = rope->interleaved;
  a.q_out = q_out, a.k_cache = k_cache, a.v_cache = v_cache, a.k_scale = k_scale, a.v_scale = v_scale;
  a.num_blocks = desc->num_blocks, a.num_q_heads = desc->num_q_heads, a.num_kv_heads = desc->num_kv_heads;
  a.status = ctx.status;
  if (axes) {
    a.num_axes = axes->num_axes;
    a.position_stride = position_stride;
    for (int i = 0; i < rope->rotary_dim / 2; ++i) a.axis_pairs[axes->axis_of_pair[i]] |= uint64_t(1) << i;
  }
  return launch_write_rope(ctx, a, fp8);
}

int pkv_write_rope(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, int64_t q_stride,
                   int64_t k_stride, int64_t v_stride, const int64_t* positions,
                   const int64_t* slot_mapping, int64_t num_tokens, const pkv_rope* rope,
                   pkv_bf16* q_out, pkv_bf16* k_cache, pkv_bf16* v_cache, const pkv_desc* desc,
                   pkv_stream_t stream) {
  return write_rope(q, k_new, v_new, q_stride, k_stride, v_stride, positions, slot_mapping, num_tokens, rope,
                    q_out, k_cache, v_cache, nullptr, nullptr, desc, stream, false);
}

int pkv_write_rope_fp8(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, const int64_t* positions,
                       const int64_t* slot_mapping, int64_t num_tokens, const pkv_rope* rope,
                       pkv_bf16* q_out, pkv_fp8* k_cache, pkv_fp8* v_cache, uint8_t* k_scale,
                       uint8_t* v_scale, const pkv_desc* desc, pkv_stream_t stream) {
  return write_rope(q, k_new, v_new, q_stride, k_stride, v_stride, positions, slot_mapping, num_tokens, rope,
                    q_out, k_cache, v_cache, k_scale, v_scale, desc, stream, true);
}

int pkv_write_rope_axes(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, int64_t q_stride,
                        int64_t k_stride, int64_t v_stride, const int64_t* positions, int64_t position_stride,
                        const int64_t* slot_mapping, int64_t num_tokens, const pkv_rope_axes* rope,
                        pkv_bf16* q_out, pkv_bf16* k_cache, pkv_bf16* v_cache, const pkv_desc* desc,
                        pkv_stream_t stream) {
  if (!rope && num_tokens != 0) return PKV_ERR_NULL;
  const pkv_rope one = one_axis(rope);
  return write_rope(q, k_new, v_new, q_stride, k_stride, v_stride, positions, slot_mapping, num_tokens, &one,
                    q_out, k_cache, v_cache, nullptr, nullptr, desc, stream, false, rope, position_stride);
}

int pkv_write_rope_axes_fp8(const pkv_bf16* q, const pkv_bf16* k_new, const pkv_bf16* v_new, int64_t q_stride,
                            int64_t k_stride, int64_t v_stride, const int64_t* positions,
                            int64_t position_stride, const int64_t* slot_mapping, int64_t num_tokens,
                            const pkv_rope_axes* rope, pkv_bf16* q_out, pkv_fp8* k_cache, pkv_fp8* v_cache,
                            uint8_t* k_scale, uint8_t* v_scale, const pkv_desc* desc, pkv_stream_t stream) {
  if (!rope && num_tokens != 0) return PKV_ERR_NULL;
  const pkv_rope one = one_axis(rope);
  return write_rope(q, k_new, v_new, q_stride, k_stride, v_stride, positions, slot_mapping, num_tokens, &one,
                    q_out, k_cache, v_cache, k_scale, v_scale, desc, stream, true, rope, position_stride);
}

int pkv_write_latent(const pkv_bf16* c_new, const pkv_bf16* k_pe, const pkv_bf16* q_pe, int64_t c_stride,
                     int64_t k_stride, int64_t q_stride, int64_t q_head_stride, const int64_t* positions,
                     const int64_t* slot_mapping, int64_t num_tokens, const pkv_rope* rope,
                     pkv_bf16* q_out, pkv_bf16* latent_cache, const pkv_desc* desc, pkv_stream_t stream) {
  if (int e = check_latent_desc(desc)) return e;
  if (num_tokens < 0) return PKV_ERR_RANGE;
  if (num_tokens == 0) return PKV_OK;
  if (!c_new || !k_pe || !positions || !slot_mapping || !latent_cache || !q_pe != !q_out) return PKV_ERR_NULL;
  if (int e = check_rope(rope, kLatentRope)) return e;
  if (rope->rotary_dim != kLatentRope) return PKV_ERR_SHAPE;
  if (!aligned(c_new, 16) || !aligned(k_pe, 16) || !aligned(q_pe, 16) || !aligned(q_out, 16) ||
      !aligned(latent_cache, 16) || !aligned(positions, 8) || !aligned(slot_mapping, 8))
    return PKV_ERR_ALIGN;
  if (bad_stride(c_stride, kLatentDim) || bad_stride(k_stride, kLatentRope) ||
      (q_pe && (bad_stride(q_head_stride, kLatentRope) ||
                bad_stride(q_stride, (desc->num_q_heads - 1) * q_head_stride + kLatentRope))))
    return PKV_ERR_SHAPE;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  LatentWriteArgs a{};
  a.c_new = c_new, a.k_pe = k_pe, a.q_pe = q_pe;
  a.c_stride = c_stride, a.k_stride = k_stride, a.q_stride = q_stride, a.q_head_stride = q_head_stride;
  a.positions = positions, a.slots = slot_mapping, a.num_tokens = num_tokens;
  a.cos_sin = rope->cos_sin;
  a.max_position = rope->max_position, a.interleaved = rope->interleaved;
  a.q_out = q_out, a.cache = latent_cache;
  a.num_blocks = desc->num_blocks, a.num_heads = desc->num_q_heads;
  a.status = ctx.status;
  return launch_write_latent(ctx, a);
}

int pkv_attend_latent_workspace_size(const pkv_desc* desc, int32_t num_seqs, int32_t num_tokens,
                                     size_t* bytes) {
  if (int e = check_latent_desc(desc)) return e;
  if (!bytes) return PKV_ERR_NULL;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0) return PKV_ERR_RANGE;
  int err = PKV_OK;
  const DeviceInfo* dev = current_device(&err);
  if (!dev) return err;
  *bytes = latent_workspace_bytes(*dev);
  return PKV_OK;
}

int pkv_attend_latent(const pkv_bf16* q, const pkv_bf16* latent_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* query_start_loc, int32_t num_seqs,
                      int32_t num_tokens, int32_t max_query_len, float scale, pkv_bf16* out,
                      void* workspace, size_t workspace_bytes, const pkv_desc* desc, pkv_stream_t stream) {
  if (int e = check_latent_desc(desc)) return e;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0) return PKV_ERR_RANGE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !latent_cache || !block_tables || !seq_lens || !query_start_loc || !out || !workspace)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(latent_cache, 16) || !aligned(out, 16) || !aligned(block_tables, 4) ||
      !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  if (int e = check_latent_range(desc, num_seqs, num_tokens)) return e;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  const LatentAttendArgs a{q,          latent_cache, block_tables, seq_lens,  query_start_loc, num_seqs,
                           num_tokens, max_query_len, scale,       out,       workspace,       workspace_bytes,
                           *desc};
  return launch_attend_latent(ctx, a);
}

// Units of work and keys are counted in 64 bits on the device, tokens, positions
// and rows of the pool in 32.
static int check_weigh(const pkv_desc* d, int32_t num_seqs, int32_t num_tokens) {
  if (int e = check_desc(d)) return e;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || num_tokens < 0 || num_tokens > INT32_MAX - 1024)
    return PKV_ERR_RANGE;
  if (int64_t(d->num_blocks) * d->num_kv_heads >= (int64_t(1) << 31) / kPage) return PKV_ERR_RANGE;
  return check_positions(d);
}

// The host's bounds as they are used: where unknown, what the call's sizes allow.
static int32_t most_rows(int32_t max_query_len, int32_t num_tokens) {
  return max_query_len > 0 ? std::min(max_query_len, num_tokens) : num_tokens;
}
// (A pool's tokens bound the keys of sequences that share no more pages than are
// free; others pass num_keys.)
static int64_t most_keys(const pkv_desc* d, int32_t num_seqs, int64_t num_keys) {
  const int64_t top = int64_t(num_seqs) * d->max_blocks_per_seq * kPage;
  return std::min(num_keys > 0 ? num_keys : int64_t(d->num_blocks) * kPage, top);
}

int pkv_weigh_workspace_size(const pkv_desc* desc, int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
                             int64_t num_keys, size_t* bytes) {
  if (int e = check_weigh(desc, num_seqs, num_tokens)) return e;
  if (!bytes) return PKV_ERR_NULL;
  int err = PKV_OK;
  const DeviceInfo* dev = current_device(&err);
  if (!dev) return err;
  *bytes = weigh_workspace_bytes(*dev, *desc, num_seqs, num_tokens, most_rows(max_query_len, num_tokens),
                                 most_keys(desc, num_seqs, num_keys));
  return PKV_OK;
}

static int weigh(const pkv_bf16* q, const void* k_cache, const uint8_t* k_scale, float* scores,
                 const int32_t* block_tables, const int32_t* seq_lens, const int32_t* query_start_loc,
                 const int32_t* first, const int32_t* scored, int32_t num_seqs, int32_t num_tokens,
                 int32_t max_query_len, int64_t num_keys, float scale, float decay, void* workspace,
                 size_t workspace_bytes, const pkv_desc* desc, pkv_stream_t stream, bool fp8) {
  if (int e = check_weigh(desc, num_seqs, num_tokens)) return e;
  // (not >=: a NaN is refused too; the kernels have the scale times log2(e))
  const float qscale = scale * 1.4426950408889634f;
  if (!(scale >= 0.f) || !std::isfinite(qscale) || !(decay >= 0.f) || !std::isfinite(decay)) return PKV_ERR_RANGE;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!q || !k_cache || (fp8 && !k_scale) || !scores || !block_tables || !seq_lens || !query_start_loc || !workspace)
    return PKV_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(k_scale, 16) || !aligned(scores, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(first, 4) ||
      !aligned(scored, 4) || !aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  WeighArgs a{};
  a.q = q, a.k_cache = k_cache, a.k_scale = k_scale, a.scores = scores;
  a.block_tables = block_tables, a.seq_lens = seq_lens, a.query_start_loc = query_start_loc;
  a.first = first, a.scored = scored;
  a.num_seqs = num_seqs, a.num_tokens = num_tokens;
  a.max_rows = most_rows(max_query_len, num_tokens);
  a.num_keys = most_keys(desc, num_seqs, num_keys);
  // (a masked score is -infinity: scale 0, all keys alike, is a scale too small to part them)
  a.qscale = std::max(qscale, std::numeric_limits<float>::min());
  a.decay = decay;
  a.workspace = workspace, a.workspace_bytes = workspace_bytes;
  a.desc = *desc;
  a.status = ctx.status;
  return launch_weigh(ctx, a, fp8);
}

int pkv_weigh(const pkv_bf16* q, const pkv_bf16* k_cache, float* scores, const int32_t* block_tables,
              const int32_t* seq_lens, const int32_t* query_start_loc, const int32_t* first, const int32_t* scored,
              int32_t num_seqs, int32_t num_tokens, int32_t max_query_len, int64_t num_keys, float scale,
              float decay, void* workspace, size_t workspace_bytes, const pkv_desc* desc, pkv_stream_t stream) {
  return weigh(q, k_cache, nullptr, scores, block_tables, seq_lens, query_start_loc, first, scored, num_seqs,
               num_tokens, max_query_len, num_keys, scale, decay, workspace, workspace_bytes, desc, stream, false);
}

int pkv_weigh_fp8(const pkv_bf16* q, const pkv_fp8* k_cache, const uint8_t* k_scale, float* scores,
                  const int32_t* block_tables, const int32_t* seq_lens, const int32_t* query_start_loc,
                  const int32_t* first, const int32_t* scored, int32_t num_seqs, int32_t num_tokens,
                  int32_t max_query_len, int64_t num_keys, float scale, float decay, void* workspace,
                  size_t workspace_bytes, const pkv_desc* desc, pkv_stream_t stream) {
  return weigh(q, k_cache, k_scale, scores, block_tables, seq_lens, query_start_loc, first, scored, num_seqs,
               num_tokens, max_query_len, num_keys, scale, decay, workspace, workspace_bytes, desc, stream, true);
}

int pkv_evict_workspace_size(const pkv_desc* desc, int32_t num_seqs, size_t* bytes) {
  if (int e = check_desc(desc)) return e;
  if (!bytes) return PKV_ERR_NULL;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS) return PKV_ERR_RANGE;
  if (int e = check_positions(desc)) return e;
  *bytes = evict_workspace_bytes(*desc, num_seqs);
  return PKV_OK;
}

static int evict(void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale, float* scores,
                 const int32_t* block_tables, const int32_t* seq_lens, const int32_t* keep, const int32_t* first,
                 int32_t recent, int32_t num_seqs, int32_t* new_lens, void* workspace, size_t workspace_bytes,
                 const pkv_desc* desc, pkv_stream_t stream, bool fp8) {
  if (int e = check_desc(desc)) return e;
  if (num_seqs < 0 || num_seqs > PKV_MAX_SEQS || recent < 0) return PKV_ERR_RANGE;
  if (int e = check_positions(desc)) return e;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !scores || !block_tables || !seq_lens || !keep || !new_lens || !workspace ||
      (fp8 && (!k_scale || !v_scale)))
    return PKV_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) ||
      !aligned(scores, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(keep, 4) ||
      !aligned(first, 4) || !aligned(new_lens, 4) || !aligned(workspace, 256))
    return PKV_ERR_ALIGN;
  // a CTA of one head writes a new length while others read the old one
  const size_t bytes = sizeof(int32_t) * size_t(num_seqs);
  if (overlap(new_lens, bytes, seq_lens, bytes) || overlap(new_lens, bytes, keep, bytes) ||
      (first && overlap(new_lens, bytes, first, bytes)))
    return PKV_ERR_RANGE;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  const EvictArgs a{k_cache, v_cache, k_scale,  v_scale,  scores,    block_tables,    seq_lens, keep,
                    first,   recent,  num_seqs, new_lens, workspace, workspace_bytes, *desc,    ctx.status};
  return launch_evict(ctx, a, fp8);
}

int pkv_evict(pkv_bf16* k_cache, pkv_bf16* v_cache, float* scores, const int32_t* block_tables,
              const int32_t* seq_lens, const int32_t* keep, const int32_t* first, int32_t recent, int32_t num_seqs,
              int32_t* new_lens, void* workspace, size_t workspace_bytes, const pkv_desc* desc,
              pkv_stream_t stream) {
  return evict(k_cache, v_cache, nullptr, nullptr, scores, block_tables, seq_lens, keep, first, recent, num_seqs,
               new_lens, workspace, workspace_bytes, desc, stream, false);
}

int pkv_evict_fp8(pkv_fp8* k_cache, pkv_fp8* v_cache, uint8_t* k_scale, uint8_t* v_scale, float* scores,
                  const int32_t* block_tables, const int32_t* seq_lens, const int32_t* keep, const int32_t* first,
                  int32_t recent, int32_t num_seqs, int32_t* new_lens, void* workspace, size_t workspace_bytes,
                  const pkv_desc* desc, pkv_stream_t stream) {
  return evict(k_cache, v_cache, k_scale, v_scale, scores, block_tables, seq_lens, keep, first, recent, num_seqs,
               new_lens, workspace, workspace_bytes, desc, stream, true);
}

int pkv_get_last_error(pkv_stream_t stream, uint32_t* flags) {
  if (!flags) return PKV_ERR_NULL;
  LaunchCtx ctx{};
  if (int e = make_ctx(stream, &ctx)) return e;
  unsigned host = 0;
  if (cudaMemcpyAsync(&host, ctx.status, sizeof(unsigned), cudaMemcpyDeviceToHost, ctx.stream) !=
          cudaSuccess ||
      cudaMemsetAsync(ctx.status, 0, sizeof(unsigned), ctx.stream) != cudaSuccess ||
      cudaStreamSynchronize(ctx.stream) != cudaSuccess)
    return PKV_ERR_LAUNCH;
  *flags = host;
  return PKV_OK;
}

const char* pkv_strerror(int code) {
  switch (code) {
    case PKV_OK: return "ok";
    case PKV_ERR_NULL: return "a required pointer is NULL";
    case PKV_ERR_ALIGN: return "a pointer is not aligned as required (16 B tensors, 256 B workspace)";
    case PKV_ERR_SHAPE: return "unsupported geometry (head_dim 128, page_size 16, Hq/Hkv in {1,2,4,8,16})";
    case PKV_ERR_RANGE: return "a count or size is out of range";
    case PKV_ERR_WORKSPACE: return "workspace smaller than pkv_attend_workspace_size";
    case PKV_ERR_LAUNCH: return "a CUDA launch or runtime call failed";
    case PKV_ERR_DEVICE: return "the current device is not an sm_103 (GB300) GPU";
    case PKV_ERR_STATE: return "trace API misuse";
    case PKV_ERR_SCRATCH: return "batch needs more scratch than PKV_STATIC_SCRATCH_BYTES (use pkv_attend with a workspace)";
    case PKV_ERR_NOSPACE: return "page pool: not enough free pages";
    default: return "unknown error";
  }
}

uint64_t pkv_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int pkv_trace_create(int32_t capacity, pkv_trace** out) {
  if (!out) return PKV_ERR_NULL;
  if (capacity <= 0) return PKV_ERR_RANGE;
  auto* tr = new pkv_trace();
  cudaGetDevice(&tr->device);
  tr->capacity = capacity;
  tr->events.resize(2 * size_t(capacity));
  tr->kernel.assign(capacity, -1);
  for (auto& e : tr->events) {
    if (cudaEventCreate(&e) != cudaSuccess) {
      e = nullptr;
      pkv_trace_destroy(tr);
      return PKV_ERR_LAUNCH;
    }
  }
  *out = tr;
  return PKV_OK;
}

int pkv_trace_attach(pkv_trace* tr) {
  if (!tr) return PKV_ERR_NULL;
  if (t_trace) return PKV_ERR_STATE;
  t_trace = tr;
  return PKV_OK;
}

int pkv_trace_detach(void) {
  if (!t_trace) return PKV_ERR_STATE;
  t_trace = nullptr;
  return PKV_OK;
}

int pkv_trace_read(pkv_trace* tr, int32_t kernel_id, double* total_ms, int64_t* launches) {
  if (!tr || !total_ms || !launches) return PKV_ERR_NULL;
  if (kernel_id < 0 || kernel_id >= PKV_K_COUNT) return PKV_ERR_RANGE;
  double ms = 0;
  int64_t n = 0;
  for (int i = 0; i < tr->used; ++i) {
    if (tr->kernel[i] != kernel_id) continue;
    if (cudaEventSynchronize(tr->events[2 * i + 1]) != cudaSuccess) return PKV_ERR_LAUNCH;
    float x = 0;
    if (cudaEventElapsedTime(&x, tr->events[2 * i], tr->events[2 * i + 1]) != cudaSuccess)
      return PKV_ERR_LAUNCH;
    ms += x;
    ++n;
  }
  *total_ms = ms;
  *launches = n + tr->untimed[kernel_id];
  return PKV_OK;
}

int pkv_trace_reset(pkv_trace* tr) {
  if (!tr) return PKV_ERR_NULL;
  tr->used = 0;
  for (auto& u : tr->untimed) u = 0;
  return PKV_OK;
}

int pkv_trace_destroy(pkv_trace* tr) {
  if (!tr) return PKV_ERR_NULL;
  if (t_trace == tr) t_trace = nullptr;
  for (auto e : tr->events)
    if (e) cudaEventDestroy(e);
  delete tr;
  return PKV_OK;
}

}  // extern "C"
