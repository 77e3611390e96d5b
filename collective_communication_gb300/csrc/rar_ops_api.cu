// rar_ops_api.cu -- the C ABI of the operators around the collectives (declared
// in include/rar.h): argument checks, workspaces, launches. Nothing here waits
// for the device; what only the device can see (lengths, positions, page and
// slot numbers) is checked by the kernels and reported through the status word.
#include <atomic>
#include <cstring>

#include "op_common.cuh"
#include "prompt_attention.cuh"
#include "rar.h"
#include "rar_launch.h"

namespace rar {
namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 256;

rar_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return RAR_OK;
  (void)cudaGetLastError();
  return RAR_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// `rows` rows of `width` bytes, `stride` bytes from row to row; of their bytes (if `every` is set) those alone that are
// less than `part` behind the base, or behind a multiple of `every` from there.
struct Span {
  uintptr_t base;
  int64_t rows, width, stride;
  int64_t part = 0, every = 0;
};
Span span(const void* p, int64_t rows, int64_t width, int64_t stride) {
  return Span{(uintptr_t)p, rows, width, stride, 0, 0};
}
Span span(const void* p, int64_t bytes) { return Span{(uintptr_t)p, 1, bytes, bytes, 0, 0}; }

// Whether parts of two rows of bytes that repeat after `stride` leave each other alone, whatever their number.
bool interleave(const Span& a, const Span& b, int64_t stride, int64_t a_width, int64_t b_width) {
  const bool first = a.base <= b.base;
  const int64_t d = (int64_t)((first ? b.base - a.base : a.base - b.base) % (uintptr_t)stride);
  return d >= (first ? a_width : b_width) && stride - d >= (first ? b_width : a_width);
}
// Whether two spans share a byte. Spans of one stride may interleave (the ranks'
// heads side by side in one row); spans of different strides must not meet at all.
bool meet(const Span& a, const Span& b) {
  if (a.base == 0 || b.base == 0 || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  const uintptr_t ae = a.base + (uintptr_t)((a.rows - 1) * a.stride + a.width);
  const uintptr_t be = b.base + (uintptr_t)((b.rows - 1) * b.stride + b.width);
  if (!(a.base < be && b.base < ae)) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride && interleave(a, b, a.stride, a.width, b.width)) return false;
  if (a.every > 0 && a.every == b.every && interleave(a, b, a.every, a.part, b.part)) return false;
  return true;
}

// Inputs and outputs of a call: an output may meet nothing else.
struct Spans {
  Span in[6 * kMaxRanks + 16];
  Span out[3 * kMaxRanks + 16];
  int nin = 0, nout = 0;
  void read(const Span& s) { in[nin++] = s; }
  void write(const Span& s) { out[nout++] = s; }
  bool clash() const {
    for (int i = 0; i < nout; i++) {
      for (int j = 0; j < nin; j++)
        if (meet(out[i], in[j])) return true;
      for (int j = 0; j < i; j++)
        if (meet(out[i], out[j])) return true;
    }
    return false;
  }
};

rar_status check_ranks(int nranks, rar_dtype dtype) {
  if (nranks < 1 || nranks > kMaxRanks) return RAR_ERR_ARG;
  if (dtype != RAR_F32 && dtype != RAR_BF16) return RAR_ERR_ARG;
  return RAR_OK;
}
int64_t size_of(rar_dtype dtype) { return dtype == RAR_F32 ? 4 : 2; }

// A rank's pointer may be null only if there is nothing behind it (rows 0).
rar_status check_pointers(const void* const* p, int nranks, int64_t rows, uintptr_t to) {
  if (p == nullptr) return RAR_ERR_ARG;
  for (int r = 0; r < nranks; r++)
    if (p[r] == nullptr && rows > 0) return RAR_ERR_ARG;
  for (int r = 0; r < nranks; r++)
    if (!aligned(p[r], to)) return RAR_ERR_ALIGN;
  return RAR_OK;
}

rar_status check_workspace(const void* ws, size_t bytes, int64_t scratch) {
  if (ws == nullptr) return RAR_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return RAR_ERR_ALIGN;
  if (bytes < (size_t)(kOpScratchOffset + scratch)) return RAR_ERR_WORKSPACE;
  return RAR_OK;
}

// log2 of a page size, or -1: pages hold 1 to 1024 tokens, a power of two.
int page_shift_of(int page_size) {
  for (int s = 0; s <= 10; s++)
    if (page_size == 1 << s) return s;
  return -1;
}
// Slots, and the cache rows that they are for each key head, are 32-bit numbers.
bool pages_ok(int num_pages, int shift, int64_t kv_heads) {
  return num_pages >= 1 && ((int64_t)num_pages << shift) <= INT32_MAX / kv_heads;
}

bool heads_ok(int q_heads, int kv_heads, int head_dim) {
  return q_heads >= 1 && q_heads <= kMaxHeads && kv_heads >= 1 && kv_heads <= kMaxHeads && head_dim >= 8 &&
         head_dim <= kMaxHeadDim && head_dim % 8 == 0;
}
// A stride in elements that keeps every row on a 16-byte boundary and rows apart.
rar_status check_stride(int64_t stride, int64_t width, int64_t rows, int64_t es) {
  if (rows > 1 && stride < width) return RAR_ERR_ARG;
  if (stride < 0 || stride > INT64_MAX / 8 / (rows > 0 ? rows : 1)) return RAR_ERR_ARG;
  if (stride * es % 16 != 0) return RAR_ERR_ALIGN;
  return RAR_OK;
}

struct NormRopeCall {
  int nranks;
  int64_t tokens, qkv_stride;
  const void* q_weight;
  const void* k_weight;
  const float* cos_sin;
  int max_pos, rot_dim;
  const int32_t* positions;
  int q_heads, kv_heads, head_dim;
  rar_dtype dtype;
};

// What the three forms of the norm and rotation share.
rar_status check_norm_rope(const NormRopeCall& c, const void* const* qkv, Spans* s) {
  rar_status st = check_ranks(c.nranks, c.dtype);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(c.dtype);
  if (!heads_ok(c.q_heads, c.kv_heads, c.head_dim)) return RAR_ERR_ARG;
  if (c.rot_dim < 8 || c.rot_dim > c.head_dim || c.rot_dim % 8 != 0 || c.max_pos < 1) return RAR_ERR_ARG;
  const int64_t heads = c.q_heads + 2 * (int64_t)c.kv_heads;
  if (c.tokens < 0 || c.tokens * heads > INT32_MAX) return RAR_ERR_ARG;
  if ((st = check_pointers(qkv, c.nranks, c.tokens, 16)) != RAR_OK) return st;
  if (c.q_weight == nullptr || c.k_weight == nullptr || c.cos_sin == nullptr) return RAR_ERR_ARG;
  if (c.tokens > 0 && c.positions == nullptr) return RAR_ERR_ARG;
  if (!aligned(c.q_weight, 16) || !aligned(c.k_weight, 16) || !aligned(c.cos_sin, 16) || !aligned(c.positions, 4))
    return RAR_ERR_ALIGN;
  if ((st = check_stride(c.qkv_stride, heads * c.head_dim, c.tokens, es)) != RAR_OK) return st;
  s->read(span(c.q_weight, c.head_dim * es));
  s->read(span(c.k_weight, c.head_dim * es));
  s->read(span(c.cos_sin, (int64_t)c.max_pos * c.rot_dim * 4));
  s->read(span(c.positions, c.tokens * 4));
  return RAR_OK;
}

struct Residency {
  std::atomic<const void*> fn;
  std::atomic<int> device, blocks;
};
constexpr int kResidencies = 128;
Residency g_residency[kResidencies];
std::atomic<int> g_residencies{0};

}  // namespace

cudaError_t resident_blocks(const void* fn, int threads, int shared, int* blocks) {
  int device = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&device, &sms);
  if (e != cudaSuccess) return e;
  const int known = g_residencies.load(std::memory_order_acquire);
  for (int i = 0; i < known && i < kResidencies; i++) {
    // an entry is complete once its kernel is set
    if (g_residency[i].fn.load(std::memory_order_acquire) == fn && g_residency[i].device.load() == device) {
      *blocks = g_residency[i].blocks.load();
      return cudaSuccess;
    }
  }
  if (shared > 0) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
    if (e != cudaSuccess) return e;
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, (size_t)shared);
  if (e != cudaSuccess) return e;
  *blocks = sms * per_sm;
  const int slot = g_residencies.fetch_add(1);
  if (slot < kResidencies) {
    g_residency[slot].device.store(device);
    g_residency[slot].blocks.store(*blocks);
    g_residency[slot].fn.store(fn, std::memory_order_release);
  } else {
    g_residencies.store(kResidencies);
  }
  return cudaSuccess;
}

__global__ void init_op_header_kernel(char* ws) {
  OpHeader* h = reinterpret_cast<OpHeader*>(ws);
  h->status = 0;
  h->magic = kOpMagic;
}

}  // namespace rar

using namespace rar;

namespace {

rar_status norm_rope_forward(const NormRopeCall& c, const void* const* qkv, int interleaved, float eps,
                             const int32_t* slots, void* const* q_out, int64_t q_stride, void* const* k_out,
                             int64_t k_stride, void* const* v_out, int num_pages, int page_size, void* ws,
                             size_t ws_bytes, void* stream) {
  const bool cache = v_out != nullptr;
  Spans s;
  rar_status st = check_norm_rope(c, qkv, &s);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(c.dtype), D = c.head_dim;
  const int64_t width = (c.q_heads + 2 * (int64_t)c.kv_heads) * D;
  if ((st = check_pointers((const void* const*)q_out, c.nranks, c.tokens, 16)) != RAR_OK) return st;
  if ((st = check_pointers((const void* const*)k_out, c.nranks, c.tokens, 16)) != RAR_OK) return st;
  if ((st = check_stride(q_stride, c.q_heads * D, c.tokens, es)) != RAR_OK) return st;
  int shift = 0;
  if (cache) {
    if ((st = check_pointers((const void* const*)v_out, c.nranks, c.tokens, 16)) != RAR_OK) return st;
    shift = page_shift_of(page_size);
    if (shift < 0 || !pages_ok(num_pages, shift, c.kv_heads) || (slots == nullptr && c.tokens > 0)) return RAR_ERR_ARG;
    if (!aligned(slots, 4)) return RAR_ERR_ALIGN;
    s.read(span(slots, c.tokens * 4));
  } else if ((st = check_stride(k_stride, c.kv_heads * D, c.tokens, es)) != RAR_OK) {
    return st;
  }
  // queries may be turned in place: q_out[r] == qkv[r] with one stride
  for (int r = 0; r < c.nranks; r++) {
    const bool in_place = q_out[r] == qkv[r] && (c.tokens <= 1 || q_stride == c.qkv_stride);
    const int64_t skip = in_place ? c.q_heads * D * es : 0;
    s.read(span((const char*)qkv[r] + skip, c.tokens, width * es - skip, c.qkv_stride * es));
    s.write(span(q_out[r], c.tokens, c.q_heads * D * es, q_stride * es));
    if (cache) {
      const int64_t bytes = ((int64_t)num_pages << shift) * c.kv_heads * D * es;
      s.write(span(k_out[r], bytes));
      s.write(span(v_out[r], bytes));
    } else {
      s.write(span(k_out[r], c.tokens, c.kv_heads * D * es, k_stride * es));
    }
  }
  s.write(span(ws, (int64_t)ws_bytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(ws, ws_bytes, 0)) != RAR_OK) return st;
  if (c.tokens == 0) return RAR_OK;
  NormRopeArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < c.nranks; r++) {
    a.qkv[r] = qkv[r];
    a.q_out[r] = q_out[r];
    a.k_out[r] = k_out[r];
    a.v_out[r] = cache ? v_out[r] : nullptr;
  }
  a.q_weight = c.q_weight;
  a.k_weight = c.k_weight;
  a.cos_sin = c.cos_sin;
  a.positions = c.positions;
  a.slots = cache ? slots : nullptr;
  a.ws = (char*)ws;
  a.qkv_stride = c.qkv_stride;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.num_slots = (int64_t)num_pages << shift;
  a.eps = eps;
  a.tokens = (int)c.tokens;
  a.nranks = c.nranks;
  a.dtype = (int)c.dtype;
  a.q_heads = c.q_heads;
  a.kv_heads = c.kv_heads;
  a.head_dim = c.head_dim;
  a.rot = c.rot_dim;
  a.max_pos = c.max_pos;
  a.interleaved = interleaved != 0;
  a.page_shift = shift;
  return from_cuda(launch_norm_rope(a, (cudaStream_t)stream));
}

// Sizes that the forms of the attention over prompts share.
bool prompt_sizes_ok(int64_t tokens, int q_heads, int kv_heads, int head_dim) {
  return heads_ok(q_heads, kv_heads, head_dim) && q_heads % kv_heads == 0 && tokens >= 0 &&
         tokens <= INT32_MAX / q_heads;
}
rar_status check_prompt(int nranks, int64_t tokens, int q_heads, int kv_heads, int head_dim, rar_dtype dtype,
                        const int32_t* starts, int sequences, Spans* s) {
  const rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  if (!prompt_sizes_ok(tokens, q_heads, kv_heads, head_dim) || sequences < 0) return RAR_ERR_ARG;
  // blocks of a launch: a tile of 32 rows or more each, and one for every sequence and key head
  if ((int64_t)sequences > INT32_MAX / 2 / ((int64_t)kv_heads * nranks)) return RAR_ERR_ARG;
  if (starts == nullptr && sequences > 0) return RAR_ERR_ARG;
  if (!aligned(starts, 4)) return RAR_ERR_ALIGN;
  s->read(span(starts, sequences > 0 ? ((int64_t)sequences + 1) * 4 : 0));
  return RAR_OK;
}
// Rows [tokens, heads, head_dim] of each rank: elements from token to token, and from head to head.
struct Rows {
  const void* const* data;
  int64_t stride, head;
};
// A token's heads may lie within its row, or the tokens within a head's; either way no two rows of head_dim share an element.
rar_status check_rows(const Rows& x, int nranks, int64_t tokens, int heads, int head_dim, int64_t es, bool out, Spans* s) {
  rar_status st = check_pointers(x.data, nranks, tokens, 16);
  if (st != RAR_OK) return st;
  const int64_t most = INT64_MAX / 32, D = head_dim;
  if (x.stride < 0 || x.head < 0 || x.stride > most / (tokens > 0 ? tokens : 1) || x.head > most / heads) return RAR_ERR_ARG;
  const int64_t of_token = (heads - 1) * x.head + D, of_head = (tokens - 1) * x.stride + D;  // a row's elements, with gaps
  const bool by_token = (heads < 2 || x.head >= D) && (tokens < 2 || x.stride >= of_token);
  const bool by_head = heads > 1 && tokens > 1 && x.stride >= D && x.head >= of_head;
  if (!by_token && !by_head) return RAR_ERR_ARG;
  if (x.stride * es % 16 != 0 || x.head * es % 16 != 0) return RAR_ERR_ALIGN;
  for (int r = 0; r < nranks && tokens > 0; r++) {
    Span y = by_token ? span(x.data[r], tokens, of_token * es, x.stride * es) : span(x.data[r], heads, of_head * es, x.head * es);
    // a head's rows of other tensors may lie between these
    if (by_token && heads > 1 && (tokens < 2 || x.stride % x.head == 0)) y.part = D * es, y.every = x.head * es;
    if (!by_token && x.head % x.stride == 0) y.part = D * es, y.every = x.stride * es;
    if (out) s->write(y);
    else s->read(y);
  }
  return RAR_OK;
}

rar_status prompt_forward(PromptArgs& a, void* const* out, float* const* lse, size_t ws_bytes, Spans& s) {
  const Rows rows = {(const void* const*)out, a.out_stride, a.out_head};
  rar_status st = check_rows(rows, a.nranks, a.tokens, a.q_heads, a.head_dim, size_of((rar_dtype)a.dtype), true, &s);
  if (st != RAR_OK) return st;
  if (lse != nullptr) {
    if ((st = check_pointers((const void* const*)lse, a.nranks, a.tokens, 4)) != RAR_OK) return st;
    for (int r = 0; r < a.nranks; r++) s.write(span(lse[r], (int64_t)a.tokens * a.q_heads * 4));
  }
  s.write(span(a.ws, (int64_t)ws_bytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(a.ws, ws_bytes,
                            prompt_attention_scratch_bytes(a.nranks, a.tokens, a.q_heads, a.kv_heads, a.head_dim))) != RAR_OK)
    return st;
  if (a.tokens == 0 || a.sequences == 0) return RAR_OK;
  for (int r = 0; r < a.nranks; r++) {
    a.out[r] = out[r];
    a.lse[r] = lse != nullptr ? lse[r] : nullptr;
  }
  return RAR_OK;
}

// Vocabulary shards of rows: the first word of each, and their spans.
rar_status check_tables(const void* const* tables, const int64_t* vocab, const int64_t* strides, int nranks, int hidden,
                        int64_t es, bool out, int64_t* first, Spans* s) {
  if (vocab == nullptr || strides == nullptr || hidden < 8 || hidden > 1 << 20 || hidden % 8 != 0) return RAR_ERR_ARG;
  rar_status st = check_pointers(tables, nranks, 1, 16);
  if (st != RAR_OK) return st;
  first[0] = 0;
  for (int r = 0; r < nranks; r++) {
    if (vocab[r] < 1 || vocab[r] > INT32_MAX) return RAR_ERR_ARG;
    if ((st = check_stride(strides[r], hidden, vocab[r], es)) != RAR_OK) return st;
    first[r + 1] = first[r] + vocab[r];
    const Span x = span(tables[r], vocab[r], hidden * es, strides[r] * es);
    if (out) s->write(x);
    else s->read(x);
  }
  return first[nranks] <= INT32_MAX ? RAR_OK : RAR_ERR_ARG;
}
bool embed_sizes_ok(int64_t tokens, int hidden) {
  return hidden >= 8 && hidden <= 1 << 20 && hidden % 8 == 0 && tokens >= 0 && tokens <= INT32_MAX / div_up(hidden, 256);
}

}  // namespace

extern "C" {

rar_status rar_op_workspace_init(void* workspace, size_t workspaceBytes, void* stream) {
  const rar_status st = check_workspace(workspace, workspaceBytes, 0);
  if (st != RAR_OK) return st;
  const cudaError_t e = cudaMemsetAsync(workspace, 0, (size_t)kOpScratchOffset, (cudaStream_t)stream);
  if (e != cudaSuccess) return from_cuda(e);
  init_op_header_kernel<<<1, 1, 0, (cudaStream_t)stream>>>((char*)workspace);
  return from_cuda(cudaGetLastError());
}

rar_status rar_page_tables(const int32_t* lens, const int32_t* new_tokens, int num_requests, const int32_t* free_pages,
                           int num_free, const int32_t* free_count, int page_size, int num_pages, int32_t* block_table,
                           int64_t table_stride, int max_blocks, int32_t* lens_out, int32_t* starts,
                           int32_t* positions, int32_t* slots, int max_tokens, int32_t* free_count_out, void* workspace,
                           size_t workspaceBytes, void* stream) {
  const int shift = page_shift_of(page_size);
  if (num_requests < 0 || num_free < 0 || max_tokens < 0 || max_blocks < 1 || shift < 0 || !pages_ok(num_pages, shift, 1))
    return RAR_ERR_ARG;
  if (num_requests > 1 && table_stride < max_blocks) return RAR_ERR_ARG;
  if (table_stride < 0 || table_stride > INT64_MAX / 8 / (num_requests > 0 ? num_requests : 1)) return RAR_ERR_ARG;
  if ((int64_t)max_blocks << shift > INT32_MAX) return RAR_ERR_ARG;
  if (free_count == nullptr || free_count_out == nullptr || starts == nullptr) return RAR_ERR_ARG;
  if (num_requests > 0 && (lens == nullptr || new_tokens == nullptr || block_table == nullptr || lens_out == nullptr))
    return RAR_ERR_ARG;
  if (num_free > 0 && free_pages == nullptr) return RAR_ERR_ARG;
  if (max_tokens > 0 && (positions == nullptr || slots == nullptr)) return RAR_ERR_ARG;
  const void* all[] = {lens,   new_tokens, free_pages, free_count, block_table, lens_out,
                       starts, positions,  slots,      free_count_out};
  for (const void* p : all)
    if (!aligned(p, 4)) return RAR_ERR_ALIGN;
  Spans s;
  s.read(span(lens, (int64_t)num_requests * 4));
  s.read(span(new_tokens, (int64_t)num_requests * 4));
  s.read(span(free_pages, (int64_t)num_free * 4));
  s.read(span(free_count, 4));
  s.write(span(block_table, num_requests, (int64_t)max_blocks * 4, table_stride * 4));
  s.write(span(lens_out, (int64_t)num_requests * 4));
  s.write(span(starts, ((int64_t)num_requests + 1) * 4));
  s.write(span(positions, (int64_t)max_tokens * 4));
  s.write(span(slots, (int64_t)max_tokens * 4));
  s.write(span(free_count_out, 4));
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  const rar_status st = check_workspace(workspace, workspaceBytes, 0);
  if (st != RAR_OK) return st;
  PageTablesArgs a = {};
  a.lens = lens;
  a.new_tokens = new_tokens;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens_out = lens_out;
  a.starts = starts;
  a.positions = positions;
  a.slots = slots;
  a.free_count_out = free_count_out;
  a.ws = (char*)workspace;
  a.requests = num_requests;
  a.num_free = num_free;
  a.page_shift = shift;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  a.max_tokens = max_tokens;
  return from_cuda(launch_page_tables(a, (cudaStream_t)stream));
}

rar_status rar_qk_norm_rope(const void* const* qkv, int nranks, int64_t tokens, int64_t qkv_stride,
                            const void* q_weight, const void* k_weight, const float* cos_sin, int max_pos, int rot_dim,
                            int interleaved, const int32_t* positions, int q_heads, int kv_heads, int head_dim,
                            rar_dtype dtype, float eps, void* const* q_out, int64_t q_stride, void* const* k_out,
                            int64_t k_stride, void* workspace, size_t workspaceBytes, void* stream) {
  const NormRopeCall c = {nranks,  tokens,  qkv_stride, q_weight, k_weight, cos_sin, max_pos,
                          rot_dim, positions, q_heads,  kv_heads, head_dim, dtype};
  return norm_rope_forward(c, qkv, interleaved, eps, nullptr, q_out, q_stride, k_out, k_stride, nullptr, 1, 1, workspace,
                           workspaceBytes, stream);
}

rar_status rar_qk_norm_rope_cached(const void* const* qkv, int nranks, int64_t tokens, int64_t qkv_stride,
                                   const void* q_weight, const void* k_weight, const float* cos_sin, int max_pos,
                                   int rot_dim, int interleaved, const int32_t* positions, const int32_t* slots,
                                   int q_heads, int kv_heads, int head_dim, rar_dtype dtype, float eps,
                                   void* const* q_out, int64_t q_stride, void* const* k_cache, void* const* v_cache,
                                   int num_pages, int page_size, void* workspace, size_t workspaceBytes,
                                   void* stream) {
  if (v_cache == nullptr) return RAR_ERR_ARG;
  const NormRopeCall c = {nranks,  tokens,  qkv_stride, q_weight, k_weight, cos_sin, max_pos,
                          rot_dim, positions, q_heads,  kv_heads, head_dim, dtype};
  return norm_rope_forward(c, qkv, interleaved, eps, slots, q_out, q_stride, k_cache, 0, v_cache, num_pages, page_size,
                           workspace, workspaceBytes, stream);
}

size_t rar_qk_norm_rope_workspace_bytes(int nranks, int head_dim) {
  if (nranks < 1 || nranks > kMaxRanks || !heads_ok(1, 1, head_dim)) return 0;
  return (size_t)(kOpScratchOffset + norm_rope_scratch_bytes(nranks, head_dim));
}

rar_status rar_qk_norm_rope_backward(const void* const* qkv, int nranks, int64_t tokens, int64_t qkv_stride,
                                     const void* q_weight, const void* k_weight, const float* cos_sin, int max_pos,
                                     int rot_dim, int interleaved, const int32_t* positions, int q_heads, int kv_heads,
                                     int head_dim, rar_dtype dtype, float eps, const void* const* dq,
                                     int64_t dq_stride, const void* const* dk, int64_t dk_stride,
                                     const void* const* dv, int64_t dv_stride, void* const* dqkv, int64_t dqkv_stride,
                                     float* const* dq_weight, float* const* dk_weight, void* workspace,
                                     size_t workspaceBytes, void* stream) {
  const NormRopeCall c = {nranks,  tokens,  qkv_stride, q_weight, k_weight, cos_sin, max_pos,
                          rot_dim, positions, q_heads,  kv_heads, head_dim, dtype};
  Spans s;
  rar_status st = check_norm_rope(c, qkv, &s);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype), D = head_dim, heads = q_heads + 2 * (int64_t)kv_heads;
  if ((st = check_pointers(dq, nranks, tokens, 16)) != RAR_OK || (st = check_pointers(dk, nranks, tokens, 16)) != RAR_OK ||
      (st = check_pointers(dv, nranks, tokens, 16)) != RAR_OK ||
      (st = check_pointers((const void* const*)dqkv, nranks, tokens, 16)) != RAR_OK ||
      (st = check_pointers((const void* const*)dq_weight, nranks, 1, 4)) != RAR_OK ||
      (st = check_pointers((const void* const*)dk_weight, nranks, 1, 4)) != RAR_OK)
    return st;
  if ((st = check_stride(dq_stride, q_heads * D, tokens, es)) != RAR_OK ||
      (st = check_stride(dk_stride, kv_heads * D, tokens, es)) != RAR_OK ||
      (st = check_stride(dv_stride, kv_heads * D, tokens, es)) != RAR_OK ||
      (st = check_stride(dqkv_stride, heads * D, tokens, es)) != RAR_OK)
    return st;
  for (int r = 0; r < nranks; r++) {
    s.read(span(qkv[r], tokens, heads * D * es, qkv_stride * es));
    s.read(span(dq[r], tokens, q_heads * D * es, dq_stride * es));
    s.read(span(dk[r], tokens, kv_heads * D * es, dk_stride * es));
    s.read(span(dv[r], tokens, kv_heads * D * es, dv_stride * es));
    s.write(span(dqkv[r], tokens, heads * D * es, dqkv_stride * es));
    s.write(span(dq_weight[r], D * 4));
    s.write(span(dk_weight[r], D * 4));
  }
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes, norm_rope_scratch_bytes(nranks, head_dim))) != RAR_OK) return st;
  NormRopeBwdArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < nranks; r++) {
    a.qkv[r] = qkv[r];
    a.dq[r] = dq[r];
    a.dk[r] = dk[r];
    a.dv[r] = dv[r];
    a.dqkv[r] = dqkv[r];
    a.dq_weight[r] = dq_weight[r];
    a.dk_weight[r] = dk_weight[r];
  }
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.cos_sin = cos_sin;
  a.positions = positions;
  a.ws = (char*)workspace;
  a.qkv_stride = qkv_stride;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.dv_stride = dv_stride;
  a.dqkv_stride = dqkv_stride;
  a.eps = eps;
  a.tokens = (int)tokens;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.rot = rot_dim;
  a.max_pos = max_pos;
  a.interleaved = interleaved != 0;
  return from_cuda(launch_norm_rope_bwd(a, (cudaStream_t)stream));
}

size_t rar_decode_attention_workspace_bytes(int nranks, int batch, int q_heads, int kv_heads, int head_dim) {
  if (nranks < 1 || nranks > kMaxRanks || batch < 0 || !heads_ok(q_heads, kv_heads, head_dim) ||
      q_heads % kv_heads != 0)
    return 0;
  return (size_t)(kOpScratchOffset + decode_attention_scratch_bytes(q_heads, kv_heads, head_dim));
}

rar_status rar_decode_attention(const void* const* q, int64_t q_stride, const void* const* k_cache,
                                const void* const* v_cache, int nranks, int batch, int q_heads, int kv_heads,
                                int head_dim, rar_dtype dtype, int num_pages, int page_size,
                                const int32_t* block_table, int64_t table_stride, int max_blocks, const int32_t* lens,
                                float scale, void* const* out, int64_t out_stride, float* const* lse, void* workspace,
                                size_t workspaceBytes, void* stream) {
  rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  const int shift = page_shift_of(page_size);
  const int64_t es = size_of(dtype), D = head_dim;
  if (!heads_ok(q_heads, kv_heads, head_dim) || q_heads % kv_heads != 0) return RAR_ERR_ARG;
  if (batch < 0 || shift < 0 || !pages_ok(num_pages, shift, kv_heads) || max_blocks < 1) return RAR_ERR_ARG;
  if ((int64_t)max_blocks << shift > INT32_MAX) return RAR_ERR_ARG;
  if (batch > 1 && table_stride < max_blocks) return RAR_ERR_ARG;
  if (table_stride < 0 || table_stride > INT64_MAX / 8 / (batch > 0 ? batch : 1)) return RAR_ERR_ARG;
  if ((st = check_pointers(q, nranks, batch, 16)) != RAR_OK || (st = check_pointers(k_cache, nranks, batch, 16)) != RAR_OK ||
      (st = check_pointers(v_cache, nranks, batch, 16)) != RAR_OK ||
      (st = check_pointers((const void* const*)out, nranks, batch, 16)) != RAR_OK)
    return st;
  if (lse != nullptr && (st = check_pointers((const void* const*)lse, nranks, batch, 4)) != RAR_OK) return st;
  if (batch > 0 && (block_table == nullptr || lens == nullptr)) return RAR_ERR_ARG;
  if (!aligned(block_table, 4) || !aligned(lens, 4)) return RAR_ERR_ALIGN;
  if ((st = check_stride(q_stride, q_heads * D, batch, es)) != RAR_OK ||
      (st = check_stride(out_stride, q_heads * D, batch, es)) != RAR_OK)
    return st;
  Spans s;
  const int64_t cache = ((int64_t)num_pages << shift) * kv_heads * D * es;
  s.read(span(block_table, batch, (int64_t)max_blocks * 4, table_stride * 4));
  s.read(span(lens, (int64_t)batch * 4));
  for (int r = 0; r < nranks; r++) {
    s.read(span(q[r], batch, q_heads * D * es, q_stride * es));
    s.read(span(k_cache[r], cache));
    s.read(span(v_cache[r], cache));
    s.write(span(out[r], batch, q_heads * D * es, out_stride * es));
    if (lse != nullptr) s.write(span(lse[r], (int64_t)batch * q_heads * 4));
  }
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes,
                            decode_attention_scratch_bytes(q_heads, kv_heads, head_dim))) != RAR_OK)
    return st;
  if (batch == 0) return RAR_OK;
  DecodeArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < nranks; r++) {
    a.q[r] = q[r];
    a.k_cache[r] = k_cache[r];
    a.v_cache[r] = v_cache[r];
    a.out[r] = out[r];
    a.lse[r] = lse != nullptr ? lse[r] : nullptr;
  }
  a.table = block_table;
  a.lens = lens;
  a.ws = (char*)workspace;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.table_stride = table_stride;
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.batch = batch;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.page_shift = shift;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  return from_cuda(launch_decode_attention(a, (cudaStream_t)stream));
}

size_t rar_token_logprobs_workspace_bytes(int64_t rows, int top) {
  if (rows < 0 || rows > INT32_MAX || top < 0 || top > kMaxTop) return 0;
  return (size_t)(kOpScratchOffset + token_logprobs_scratch_bytes());
}

rar_status rar_token_logprobs(const void* const* logits, const int64_t* vocab, const int64_t* row_strides, int nranks,
                              int64_t rows, rar_dtype dtype, const int32_t* tokens, float* logprob, float* entropy,
                              float* lse, int top, float* top_values, int32_t* top_ids, void* workspace,
                              size_t workspaceBytes, void* stream) {
  rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype);
  if (rows < 0 || rows > INT32_MAX || top < 0 || top > kMaxTop || vocab == nullptr || row_strides == nullptr)
    return RAR_ERR_ARG;
  if ((st = check_pointers(logits, nranks, rows, (uintptr_t)es)) != RAR_OK) return st;
  LogprobArgs a;
  std::memset(&a, 0, sizeof a);
  Spans s;
  int64_t tiles = 0;  // of a row
  for (int r = 0; r < nranks; r++) {
    if (vocab[r] < 1 || vocab[r] > INT32_MAX) return RAR_ERR_ARG;
    if (rows > 1 && row_strides[r] < vocab[r]) return RAR_ERR_ARG;
    if (row_strides[r] < 0 || row_strides[r] > INT64_MAX / 8 / (rows > 0 ? rows : 1)) return RAR_ERR_ARG;
    a.logits[r] = logits[r];
    a.row_stride[r] = row_strides[r];
    a.first[r + 1] = a.first[r] + vocab[r];
    tiles += div_up(vocab[r], kLpTile);
    s.read(span(logits[r], rows, vocab[r] * es, row_strides[r] * es));
  }
  if (a.first[nranks] > INT32_MAX || top > a.first[nranks] || rows * tiles > INT32_MAX) return RAR_ERR_ARG;
  if (rows > 0 && (tokens == nullptr || logprob == nullptr || entropy == nullptr || lse == nullptr)) return RAR_ERR_ARG;
  if (rows > 0 && top > 0 && (top_values == nullptr || top_ids == nullptr)) return RAR_ERR_ARG;
  const void* all[] = {tokens, logprob, entropy, lse, top_values, top_ids};
  for (const void* p : all)
    if (!aligned(p, 4)) return RAR_ERR_ALIGN;
  s.read(span(tokens, rows * 4));
  s.write(span(logprob, rows * 4));
  s.write(span(entropy, rows * 4));
  s.write(span(lse, rows * 4));
  s.write(span(top_values, rows * top * 4));
  s.write(span(top_ids, rows * top * 4));
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes, token_logprobs_scratch_bytes())) != RAR_OK)
    return st;
  if (rows == 0) return RAR_OK;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_values = top_values;
  a.top_ids = top_ids;
  a.ws = (char*)workspace;
  a.rows = (int)rows;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.top = top;
  return from_cuda(launch_token_logprobs(a, (cudaStream_t)stream));
}

rar_status rar_token_logprobs_backward(const void* const* logits, const int64_t* vocab, const int64_t* row_strides,
                                       int nranks, int64_t rows, rar_dtype dtype, const int32_t* tokens,
                                       const float* lse, const float* entropy, const float* grad_logprob,
                                       const float* grad_entropy, void* const* dlogits,
                                       const int64_t* drow_strides, void* workspace, size_t workspaceBytes,
                                       void* stream) {
  rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype);
  if (rows < 0 || rows > INT32_MAX || vocab == nullptr || row_strides == nullptr || drow_strides == nullptr)
    return RAR_ERR_ARG;
  if ((st = check_pointers(logits, nranks, rows, (uintptr_t)es)) != RAR_OK ||
      (st = check_pointers((const void* const*)dlogits, nranks, rows, (uintptr_t)es)) != RAR_OK)
    return st;
  LogprobBwdArgs a;
  std::memset(&a, 0, sizeof a);
  Spans s;
  for (int r = 0; r < nranks; r++) {
    if (vocab[r] < 1 || vocab[r] > INT32_MAX) return RAR_ERR_ARG;
    if (rows > 1 && (row_strides[r] < vocab[r] || drow_strides[r] < vocab[r])) return RAR_ERR_ARG;
    const int64_t most = INT64_MAX / 8 / (rows > 0 ? rows : 1);
    if (row_strides[r] < 0 || row_strides[r] > most || drow_strides[r] < 0 || drow_strides[r] > most)
      return RAR_ERR_ARG;
    a.logits[r] = logits[r];
    a.dlogits[r] = dlogits[r];
    a.row_stride[r] = row_strides[r];
    a.drow_stride[r] = drow_strides[r];
    a.first[r + 1] = a.first[r] + vocab[r];
    // in place is allowed: dlogits[r] == logits[r] with one stride
    if (dlogits[r] != logits[r] || (rows > 1 && drow_strides[r] != row_strides[r]))
      s.read(span(logits[r], rows, vocab[r] * es, row_strides[r] * es));
    s.write(span(dlogits[r], rows, vocab[r] * es, drow_strides[r] * es));
  }
  if (a.first[nranks] > INT32_MAX) return RAR_ERR_ARG;
  if (rows > 0 && (tokens == nullptr || lse == nullptr || entropy == nullptr || grad_logprob == nullptr))
    return RAR_ERR_ARG;
  const void* all[] = {tokens, lse, entropy, grad_logprob, grad_entropy};
  for (const void* p : all) {
    if (!aligned(p, 4)) return RAR_ERR_ALIGN;
    s.read(span(p, rows * 4));
  }
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes, 0)) != RAR_OK) return st;
  if (rows == 0) return RAR_OK;
  a.tokens = tokens;
  a.lse = lse;
  a.entropy = entropy;
  a.grad_logprob = grad_logprob;
  a.grad_entropy = grad_entropy;
  a.ws = (char*)workspace;
  a.rows = (int)rows;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  return from_cuda(launch_token_logprobs_bwd(a, (cudaStream_t)stream));
}

size_t rar_prompt_attention_workspace_bytes(int nranks, int64_t tokens, int q_heads, int kv_heads, int head_dim) {
  if (nranks < 1 || nranks > kMaxRanks || !prompt_sizes_ok(tokens, q_heads, kv_heads, head_dim)) return 0;
  return (size_t)(kOpScratchOffset + prompt_attention_scratch_bytes(nranks, tokens, q_heads, kv_heads, head_dim));
}

rar_status rar_prompt_attention_ex(const void* const* q, int64_t q_stride, int64_t q_head_stride, const void* const* k,
                                   int64_t k_stride, int64_t k_head_stride, const void* const* v, int64_t v_stride,
                                   int64_t v_head_stride, int nranks, int64_t tokens, int q_heads, int kv_heads, int head_dim,
                                   rar_dtype dtype, const int32_t* starts, int num_sequences, float scale, void* const* out,
                                   int64_t out_stride, int64_t out_head_stride, float* const* lse, void* workspace,
                                   size_t workspaceBytes, void* stream) {
  Spans s;
  rar_status st = check_prompt(nranks, tokens, q_heads, kv_heads, head_dim, dtype, starts, num_sequences, &s);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype);
  if ((st = check_rows({q, q_stride, q_head_stride}, nranks, tokens, q_heads, head_dim, es, false, &s)) != RAR_OK ||
      (st = check_rows({k, k_stride, k_head_stride}, nranks, tokens, kv_heads, head_dim, es, false, &s)) != RAR_OK ||
      (st = check_rows({v, v_stride, v_head_stride}, nranks, tokens, kv_heads, head_dim, es, false, &s)) != RAR_OK)
    return st;
  PromptArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < nranks; r++) {
    a.q[r] = q[r];
    a.k[r] = k[r];
    a.v[r] = v[r];
  }
  a.starts = starts;
  a.ws = (char*)workspace;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out_stride = out_stride;
  a.q_head = q_head_stride;
  a.k_head = k_head_stride;
  a.v_head = v_head_stride;
  a.out_head = out_head_stride;
  a.wait_ns = spin_timeout_ns();
  a.fault = debug_fault();
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.tokens = (int)tokens;
  a.sequences = num_sequences;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  if ((st = prompt_forward(a, out, lse, workspaceBytes, s)) != RAR_OK || tokens == 0 || num_sequences == 0) return st;
  return from_cuda(launch_prompt_attention(a, (cudaStream_t)stream));
}

rar_status rar_prompt_attention(const void* const* q, int64_t q_stride, const void* const* k, int64_t k_stride,
                                const void* const* v, int64_t v_stride, int nranks, int64_t tokens, int q_heads,
                                int kv_heads, int head_dim, rar_dtype dtype, const int32_t* starts, int num_sequences,
                                float scale, void* const* out, int64_t out_stride, float* const* lse, void* workspace,
                                size_t workspaceBytes, void* stream) {
  return rar_prompt_attention_ex(q, q_stride, head_dim, k, k_stride, head_dim, v, v_stride, head_dim, nranks, tokens, q_heads,
                                 kv_heads, head_dim, dtype, starts, num_sequences, scale, out, out_stride, head_dim, lse,
                                 workspace, workspaceBytes, stream);
}

rar_status rar_prompt_attention_cached_ex(const void* const* q, int64_t q_stride, int64_t q_head_stride,
                                          const void* const* k_cache, const void* const* v_cache, int nranks, int64_t tokens,
                                          int q_heads, int kv_heads, int head_dim, rar_dtype dtype, int num_pages,
                                          int page_size, const int32_t* block_table, int64_t table_stride, int max_blocks,
                                          const int32_t* starts, const int32_t* lens, int num_sequences, float scale,
                                          void* const* out, int64_t out_stride, int64_t out_head_stride, float* const* lse,
                                          void* workspace, size_t workspaceBytes, void* stream) {
  Spans s;
  rar_status st = check_prompt(nranks, tokens, q_heads, kv_heads, head_dim, dtype, starts, num_sequences, &s);
  if (st != RAR_OK) return st;
  const int shift = page_shift_of(page_size);
  const int64_t es = size_of(dtype), D = head_dim, n = num_sequences;
  if (shift < 0 || !pages_ok(num_pages, shift, kv_heads) || max_blocks < 1 || (int64_t)max_blocks << shift > INT32_MAX)
    return RAR_ERR_ARG;
  if ((n > 1 && table_stride < max_blocks) || table_stride < 0 || table_stride > INT64_MAX / 8 / (n > 0 ? n : 1))
    return RAR_ERR_ARG;
  if ((st = check_rows({q, q_stride, q_head_stride}, nranks, tokens, q_heads, head_dim, es, false, &s)) != RAR_OK ||
      (st = check_pointers(k_cache, nranks, tokens, 16)) != RAR_OK ||
      (st = check_pointers(v_cache, nranks, tokens, 16)) != RAR_OK)
    return st;
  if (n > 0 && (block_table == nullptr || lens == nullptr)) return RAR_ERR_ARG;
  if (!aligned(block_table, 4) || !aligned(lens, 4)) return RAR_ERR_ALIGN;
  s.read(span(block_table, n, (int64_t)max_blocks * 4, table_stride * 4));
  s.read(span(lens, n * 4));
  PromptArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < nranks; r++) {
    const int64_t cache = ((int64_t)num_pages << shift) * kv_heads * D * es;
    s.read(span(k_cache[r], cache));
    s.read(span(v_cache[r], cache));
    a.q[r] = q[r];
    a.k[r] = k_cache[r];
    a.v[r] = v_cache[r];
  }
  a.starts = starts;
  a.lens = lens;
  a.table = block_table;
  a.ws = (char*)workspace;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.q_head = q_head_stride;
  a.out_head = out_head_stride;
  a.table_stride = table_stride;
  a.wait_ns = spin_timeout_ns();
  a.fault = debug_fault();
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.tokens = (int)tokens;
  a.sequences = num_sequences;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.page_shift = shift;
  a.num_pages = num_pages;
  a.max_blocks = max_blocks;
  if ((st = prompt_forward(a, out, lse, workspaceBytes, s)) != RAR_OK || tokens == 0 || n == 0) return st;
  return from_cuda(launch_prompt_attention(a, (cudaStream_t)stream));
}

rar_status rar_prompt_attention_cached(const void* const* q, int64_t q_stride, const void* const* k_cache,
                                       const void* const* v_cache, int nranks, int64_t tokens, int q_heads, int kv_heads,
                                       int head_dim, rar_dtype dtype, int num_pages, int page_size,
                                       const int32_t* block_table, int64_t table_stride, int max_blocks,
                                       const int32_t* starts, const int32_t* lens, int num_sequences, float scale,
                                       void* const* out, int64_t out_stride, float* const* lse, void* workspace,
                                       size_t workspaceBytes, void* stream) {
  return rar_prompt_attention_cached_ex(q, q_stride, head_dim, k_cache, v_cache, nranks, tokens, q_heads, kv_heads, head_dim,
                                        dtype, num_pages, page_size, block_table, table_stride, max_blocks, starts, lens,
                                        num_sequences, scale, out, out_stride, head_dim, lse, workspace, workspaceBytes, stream);
}

rar_status rar_prompt_attention_backward_ex(const void* const* q, int64_t q_stride, int64_t q_head_stride,
                                            const void* const* k, int64_t k_stride, int64_t k_head_stride,
                                            const void* const* v, int64_t v_stride, int64_t v_head_stride, int nranks,
                                            int64_t tokens, int q_heads, int kv_heads, int head_dim, rar_dtype dtype,
                                            const int32_t* starts, int num_sequences, float scale, const void* const* out,
                                            int64_t out_stride, int64_t out_head_stride, const float* const* lse,
                                            const void* const* dout, int64_t dout_stride, int64_t dout_head_stride,
                                            void* const* dq, int64_t dq_stride, int64_t dq_head_stride, void* const* dk,
                                            int64_t dk_stride, int64_t dk_head_stride, void* const* dv, int64_t dv_stride,
                                            int64_t dv_head_stride, void* workspace, size_t workspaceBytes, void* stream) {
  Spans s;
  rar_status st = check_prompt(nranks, tokens, q_heads, kv_heads, head_dim, dtype, starts, num_sequences, &s);
  if (st != RAR_OK) return st;
  const Rows of_queries[] = {{q, q_stride, q_head_stride}, {out, out_stride, out_head_stride}, {dout, dout_stride, dout_head_stride},
                             {(const void* const*)dq, dq_stride, dq_head_stride}};
  const Rows of_keys[] = {{k, k_stride, k_head_stride}, {v, v_stride, v_head_stride},
                          {(const void* const*)dk, dk_stride, dk_head_stride}, {(const void* const*)dv, dv_stride, dv_head_stride}};
  for (int i = 0; i < 4; i++)
    if ((st = check_rows(of_queries[i], nranks, tokens, q_heads, head_dim, size_of(dtype), i == 3, &s)) != RAR_OK ||
        (st = check_rows(of_keys[i], nranks, tokens, kv_heads, head_dim, size_of(dtype), i >= 2, &s)) != RAR_OK)
      return st;
  if ((st = check_pointers((const void* const*)lse, nranks, tokens, 4)) != RAR_OK) return st;
  PromptBwdArgs a;
  std::memset(&a, 0, sizeof a);
  for (int r = 0; r < nranks; r++) {
    s.read(span(lse[r], tokens * q_heads * 4));
    a.q[r] = q[r];
    a.k[r] = k[r];
    a.v[r] = v[r];
    a.out[r] = out[r];
    a.dout[r] = dout[r];
    a.lse[r] = lse[r];
    a.dq[r] = dq[r];
    a.dk[r] = dk[r];
    a.dv[r] = dv[r];
  }
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes,
                            prompt_attention_scratch_bytes(nranks, tokens, q_heads, kv_heads, head_dim))) != RAR_OK)
    return st;
  if (tokens == 0 || num_sequences == 0) return RAR_OK;
  a.starts = starts;
  a.ws = (char*)workspace;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out_stride = out_stride;
  a.dout_stride = dout_stride;
  a.dq_stride = dq_stride;
  a.dk_stride = dk_stride;
  a.dv_stride = dv_stride;
  a.q_head = q_head_stride;
  a.k_head = k_head_stride;
  a.v_head = v_head_stride;
  a.out_head = out_head_stride;
  a.dout_head = dout_head_stride;
  a.dq_head = dq_head_stride;
  a.dk_head = dk_head_stride;
  a.dv_head = dv_head_stride;
  a.wait_ns = spin_timeout_ns();
  a.fault = debug_fault();
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.tokens = (int)tokens;
  a.sequences = num_sequences;
  a.q_heads = q_heads;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  return from_cuda(launch_prompt_attention_bwd(a, (cudaStream_t)stream));
}

rar_status rar_prompt_attention_backward(const void* const* q, int64_t q_stride, const void* const* k, int64_t k_stride,
                                         const void* const* v, int64_t v_stride, int nranks, int64_t tokens, int q_heads,
                                         int kv_heads, int head_dim, rar_dtype dtype, const int32_t* starts,
                                         int num_sequences, float scale, const void* const* out, int64_t out_stride,
                                         const float* const* lse, const void* const* dout, int64_t dout_stride,
                                         void* const* dq, int64_t dq_stride, void* const* dk, int64_t dk_stride,
                                         void* const* dv, int64_t dv_stride, void* workspace, size_t workspaceBytes,
                                         void* stream) {
  return rar_prompt_attention_backward_ex(q, q_stride, head_dim, k, k_stride, head_dim, v, v_stride, head_dim, nranks, tokens,
                                          q_heads, kv_heads, head_dim, dtype, starts, num_sequences, scale, out, out_stride,
                                          head_dim, lse, dout, dout_stride, head_dim, dq, dq_stride, head_dim, dk, dk_stride,
                                          head_dim, dv, dv_stride, head_dim, workspace, workspaceBytes, stream);
}

rar_status rar_embed_tokens(const int32_t* tokens, int64_t num_tokens, const void* const* tables, const int64_t* vocab,
                            const int64_t* row_strides, int nranks, int hidden, rar_dtype dtype, float scale, void* out,
                            int64_t out_stride, void* workspace, size_t workspaceBytes, void* stream) {
  rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype);
  if (!embed_sizes_ok(num_tokens, hidden)) return RAR_ERR_ARG;
  Spans s;
  EmbedArgs a;
  std::memset(&a, 0, sizeof a);
  if ((st = check_tables(tables, vocab, row_strides, nranks, hidden, es, false, a.first, &s)) != RAR_OK) return st;
  if (num_tokens > 0 && (tokens == nullptr || out == nullptr)) return RAR_ERR_ARG;
  if (!aligned(tokens, 4) || !aligned(out, 16)) return RAR_ERR_ALIGN;
  if ((st = check_stride(out_stride, hidden, num_tokens, es)) != RAR_OK) return st;
  s.read(span(tokens, num_tokens * 4));
  s.write(span(out, num_tokens, hidden * es, out_stride * es));
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes, 0)) != RAR_OK) return st;
  if (num_tokens == 0) return RAR_OK;
  for (int r = 0; r < nranks; r++) {
    a.tables[r] = tables[r];
    a.row_stride[r] = row_strides[r];
  }
  a.tokens_in = tokens;
  a.out = out;
  a.ws = (char*)workspace;
  a.tokens = num_tokens;
  a.out_stride = out_stride;
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.hidden = hidden;
  return from_cuda(launch_embed_tokens(a, (cudaStream_t)stream));
}

size_t rar_embed_tokens_workspace_bytes(int64_t num_tokens, int hidden) {
  if (!embed_sizes_ok(num_tokens, hidden)) return 0;
  return (size_t)(kOpScratchOffset + embed_tokens_scratch_bytes(num_tokens, hidden));
}

rar_status rar_embed_tokens_backward(const int32_t* tokens, int64_t num_tokens, const void* dout, int64_t dout_stride,
                                     rar_dtype dtype, float scale, float* const* dtables, const int64_t* vocab,
                                     const int64_t* drow_strides, int nranks, int hidden, int accumulate, void* workspace,
                                     size_t workspaceBytes, void* stream) {
  rar_status st = check_ranks(nranks, dtype);
  if (st != RAR_OK) return st;
  const int64_t es = size_of(dtype);
  if (!embed_sizes_ok(num_tokens, hidden)) return RAR_ERR_ARG;
  Spans s;
  EmbedBwdArgs a;
  std::memset(&a, 0, sizeof a);
  if ((st = check_tables((const void* const*)dtables, vocab, drow_strides, nranks, hidden, 4, true, a.first, &s)) != RAR_OK)
    return st;
  if (num_tokens > 0 && (tokens == nullptr || dout == nullptr)) return RAR_ERR_ARG;
  if (!aligned(tokens, 4) || !aligned(dout, 16)) return RAR_ERR_ALIGN;
  if ((st = check_stride(dout_stride, hidden, num_tokens, es)) != RAR_OK) return st;
  s.read(span(tokens, num_tokens * 4));
  s.read(span(dout, num_tokens, hidden * es, dout_stride * es));
  s.write(span(workspace, (int64_t)workspaceBytes));
  if (s.clash()) return RAR_ERR_ARG;
  if ((st = check_workspace(workspace, workspaceBytes, embed_tokens_scratch_bytes(num_tokens, hidden))) != RAR_OK) return st;
  for (int r = 0; r < nranks; r++) {
    a.dtables[r] = dtables[r];
    a.drow_stride[r] = drow_strides[r];
  }
  a.tokens_in = tokens;
  a.dout = dout;
  a.ws = (char*)workspace;
  a.tokens = num_tokens;
  a.dout_stride = dout_stride;
  a.scale = scale;
  a.nranks = nranks;
  a.dtype = (int)dtype;
  a.hidden = hidden;
  a.accumulate = accumulate != 0;
  return from_cuda(launch_embed_tokens_bwd(a, (cudaStream_t)stream));
}

}  // extern "C"
