// op_common.cuh -- what the operators around the collectives share: their
// workspace, their kernel arguments and a few device helpers.
//
// An operator runs all virtual ranks in one launch, as the collectives do: a
// rank's heads or vocabulary shard is one pointer of an array of nranks, and
// lengths, tables and positions are shared by all ranks.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "rar_device.cuh"

namespace rar {

// Workspace of the operators (device memory owned by the caller):
//   [0, 4096)        OpHeader (the status word where the ring header has it)
//   [4096, 36864)    arrival counters, zero between calls: the block or warp that
//                    arrives last at a join sets its counter back to zero
//   [36864, ...)     scratch of the call (partial results); nothing is kept
constexpr uint32_t kOpMagic = 0x31504f52u;  // "ROP1"
constexpr int kOpCounters = 8192;
constexpr int64_t kOpScratchOffset = kHeaderBytes + 4 * (int64_t)kOpCounters;

struct OpHeader {
  uint32_t magic;
  uint32_t status;  // first device failure (rar_status), 0 if none
};
static_assert(offsetof(OpHeader, status) == offsetof(WsHeader, status), "status word at one offset");

constexpr uint32_t kErrCapacity = 10;  // mirrors RAR_ERR_CAPACITY

__device__ __forceinline__ void op_report(char* ws, uint32_t code) {
  atomicCAS(&reinterpret_cast<OpHeader*>(ws)->status, 0u, code);
}
// Every thread of an operator's kernel starts here, before it reads or writes
// anything or returns: its blocks may be on the SMs before the kernel ahead of it
// in the stream has ended, and wait here until that one's results are there.
// Its own successor may then come up likewise. Returns the header's magic number,
// which kernels test before their first store: the load overlaps those of the inputs.
__device__ __forceinline__ uint32_t op_start(char* ws) {
  uint32_t v;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(&reinterpret_cast<OpHeader*>(ws)->magic));
  return v;
}
// True if the workspace was initialised; else the status word says so.
__device__ __forceinline__ bool op_ready(char* ws, uint32_t magic) {
  if (magic == kOpMagic) return true;
  if (threadIdx.x == 0) op_report(ws, kErrWorkspace);
  return false;
}

// Launches an operator's kernel, which begins with op_start: it may come up while
// the kernel ahead of it in the stream runs its last blocks. In rows of calls that
// takes about 2 us off each (attention of one short request 12.3 -> 10.4 us, log
// probabilities of 3 rows 13.6 -> 11.2, norm and rotation of 8192 tokens 66 -> 63.6).
inline cudaError_t launch_op(const void* fn, dim3 grid, int threads, int shared, cudaStream_t stream, void** params) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)shared;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, params);
}

// Returns the old value.
__device__ __forceinline__ uint32_t atom_add_acq_rel_u32(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// Two floats rounded to nearest even, a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Two binary32 values in a register pair, and two operations in one instruction.
struct F2 {
  uint64_t u;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.u));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
}

// Eight consecutive elements of a row, widened to binary32 (T: float or
// uint16_t holding bf16 bits; 16-byte aligned). load_stream: read once, past L1;
// absent: -inf in all eight; zero: 0.
template <typename T>
struct Pack8;
template <>
struct Pack8<uint16_t> {
  uint4 u;
  __device__ __forceinline__ void load(const uint16_t* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_stream(const uint16_t* p) { u = ld_stream_v4(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void absent() { u = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z); v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    u = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = u; }
};
template <>
struct Pack8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_stream(const float* p) {
    const uint4 u = ld_stream_v4(p), v = ld_stream_v4(p + 4);
    a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void absent() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void narrow(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ void from_float(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_float(uint16_t* p, float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  *p = *reinterpret_cast<const uint16_t*>(&b);
}
// Four consecutive elements, 16-byte (f32) or 8-byte (bf16) aligned.
__device__ __forceinline__ void store4(float* p, float x, float y, float z, float w) {
  *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}
__device__ __forceinline__ void store4(uint16_t* p, float x, float y, float z, float w) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(x, y), bf16_pair(z, w));
}

// ---- kernel arguments ----
struct PageTablesArgs {
  const int32_t* lens;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* table;
  int64_t table_stride;
  int32_t* lens_out;
  int32_t* starts;
  int32_t* positions;
  int32_t* slots;
  int32_t* free_count_out;
  char* ws;
  int requests, num_free, page_shift, num_pages, max_blocks, max_tokens;
};

struct NormRopeArgs {
  const void* qkv[kMaxRanks];
  void* q_out[kMaxRanks];
  void* k_out[kMaxRanks];  // dense keys, or the key cache if slots is set
  void* v_out[kMaxRanks];  // the value cache
  const void* q_weight;
  const void* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* slots;
  char* ws;
  int64_t qkv_stride, q_stride, k_stride;
  int64_t num_slots;
  float eps;
  int tokens, nranks, dtype, q_heads, kv_heads, head_dim, rot, max_pos, interleaved, page_shift;
};

struct NormRopeBwdArgs {
  const void* qkv[kMaxRanks];
  const void* dq[kMaxRanks];
  const void* dk[kMaxRanks];
  const void* dv[kMaxRanks];
  void* dqkv[kMaxRanks];
  float* dq_weight[kMaxRanks];
  float* dk_weight[kMaxRanks];
  const void* q_weight;
  const void* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  char* ws;
  int64_t qkv_stride, dq_stride, dk_stride, dv_stride, dqkv_stride;
  float eps;
  int tokens, nranks, dtype, q_heads, kv_heads, head_dim, rot, max_pos, interleaved;
};

struct DecodeArgs {
  const void* q[kMaxRanks];
  const void* k_cache[kMaxRanks];
  const void* v_cache[kMaxRanks];
  void* out[kMaxRanks];
  float* lse[kMaxRanks];  // null: not wanted
  const int32_t* table;
  const int32_t* lens;
  char* ws;
  int64_t q_stride, out_stride, table_stride;
  float scale;
  int nranks, dtype, batch, q_heads, kv_heads, head_dim, page_shift, num_pages, max_blocks;
};

struct LogprobArgs {
  const void* logits[kMaxRanks];
  int64_t row_stride[kMaxRanks];
  int64_t first[kMaxRanks + 1];  // vocabulary index of each shard's first column; the last entry is the total
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_values;
  int32_t* top_ids;
  char* ws;
  int rows, nranks, dtype, top;
  // set by the launcher: tiles before each shard's in a row, warps with work; parts of a row, or 0 and the units (of so
  // many tiles: 1, or a row's) of each warp and how many have one more
  int first_tile[kMaxRanks + 1];
  uint32_t workers, cuts, unit, each, more;
};

struct LogprobBwdArgs {
  const void* logits[kMaxRanks];
  void* dlogits[kMaxRanks];
  int64_t row_stride[kMaxRanks];
  int64_t drow_stride[kMaxRanks];
  int64_t first[kMaxRanks + 1];
  const int32_t* tokens;
  const float* lse;
  const float* entropy;
  const float* grad_logprob;
  const float* grad_entropy;  // null: no entropy term
  char* ws;
  int rows, nranks, dtype;
};

struct EmbedArgs {
  const void* tables[kMaxRanks];
  int64_t row_stride[kMaxRanks];
  int64_t first[kMaxRanks + 1];  // word of each shard's first row; the last entry is the total
  const int32_t* tokens_in;
  void* out;
  char* ws;
  int64_t tokens, out_stride;
  float scale;
  int nranks, dtype, hidden;
  int spans;  // set by the launcher: warps of a row
};

struct EmbedBwdArgs {
  float* dtables[kMaxRanks];
  int64_t drow_stride[kMaxRanks];
  int64_t first[kMaxRanks + 1];
  const int32_t* tokens_in;
  const void* dout;
  char* ws;
  int64_t tokens, dout_stride;
  float scale;
  int nranks, dtype, hidden, accumulate;
  // set by the launcher: pairs (word, token) in tiles and in one row, parts of sums; a tile's pairs, tiles, warps of a row
  uint64_t* sorted_tiles;
  uint64_t* sorted;
  float* parts;
  int64_t sum_blocks;  // blocks that sum; the warps of those behind them clear rows, so many each
  int64_t clear_first, clear_end;  // words up to which rows are cleared beside the sort, and beside the merge
  int tile, tiles, spans, clear_rows;
};
constexpr int kMaxTop = 32;
constexpr int kLpTile = 1024;  // columns of a tile of the log probabilities; a call's tiles are counted in 32 bits

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream);
cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);
cudaError_t launch_norm_rope_bwd(const NormRopeBwdArgs& a, cudaStream_t stream);
cudaError_t launch_decode_attention(const DecodeArgs& a, cudaStream_t stream);
cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream);
cudaError_t launch_token_logprobs_bwd(const LogprobBwdArgs& a, cudaStream_t stream);
cudaError_t launch_embed_tokens(EmbedArgs& a, cudaStream_t stream);  // fills in what the launcher sets
cudaError_t launch_embed_tokens_bwd(EmbedBwdArgs& a, cudaStream_t stream);

int64_t norm_rope_scratch_bytes(int nranks, int head_dim);
int64_t decode_attention_scratch_bytes(int q_heads, int kv_heads, int head_dim);
int64_t token_logprobs_scratch_bytes();
int64_t embed_tokens_scratch_bytes(int64_t tokens, int hidden);

}  // namespace rar
