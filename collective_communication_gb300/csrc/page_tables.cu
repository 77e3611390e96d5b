// page_tables.cu -- block tables and slot maps of a step, built on the GPU from
// the requests' lengths.
//
// have = ceil(len / P), need = ceil((len + new) / P) - have; off = exclusive
// sum of need, starts = exclusive sum of new over the requests. Page k handed
// out is free_pages[free_count - 1 - k]; request r takes pages off .. off+need.
// Token j of r sits at position len + j and slot table[r][pos / P] * P + pos % P.
//
// One launch without a second pass: every block computes the two prefix sums
// over all requests itself, kChunk requests at a time (8 bytes a request, from
// L2), and writes the part of the outputs that is its own: the tokens
// [b * kTokens, (b + 1) * kTokens), and the requests of every gridDim-th chunk.
// A token's page that is new in this call is read from the free list, not from
// the table that another block may still be writing. What bounds it is the
// launch and the chain of dependent loads; the bytes are a few MB at most.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kPtThreads = 1024;
constexpr int kPtPer = 4;                     // consecutive requests of a thread
constexpr int kPtChunk = kPtThreads * kPtPer;  // requests of a chunk
constexpr int kPtTokens = 2048;               // tokens of a block

namespace {

struct Sums {
  int64_t need, tokens;
};

// Exclusive prefix sum over the block's threads; `total` gets the sum of all.
__device__ __forceinline__ Sums block_exclusive(Sums mine, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums s = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = __shfl_up_sync(~0u, s.need, d), b = __shfl_up_sync(~0u, s.tokens, d);
    if (lane >= d) { s.need += a; s.tokens += b; }
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  Sums w = warp_sums[lane];  // kPtThreads / 32 == 32 warps
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = __shfl_up_sync(~0u, w.need, d), b = __shfl_up_sync(~0u, w.tokens, d);
    if (lane >= d) { w.need += a; w.tokens += b; }
  }
  total->need = __shfl_sync(~0u, w.need, 31);
  total->tokens = __shfl_sync(~0u, w.tokens, 31);
  const int64_t bn = __shfl_sync(~0u, w.need, warp == 0 ? 0 : warp - 1);
  const int64_t bt = __shfl_sync(~0u, w.tokens, warp == 0 ? 0 : warp - 1);
  s.need += (warp == 0 ? 0 : bn) - mine.need;
  s.tokens += (warp == 0 ? 0 : bt) - mine.tokens;
  return s;
}

__device__ __forceinline__ int32_t clamp_i32(int64_t v) { return (int32_t)(v < INT32_MAX ? v : INT32_MAX); }

}  // namespace

__global__ void __launch_bounds__(kPtThreads) page_tables_kernel(const __grid_constant__ PageTablesArgs a) {
  __shared__ Sums warp_sums[32];
  __shared__ int32_t s_start[kPtChunk];  // first token of the request, relative to the chunk's
  __shared__ int32_t s_off[kPtChunk];    // first page handed out to it; -1: the request gets nothing
  __shared__ int s_taken;
  const uint32_t magic = op_magic(a.ws);
  const int tid = threadIdx.x;
  const int P = 1 << a.page_shift;
  const int64_t width = (int64_t)a.max_blocks << a.page_shift;  // tokens that a table row can address
  const int64_t t0 = (int64_t)blockIdx.x * kPtTokens;
  const int64_t t1 = imin(t0 + kPtTokens, a.max_tokens);
  int count = *a.free_count;
  bool bad = count < 0 || count > a.num_free;
  count = count < 0 ? 0 : count > a.num_free ? a.num_free : count;
  if (!op_ready(a.ws, magic)) return;
  if (tid == 0) s_taken = 0;
  int64_t need0 = 0, tok0 = 0;  // sums over the chunks before this one
  const int chunks = (int)div_up(a.requests, kPtChunk);
  for (int c = 0; c < chunks; c++) {
    const int base = c * kPtChunk;
    int len[kPtPer], add[kPtPer], need[kPtPer];
    bool ok[kPtPer];
    Sums mine = {0, 0};
#pragma unroll
    for (int i = 0; i < kPtPer; i++) {
      const int r = base + tid * kPtPer + i;
      len[i] = r < a.requests ? a.lens[r] : 0;
      add[i] = r < a.requests ? a.new_tokens[r] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPtPer; i++) {
      ok[i] = len[i] >= 0 && add[i] >= 0 && (int64_t)len[i] + add[i] <= width;
      if (!ok[i]) { bad = true; add[i] = 0; }
      const int64_t have = ((int64_t)len[i] + P - 1) >> a.page_shift;
      need[i] = ok[i] ? (int)((((int64_t)len[i] + add[i] + P - 1) >> a.page_shift) - have) : 0;
      mine.need += need[i];
      mine.tokens += add[i];
    }
    Sums total;
    Sums at = block_exclusive(mine, warp_sums, &total);
    const bool my_requests = c % (int)gridDim.x == (int)blockIdx.x;
    int taken = 0;
#pragma unroll
    for (int i = 0; i < kPtPer; i++) {
      const int r = base + tid * kPtPer + i;
      const int64_t off = need0 + at.need, start = tok0 + at.tokens;
      // all or nothing: a request that does not fit whole gets no page and no slot
      const bool served = ok[i] && (need[i] == 0 || off + need[i] <= count) && start + add[i] <= a.max_tokens;
      if (!served && add[i] > 0) bad = true;
      if (served && need[i] > 0) taken = (int)(off + need[i]);
      s_start[tid * kPtPer + i] = clamp_i32(at.tokens);
      s_off[tid * kPtPer + i] = served ? (int)off : -1;
      if (my_requests && r < a.requests) {
        a.starts[r] = clamp_i32(start);
        a.lens_out[r] = served ? len[i] + add[i] : len[i];
        if (served) {
          const int have = (int)(((int64_t)len[i] + P - 1) >> a.page_shift);
          for (int k = 0; k < need[i]; k++) {
            const int page = a.free_pages[count - 1 - (off + k)];
            const bool fine = page >= 0 && page < a.num_pages;
            if (!fine) bad = true;
            a.table[(int64_t)r * a.table_stride + have + k] = fine ? page : -1;
          }
        }
      }
      at.need += need[i];
      at.tokens += add[i];
    }
    if (taken > 0) atomicMax(&s_taken, taken);
    __syncthreads();
    // the block's tokens that belong to this chunk
    const int64_t lo = t0 > tok0 ? t0 : tok0, hi = imin(t1, tok0 + total.tokens);
    for (int64_t t = lo + tid; t < hi; t += kPtThreads) {
      const int rel = (int)(t - tok0);
      int x = 0, y = kPtChunk;  // the last request whose first token is not after t
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (s_start[mid] <= rel) x = mid; else y = mid;
      }
      const int r = base + x;
      int slot = -1, pos = 0;
      if (r < a.requests && s_off[x] >= 0) {
        const int len_r = a.lens[r];
        pos = len_r + (rel - s_start[x]);
        const int have = (int)(((int64_t)len_r + P - 1) >> a.page_shift), col = pos >> a.page_shift;
        const int page = col < have ? a.table[(int64_t)r * a.table_stride + col]
                                    : a.free_pages[count - 1 - (s_off[x] + col - have)];
        if (page >= 0 && page < a.num_pages) slot = (page << a.page_shift) + (pos & (P - 1));
        else bad = true;
      }
      a.positions[t] = pos;
      a.slots[t] = slot;
    }
    need0 += total.need;
    tok0 += total.tokens;
    __syncthreads();  // s_start and s_off are written again
  }
  for (int64_t t = (t0 > tok0 ? t0 : tok0) + tid; t < t1; t += kPtThreads) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.starts[a.requests] = clamp_i32(tok0);
    *a.free_count_out = count - s_taken;
  }
  if (bad) op_report(a.ws, kErrCapacity);
}

cudaError_t launch_page_tables(const PageTablesArgs& a, cudaStream_t stream) {
  int64_t grid = div_up(a.max_tokens, kPtTokens);
  if (grid < 1) grid = 1;
  if (trace_on())
    std::fprintf(stderr, "rar trace: page_tables requests=%d tokens=%d page=%d grid=%lld threads=%d\n", a.requests,
                 a.max_tokens, 1 << a.page_shift, (long long)grid, kPtThreads);
  page_tables_kernel<<<(unsigned)grid, kPtThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rar
