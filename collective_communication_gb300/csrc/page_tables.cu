// page_tables.cu -- block tables and slot maps of a step, built on the GPU from
// the requests' lengths.
//
// have = ceil(len / P), need = ceil((len + new) / P) - have; off = exclusive
// sum of need, starts = exclusive sum of new over the requests. Page k handed
// out is free_pages[free_count - 1 - k]; request r takes pages off .. off+need.
// Token j of r sits at position len + j and slot table[r][pos / P] * P + pos % P.
//
// One launch without a second pass: every block computes the two prefix sums
// over all requests itself, a chunk of 4 requests a thread at a time (8 bytes a
// request, from L2), and writes its share of the outputs: a run of the tokens,
// and of every chunk's requests and new pages. (One block that wrote all
// requests' new pages, a dependent load and store each, took 23 us for 4096
// requests and 16000 pages; shared out it is 7.5.) A token's page that is new in
// this call is read from the free list, not from the table that another block
// may still be writing. What bounds it is the launch and the chain of dependent
// loads, so a thread's two tokens go through theirs side by side (7.5 us against
// 8.6 one after the other); the bytes are a few MB at most. Blocks of 256 threads for up to 1024
// requests, one chunk (3.1 us against 5.4 for 8 requests, where a larger block's
// start and barriers are what there is to save), of 1024 above (one pass over
// 4096 requests instead of four).
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kPtPer = 4;  // consecutive requests of a thread

namespace {

struct Sums {
  int64_t need, tokens;
};

// Exclusive prefix sum over the block's threads; `total` gets the sum of all.
template <int THREADS>
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
  Sums w = lane < THREADS / 32 ? warp_sums[lane] : Sums{0, 0};
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS) page_tables_kernel(const __grid_constant__ PageTablesArgs a) {
  constexpr int kChunk = THREADS * kPtPer, kTokens = 2 * THREADS;  // requests of a chunk, tokens of a block
  __shared__ Sums warp_sums[THREADS / 32];
  // of each request of the chunk, relative to the chunk: its first token; its first new page, with the bits
  // inverted (so below zero) if the request gets nothing
  __shared__ int32_t s_start[kChunk], s_off[kChunk];
  __shared__ int s_taken;
  const uint32_t magic = op_start(a.ws);
  const int tid = threadIdx.x;
  const int P = 1 << a.page_shift;
  const int64_t width = (int64_t)a.max_blocks << a.page_shift;  // tokens that a table row can address
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int64_t t1 = imin(t0 + kTokens, a.max_tokens);
  int count = *a.free_count;
  bool bad = count < 0 || count > a.num_free;
  count = count < 0 ? 0 : count > a.num_free ? a.num_free : count;
  if (!op_ready(a.ws, magic)) return;
  if (tid == 0) s_taken = 0;
  int64_t need0 = 0, tok0 = 0;  // sums over the chunks before this one
  const int chunks = (int)div_up(a.requests, kChunk);
  for (int c = 0; c < chunks; c++) {
    const int base = c * kChunk;
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
    Sums at = block_exclusive<THREADS>(mine, warp_sums, &total);
    // the block's share of the chunk's requests
    const int share = (kChunk + (int)gridDim.x - 1) / (int)gridDim.x;
    const int r0 = base + (int)blockIdx.x * share, r1 = min(min(r0 + share, base + kChunk), a.requests);
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
      s_off[tid * kPtPer + i] = served ? clamp_i32(at.need) : ~clamp_i32(at.need);
      if (r >= r0 && r < r1) {
        a.starts[r] = clamp_i32(start);
        a.lens_out[r] = served ? len[i] + add[i] : len[i];
      }
      at.need += need[i];
      at.tokens += add[i];
    }
    if (taken > 0) atomicMax(&s_taken, taken);
    __syncthreads();
    // The block's share of the chunk's new pages. The last request whose first page is not after p has page p.
    auto first_page = [&](int i) { return s_off[i] < 0 ? ~s_off[i] : s_off[i]; };
    const int64_t pages = imin(total.need, (int64_t)count - need0);  // those after it go to nobody
    const int64_t p1 = pages * (blockIdx.x + 1) / gridDim.x;
    for (int64_t p = pages * blockIdx.x / gridDim.x + tid; p < p1; p += THREADS) {
      int x = 0, y = kChunk;
      while (y - x > 1) {
        const int mid = (x + y) >> 1;
        if (first_page(mid) <= p) x = mid; else y = mid;
      }
      const int r = base + x;
      if (s_off[x] < 0) continue;
      const int have = (int)(((int64_t)a.lens[r] + P - 1) >> a.page_shift);
      const int page = a.free_pages[count - 1 - (need0 + p)];
      const bool fine = page >= 0 && page < a.num_pages;
      if (!fine) bad = true;
      a.table[(int64_t)r * a.table_stride + have + (p - s_off[x])] = fine ? page : -1;
    }
    // the block's tokens that belong to this chunk
    const int64_t lo = t0 > tok0 ? t0 : tok0, hi = imin(t1, tok0 + total.tokens);
    static_assert(kTokens == 2 * THREADS, "a thread's two tokens, whose searches and loads go side by side");
    {
      int x[2] = {0, 0}, rel[2], page[2], col[2], pos[2];
      bool live[2], had[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int64_t t = lo + tid + i * THREADS;
        live[i] = t < hi;
        rel[i] = live[i] ? (int)(t - tok0) : 0;
      }
      // the last request whose first token is not after the token
      for (int step = kChunk / 2; step > 0; step >>= 1)
#pragma unroll
        for (int i = 0; i < 2; i++)
          if (s_start[x[i] + step] <= rel[i]) x[i] += step;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        live[i] = live[i] && base + x[i] < a.requests;
        had[i] = live[i] && s_off[x[i]] >= 0;
        pos[i] = had[i] ? a.lens[base + x[i]] : 0;
      }
#pragma unroll
      for (int i = 0; i < 2; i++) {
        page[i] = -1;
        if (!had[i]) continue;
        const int r = base + x[i], have = (int)(((int64_t)pos[i] + P - 1) >> a.page_shift);
        pos[i] += rel[i] - s_start[x[i]];
        col[i] = pos[i] >> a.page_shift;
        page[i] = col[i] < have ? a.table[(int64_t)r * a.table_stride + col[i]]
                                : a.free_pages[count - 1 - (need0 + s_off[x[i]] + col[i] - have)];
      }
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int64_t t = lo + tid + i * THREADS;
        if (t >= hi) continue;
        const bool fine = page[i] >= 0 && page[i] < a.num_pages;
        if (had[i] && !fine) bad = true;
        a.positions[t] = pos[i];
        a.slots[t] = fine ? (page[i] << a.page_shift) + (pos[i] & (P - 1)) : -1;
      }
    }
    need0 += total.need;
    tok0 += total.tokens;
    __syncthreads();  // s_start and s_off are written again
  }
  for (int64_t t = (t0 > tok0 ? t0 : tok0) + tid; t < t1; t += THREADS) {
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
  const int threads = a.requests > 256 * kPtPer ? 1024 : 256;
  const int64_t grid = imax(1, div_up(a.max_tokens, 2 * threads));
  if (trace_on())
    std::fprintf(stderr, "rar trace: page_tables requests=%d tokens=%d page=%d grid=%lld threads=%d\n", a.requests,
                 a.max_tokens, 1 << a.page_shift, (long long)grid, threads);
  void* params[] = {const_cast<PageTablesArgs*>(&a)};
  const void* fn = threads == 1024 ? (const void*)page_tables_kernel<1024> : (const void*)page_tables_kernel<256>;
  return launch_op(fn, dim3((unsigned)grid), threads, 0, stream, params);
}

}  // namespace rar
