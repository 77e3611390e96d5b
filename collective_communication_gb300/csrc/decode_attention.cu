// decode_attention.cu -- attention of one new token per request over a paged
// key-value cache, all virtual ranks in one launch.
//
//   s_t = scale * (q . k_t),  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
// over the t < len cached tokens of the request, with the running maximum m and
// sum of the softmax in binary32; lse = m + log(sum). A request of length 0
// gives o = 0 and lse = -inf.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kDaThreads = 128;
constexpr int kDaTile = 64;

// One block per (query head, request, rank).
template <typename T>
__global__ void __launch_bounds__(kDaThreads) decode_attention_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float s_q[256], s_s[kDaTile];
  __shared__ int64_t s_row[kDaTile];
  if (!op_workspace_ok(a.ws)) return;
  const int h = blockIdx.x, b = blockIdx.y, rank = blockIdx.z, D = a.head_dim, tid = threadIdx.x;
  const int kvh = h / (a.q_heads / a.kv_heads);
  const T* q = reinterpret_cast<const T*>(a.q[rank]) + (int64_t)b * a.q_stride + (int64_t)h * D;
  const T* kc = reinterpret_cast<const T*>(a.k_cache[rank]);
  const T* vc = reinterpret_cast<const T*>(a.v_cache[rank]);
  int len = a.lens[b];
  bool bad = len < 0 || len > (int64_t)a.max_blocks << a.page_shift;
  if (bad) len = len < 0 ? 0 : (int)((int64_t)a.max_blocks << a.page_shift);
  for (int d = tid; d < D; d += kDaThreads) s_q[d] = to_float(q[d]) * a.scale;
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  for (int t0 = 0; t0 < len; t0 += kDaTile) {
    __syncthreads();
    const int n = len - t0 < kDaTile ? len - t0 : kDaTile;
    if (tid < n) {
      const int t = t0 + tid;
      const int page = a.table[(int64_t)b * a.table_stride + (t >> a.page_shift)];
      const bool fine = page >= 0 && page < a.num_pages;
      if (!fine) bad = true;
      s_row[tid] = fine ? ((((int64_t)page * a.kv_heads + kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1))) * D
                        : -1;
    }
    __syncthreads();
    for (int i = tid >> 5; i < n; i += kDaThreads / 32) {
      float s = 0.f;
      const int64_t row = s_row[i];
      if (row >= 0)
        for (int d = tid & 31; d < D; d += 32) s += s_q[d] * to_float(kc[row + d]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
      if ((tid & 31) == 0) s_s[i] = row >= 0 ? s : -INFINITY;
    }
    __syncthreads();
    float top = m;
    for (int i = 0; i < n; i++) top = fmaxf(top, s_s[i]);
    if (top == -INFINITY) continue;
    const float keep = expf(m - top);
    m = top;
    l *= keep;
    acc[0] *= keep;
    acc[1] *= keep;
    for (int i = 0; i < n; i++) {
      if (s_row[i] < 0) continue;
      const float p = expf(s_s[i] - m);
      l += p;
      for (int j = 0; j < 2; j++) {
        const int d = tid + j * kDaThreads;
        if (d < D) acc[j] += p * to_float(vc[s_row[i] + d]);
      }
    }
  }
  T* out = reinterpret_cast<T*>(a.out[rank]) + (int64_t)b * a.out_stride + (int64_t)h * D;
  for (int j = 0; j < 2; j++) {
    const int d = tid + j * kDaThreads;
    if (d < D) from_float(out + d, len == 0 ? 0.f : acc[j] / l);
  }
  if (tid == 0 && a.lse[rank] != nullptr) a.lse[rank][(int64_t)b * a.q_heads + h] = m + logf(l);
  if (bad) op_report(a.ws, kErrCapacity);
}

int64_t decode_attention_scratch_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_decode_attention(const DecodeArgs& a, cudaStream_t stream) {
  dim3 grid((unsigned)a.q_heads, (unsigned)a.batch, (unsigned)a.nranks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: decode_attention nranks=%d batch=%d heads=%d/%d dim=%d grid=%ux%ux%u\n", a.nranks,
                 a.batch, a.q_heads, a.kv_heads, a.head_dim, grid.x, grid.y, grid.z);
  if (a.dtype == kF32) decode_attention_kernel<float><<<grid, kDaThreads, 0, stream>>>(a);
  else decode_attention_kernel<uint16_t><<<grid, kDaThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rar
