// token_logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives over vocabulary shards of virtual ranks, and their gradient.
//
//   m = max x, s = sum exp(x - m), lse = m + log s, logprob = x[token] - lse
//   entropy = log s - sum exp(x - m) (x - m) / s
// over a row's shards in rank order; the top alternatives are the largest
// values, the lower index first among equal ones.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kLpThreads = 256;

namespace {

// The order of the alternatives as one number: the value's bits made monotonic
// (a NaN above all), then the lower index first.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t index) {
  uint32_t u = __float_as_uint(v);
  u = v != v ? 0xffffffffu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (uint64_t)u << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

struct Stat {
  float m, s, w;  // maximum, sum of exp(x - m), sum of exp(x - m) (x - m)
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  if (a.m == -INFINITY) return b;
  if (b.m == -INFINITY) return a;
  if (a.m < b.m) { const Stat t = a; a = b; b = t; }
  const float d = b.m - a.m, e = expf(d);
  if (b.s > 0.f || b.s != b.s) {
    a.w += e > 0.f ? e * (b.w + d * b.s) : e * b.s;
    a.s += e * b.s;
  }
  return a;
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ Stat s_stat[kLpThreads];
  __shared__ uint64_t s_key[kLpThreads];
  if (!op_workspace_ok(a.ws)) return;
  const int row = blockIdx.x, tid = threadIdx.x;
  Stat st = {-INFINITY, 0.f, 0.f};
  for (int r = 0; r < a.nranks; r++) {
    const T* x = reinterpret_cast<const T*>(a.logits[r]) + (int64_t)row * a.row_stride[r];
    const int64_t n = a.first[r + 1] - a.first[r];
    for (int64_t i = tid; i < n; i += kLpThreads) {
      const float v = to_float(x[i]);
      if (v == -INFINITY) continue;
      st = join(st, Stat{v, 1.f, 0.f});
    }
  }
  s_stat[tid] = st;
  __syncthreads();
  for (int d = kLpThreads / 2; d > 0; d >>= 1) {
    if (tid < d) s_stat[tid] = join(s_stat[tid], s_stat[tid + d]);
    __syncthreads();
  }
  st = s_stat[0];
  if (st.m == INFINITY) st.s = NAN;  // exp(inf - inf)
  const float log_s = logf(st.s), lse = st.m + log_s;
  if (tid == 0) {
    const int64_t token = a.tokens[row];
    float lp = 0.f;
    for (int r = 0; r < a.nranks; r++)
      if (token >= a.first[r] && token < a.first[r + 1])
        lp = to_float(reinterpret_cast<const T*>(a.logits[r])[(int64_t)row * a.row_stride[r] + token - a.first[r]]) - lse;
    a.logprob[row] = lp;
    a.entropy[row] = log_s - st.w / st.s;
    a.lse[row] = lse;
  }
  uint64_t below = ~0ull;
  for (int k = 0; k < a.top; k++) {
    uint64_t best = 0;
    for (int r = 0; r < a.nranks; r++) {
      const T* x = reinterpret_cast<const T*>(a.logits[r]) + (int64_t)row * a.row_stride[r];
      const int64_t n = a.first[r + 1] - a.first[r];
      for (int64_t i = tid; i < n; i += kLpThreads) {
        const uint64_t key = top_key(to_float(x[i]), (uint32_t)(a.first[r] + i));
        if (key < below && key > best) best = key;
      }
    }
    s_key[tid] = best;
    __syncthreads();
    for (int d = kLpThreads / 2; d > 0; d >>= 1) {
      if (tid < d && s_key[tid + d] > s_key[tid]) s_key[tid] = s_key[tid + d];
      __syncthreads();
    }
    below = s_key[0];
    __syncthreads();
    if (tid == 0) {
      a.top_values[(int64_t)row * a.top + k] = key_value(below) - lse;
      a.top_ids[(int64_t)row * a.top + k] = (int32_t)~(uint32_t)below;
    }
  }
}

// dx = g ([i == token] - p) - h p (log p + entropy), p = exp(x - lse); g counts
// only if a token was asked for. One pass; a shard's row may start on any
// element, so its ends up to the first 16-byte boundary go one by one.
template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(const __grid_constant__ LogprobBwdArgs a) {
  if (!op_workspace_ok(a.ws)) return;
  const int row = blockIdx.x, rank = blockIdx.y, tid = threadIdx.x;
  const T* x = reinterpret_cast<const T*>(a.logits[rank]) + (int64_t)row * a.row_stride[rank];
  T* dx = reinterpret_cast<T*>(a.dlogits[rank]) + (int64_t)row * a.drow_stride[rank];
  const int64_t n = a.first[rank + 1] - a.first[rank];
  const float lse = a.lse[row], H = a.entropy[row];
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.f;
  const int64_t token = a.tokens[row];
  const bool asked = token >= 0 && token < a.first[a.nranks];
  const float g = asked ? a.grad_logprob[row] : 0.f;
  const int64_t mine = token - a.first[rank];
  for (int64_t i = tid; i < n; i += kLpThreads) {
    const float y = to_float(x[i]) - lse, p = expf(y);
    float d = p == 0.f ? 0.f : -p * (g + h * (y + H));
    if (i == mine && asked) d += g;
    from_float(dx + i, d);
  }
}

int64_t token_logprobs_scratch_bytes(int, int) { return 0; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs nranks=%d rows=%d vocab=%lld top=%d\n", a.nranks, a.rows,
                 (long long)a.first[a.nranks], a.top);
  if (a.dtype == kF32) token_logprobs_kernel<float><<<a.rows, kLpThreads, 0, stream>>>(a);
  else token_logprobs_kernel<uint16_t><<<a.rows, kLpThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_token_logprobs_bwd(const LogprobBwdArgs& a, cudaStream_t stream) {
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs_backward nranks=%d rows=%d vocab=%lld\n", a.nranks, a.rows,
                 (long long)a.first[a.nranks]);
  dim3 grid((unsigned)a.rows, (unsigned)a.nranks);
  if (a.dtype == kF32) token_logprobs_bwd_kernel<float><<<grid, kLpThreads, 0, stream>>>(a);
  else token_logprobs_bwd_kernel<uint16_t><<<grid, kLpThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rar
