// token_logprobs.cu -- log probabilities of given tokens, entropy and the top
// alternatives over vocabulary shards of virtual ranks, and their gradient.
//
//   m = max x, s = sum 2^t, w = sum 2^t t, t = (x - m) log2(e)
//   lse = m + ln s, logprob = x[token] - lse, entropy = ln 2 (log2 s - w / s)
// over a row's shards in rank order; the top alternatives are the largest
// values, the lower index first among equal ones. One pass: m only has to be
// near the maximum, so a lane keeps its own and moves it when a value is more
// than 8 above it (sums to 2^12 times larger lose nothing in binary32); sums
// with their own m join exactly as partial softmaxes do.
//
// The bytes of the logits bound it; about 8 instructions a word leave room for
// twice the words that memory delivers. Tiles of 2048 columns of all rows are
// cut into one equal range per resident block, so few rows use all SMs and many
// rows leave none idle; a row that a cut divides is joined by the block that
// arrives last at it.
//
// Alternatives. Value and index make one 64-bit key. Each warp holds its 32
// best keys sorted over its lanes and a bound below which nothing can matter.
// The first words' bound is the top-th largest of the threads' own maxima; it
// is renewed from all warps' lists whenever the words read have doubled. A word
// at or above the bound is rare then (about top / (words read) of them), and is
// read again and inserted where it belongs.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpTile = kLpThreads * 8;   // columns of a tile
constexpr int kLpBytesAhead = 64;          // bytes a thread has in flight
constexpr int kLpMaxBlocks = 1216;        // most blocks of a forward launch: a partial result and a counter each
constexpr int kLpPartFloats = 4 + 2 * 32;  // m, s, w, then 32 keys
static_assert(kLpMaxBlocks <= kOpCounters, "one arrival counter per block");

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFloorT = -1e4f;  // 2^t is 0 far above this; keeps 0 * t finite for words of -inf

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A value's bits made monotonic, a NaN above all.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return v != v ? 0xffffffffu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// Larger value first, then the lower index. 0 is below every key.
__device__ __forceinline__ uint64_t top_key(float v, uint32_t index) { return (uint64_t)ordered(v) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) { return (int32_t)~(uint32_t)key; }

struct Stat {
  float m, s, w;
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  if (a.m < b.m) {
    const Stat t = a;
    a = b;
    b = t;
  }
  if (b.m == -INFINITY) {
    // b has no word of probability: nothing to add, but a NaN among its words counts
    if (b.s != b.s) a.s = b.s;
    return a;
  }
  const float d = (b.m - a.m) * kLog2e, e = exp2_fast(d);
  if (e > 0.f) a.w += e * (b.w + d * b.s);
  a.s += e * b.s;
  return a;
}
__device__ __forceinline__ Stat warp_join(Stat a) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Stat b;
    b.m = __shfl_xor_sync(~0u, a.m, d);
    b.s = __shfl_xor_sync(~0u, a.s, d);
    b.w = __shfl_xor_sync(~0u, a.w, d);
    a = join(a, b);
  }
  return a;
}

// ---- 32 keys sorted over the lanes of a warp, largest in lane 0 ----
__device__ __forceinline__ uint64_t exchange(uint64_t k, int d, bool keep_large) {
  const uint64_t o = __shfl_xor_sync(~0u, k, d);
  return (k > o) == keep_large ? k : o;
}
__device__ __forceinline__ uint64_t merge_bitonic(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) k = exchange(k, d, (lane & d) == 0);
  return k;
}
__device__ __forceinline__ uint64_t sort32(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) k = exchange(k, d, ((lane & d) == 0) == ((lane & size) == 0 || size == 32));
  return k;
}
// The 32 best of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b) {
  const uint64_t o = __shfl_sync(~0u, b, 31 - (threadIdx.x & 31));
  return merge_bitonic(a > o ? a : o);
}

// The list with one more key, without its last.
__device__ __forceinline__ uint64_t insert32(uint64_t list, uint64_t key) {
  const int lane = threadIdx.x & 31, at = __popc(__ballot_sync(~0u, list > key));
  const uint64_t up = __shfl_up_sync(~0u, list, 1);
  return lane < at ? list : lane == at ? key : up;
}

// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%6, %7};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}

// The largest of eight values, NaN left out.
__device__ __forceinline__ float largest(const Pack8<uint16_t>& u) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u.u);
  const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
  return fmaxf(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ float largest(const Pack8<float>& u) {
  return fmaxf(fmaxf(fmaxf(u.a.x, u.a.y), fmaxf(u.a.z, u.a.w)), fmaxf(fmaxf(u.b.x, u.b.y), fmaxf(u.b.z, u.b.w)));
}

}  // namespace

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ Stat s_stat[kLpWarps];
  __shared__ uint64_t s_list[TOP ? kLpWarps : 1][32];
  __shared__ uint64_t s_bound;
  __shared__ int s_tiles[kMaxRanks + 1];
  __shared__ bool s_last;
  if (!op_workspace_ok(a.ws)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    int n = 0;
    for (int r = 0; r < a.nranks; r++) {
      s_tiles[r] = n;
      n += (int)((a.first[r + 1] - a.first[r] + kLpTile - 1) / kLpTile);
    }
    s_tiles[a.nranks] = n;
  }
  __syncthreads();
  const int per_row = s_tiles[a.nranks];
  const int64_t total = (int64_t)a.rows * per_row;
  const int64_t blocks = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= blocks) return;
  auto start_of = [&](int64_t block) { return block * total / blocks; };
  auto block_of = [&](int64_t tile) { return ((tile + 1) * blocks - 1) / total; };
  const int64_t end = start_of(blockIdx.x + 1);

  for (int64_t at = start_of(blockIdx.x); at < end;) {
    const int row = (int)(at / per_row);
    const int64_t row_first = (int64_t)row * per_row;
    const int t0 = (int)(at - row_first), t1 = (int)(end - row_first < per_row ? end - row_first : per_row);
    Stat st = {-INFINITY, 0.f, 0.f};
    float2 s2 = make_float2(0.f, 0.f), w2 = s2;  // st.s and st.w in two halves, added at the end
    uint64_t list = 0, bound = 0;  // sorted over the lanes; keys not above the bound cannot be among the top
    float bound_value = 0.f;       // value of the bound, for the quick test
    auto add = [&](const Pack8<T>& u, float pm) {
      if (pm > st.m + 8.f) {
        if (st.m != -INFINITY) {
          const float d = (st.m - pm) * kLog2e, e = exp2_fast(d);
          w2 = e > 0.f ? make_float2(e * (w2.x + d * s2.x), e * (w2.y + d * s2.y)) : make_float2(0.f, 0.f);
          s2 = make_float2(s2.x * e, s2.y * e);
        }
        st.m = pm;
      }
      const float m = st.m == -INFINITY ? 0.f : st.m;
      float v[8];
      u.widen(v);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float2 t = mul2(add2(make_float2(v[j], v[j + 1]), make_float2(-m, -m)), make_float2(kLog2e, kLog2e));
        t = make_float2(max_nan(t.x, kFloorT), max_nan(t.y, kFloorT));
        const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
        s2 = add2(s2, e);
        w2 = fma2(e, t, w2);
      }
    };
    // The top-th key of the warps' sorted keys together, for all threads; every thread of the block calls it.
    auto block_bound = [&](uint64_t k) {
#pragma unroll
      for (int d = kLpWarps / 2; d > 0; d >>= 1) {
        if (warp >= d && warp < 2 * d) s_list[warp][lane] = k;
        __syncthreads();
        if (warp < d) k = merge32(k, s_list[warp + d][lane]);
      }
      if (warp == 0 && lane == a.top - 1) s_bound = k;
      __syncthreads();
      return s_bound;
    };
    // Words that may be among the top: bit b of a lane's mask is word[8 kLpThreads (b / 8) + b % 8].
    auto consider = [&](const T* word, uint32_t index, uint32_t mask) {
      while (__any_sync(~0u, mask != 0)) {
        uint64_t key = 0;
        if (mask != 0) {
          const int bit = __ffs(mask) - 1, off = (bit >> 3) * (kLpThreads * 8) + (bit & 7);
          key = top_key(to_float(word[off]), index + off);
          mask &= mask - 1;
        }
        uint32_t votes = __ballot_sync(~0u, key > bound);
        while (votes != 0) {
          const int src = __ffs(votes) - 1;
          list = insert32(list, __shfl_sync(~0u, key, src));
          const uint64_t last = __shfl_sync(~0u, list, a.top - 1);
          bound = last > bound ? last : bound;
          votes = __ballot_sync(~0u, key > bound) & (~0u << src) << 1;
        }
      }
      bound_value = bound == 0 ? -INFINITY : key_value(bound);
    };

    constexpr int kAhead = kLpBytesAhead / (8 * (int)sizeof(T));
    int round = 0;  // of kAhead packs a thread
    const bool alone = t1 - t0 <= kAhead;  // one round has all words: a bound of the warp will do
    for (int t = t0; t < t1;) {
      int rank = 0;
      while (t >= s_tiles[rank + 1]) rank++;
      const int ts = t - s_tiles[rank], te = min(t1, s_tiles[rank + 1]) - s_tiles[rank];
      const int64_t width = a.first[rank + 1] - a.first[rank];
      const int64_t c0 = (int64_t)ts * kLpTile, c1 = imin((int64_t)te * kLpTile, width);
      const T* x = reinterpret_cast<const T*>(a.logits[rank]) + (int64_t)row * a.row_stride[rank] + c0;
      const int n = (int)(c1 - c0);
      const uint32_t word = (uint32_t)(a.first[rank] + c0);
      // words before the first and after the last 16-byte boundary go one to a lane
      const int head = min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
      const int packs = (n - head) / 8, tail = n - head - packs * 8;
      const T* body = x + head;
      // a thread's packs are kLpThreads apart
      for (int p = tid; p - tid < packs; p += kLpThreads * kAhead) {
        Pack8<T> u[kAhead];
        float best = -INFINITY;
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          if (p + i * kLpThreads < packs) u[i].load_stream(body + (int64_t)(p + i * kLpThreads) * 8);
          else u[i].absent();
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          const float pm = largest(u[i]);
          best = fmaxf(best, pm);
          add(u[i], pm);
        }
        if constexpr (TOP) {
          if (round == 0) {
            const uint64_t k = sort32(best == -INFINITY ? 0 : (uint64_t)ordered(best) << 32);
            const uint64_t b = alone ? __shfl_sync(~0u, k, a.top - 1) : block_bound(k);
            if (b > bound) bound = b - 1;
            bound_value = b == 0 ? -INFINITY : key_value(b);
          } else if ((round & (round - 1)) == 0) {
            const uint64_t b = block_bound(list);
            if (b > bound) {
              bound = b;
              bound_value = key_value(b);
            }
          }
          round++;
          // a NaN, which the maxima leave out, shows in the sum; !(<) lets it, and all words under a NaN bound, in
          const bool nan = s2.x != s2.x || s2.y != s2.y;
          if (__any_sync(~0u, !(best < bound_value) || nan)) {
            uint32_t mask = 0;
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
              const bool in = p + i * kLpThreads < packs && (!(largest(u[i]) < bound_value) || nan);
              if (__any_sync(~0u, in)) {
                float v[8];
                u[i].widen(v);
#pragma unroll
                for (int j = 0; j < 8; j++) mask |= in && !(v[j] < bound_value) ? 1u << (8 * i + j) : 0u;
              }
            }
            consider(body + (int64_t)p * 8, word + head + p * 8, mask);
          }
        }
      }
      if (head + tail > 0 && warp == 0) {
        const int e = lane < head ? lane : lane - head < tail ? head + packs * 8 + lane - head : -1;
        const float v = e >= 0 ? to_float(x[e]) : -INFINITY;
        Stat one = {v, v == -INFINITY ? 0.f : 1.f, 0.f};
        if (v != v) one = {-INFINITY, v, 0.f};
        st = join(Stat{st.m, s2.x + s2.y, w2.x + w2.y}, one);
        s2 = make_float2(st.s, 0.f);
        w2 = make_float2(st.w, 0.f);
        if constexpr (TOP) {
          if (round == 0) bound_value = -INFINITY;
          consider(x + e, word + e, e >= 0 && !(v < bound_value) ? 1u : 0u);
        }
      }
      t = te + s_tiles[rank];
    }

    // the block's warps join
    st = warp_join(Stat{st.m, s2.x + s2.y, w2.x + w2.y});
    if (lane == 0) s_stat[warp] = st;
    auto join_lists = [&]() {  // list of all warps -> s_list[0]
      if constexpr (TOP) {
#pragma unroll
        for (int d = kLpWarps / 2; d > 0; d >>= 1) {
          if (warp >= d && warp < 2 * d) s_list[warp][lane] = list;
          __syncthreads();
          if (warp < d) list = merge32(list, s_list[warp + d][lane]);
        }
      }
    };
    join_lists();
    __syncthreads();
    if (warp == 0) st = warp_join(lane < kLpWarps ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f});

    bool mine = true;  // this block has the whole row's result
    if (t0 != 0 || t1 != per_row) {
      const int cf = (int)block_of(row_first), cl = (int)block_of(row_first + per_row - 1);
      float* parts = reinterpret_cast<float*>(a.ws + kOpScratchOffset);
      const bool starts_at_cf = start_of(cf) == row_first;
      auto part_of = [&](int block) {  // of its first row, or of the row that starts in it and goes on
        return parts + (2 * block + (block == cf && !starts_at_cf)) * kLpPartFloats;
      };
      if (warp == 0) {
        float* part = part_of(blockIdx.x);
        if (lane == 0) {
          part[0] = st.m;
          part[1] = st.s;
          part[2] = st.w;
        }
        if (TOP) reinterpret_cast<uint64_t*>(part + 4)[lane] = list;
        __threadfence();
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t* counter = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes) + cf;
        s_last = atomicAdd(counter, 1u) == (uint32_t)(cl - cf);
        if (s_last) *counter = 0;
      }
      __syncthreads();
      mine = s_last;
      if (mine) {
        __threadfence();
        st = {-INFINITY, 0.f, 0.f};
        list = 0;
        for (int p = cf + tid; p <= cl; p += kLpThreads) {
          const float* part = part_of(p);
          st = join(st, Stat{__ldcg(part), __ldcg(part + 1), __ldcg(part + 2)});
        }
        if (TOP)
          for (int p = cf + warp; p <= cl; p += kLpWarps)
            list = merge32(list, __ldcg(reinterpret_cast<const unsigned long long*>(part_of(p) + 4) + lane));
        st = warp_join(st);
        if (lane == 0) s_stat[warp] = st;
        join_lists();
        __syncthreads();
        if (warp == 0) st = warp_join(lane < kLpWarps ? s_stat[lane] : Stat{-INFINITY, 0.f, 0.f});
      }
    }
    if (mine && warp == 0) {
      if (st.m == INFINITY) st.s = NAN;  // exp(inf - inf)
      const float log2_s = log2f(st.s), lse = st.m + kLn2 * log2_s;
      if (lane == 0) {
        const int64_t token = a.tokens[row];
        float lp = 0.f;
        for (int r = 0; r < a.nranks; r++)
          if (token >= a.first[r] && token < a.first[r + 1])
            lp = to_float(reinterpret_cast<const T*>(a.logits[r])[(int64_t)row * a.row_stride[r] + token - a.first[r]]) - lse;
        a.logprob[row] = lp;
        a.entropy[row] = kLn2 * (log2_s - st.w / st.s);
        a.lse[row] = lse;
      }
      if (TOP && lane < a.top) {
        a.top_values[(int64_t)row * a.top + lane] = key_value(list) - lse;
        a.top_ids[(int64_t)row * a.top + lane] = key_index(list);
      }
    }
    at = row_first + t1;
  }
}

// dx = g ([i == token] - p) - h p (y + entropy), y = x - lse, p = exp(y); g counts
// only if a token was asked for. One pass, read and written once; a block takes
// kLpBwdTile columns of a row of a shard.
constexpr int kLpBwdTile = kLpThreads * 8 * 8;

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(const __grid_constant__ LogprobBwdArgs a,
                                                                       int tiles) {
  if (!op_workspace_ok(a.ws)) return;
  const int row = (int)(blockIdx.x / (unsigned)tiles), tile = (int)(blockIdx.x % (unsigned)tiles);
  const int rank = blockIdx.y, tid = threadIdx.x;
  const int64_t width = a.first[rank + 1] - a.first[rank], c0 = (int64_t)tile * kLpBwdTile;
  if (c0 >= width) return;
  const int n = (int)imin(kLpBwdTile, width - c0);
  const T* x = reinterpret_cast<const T*>(a.logits[rank]) + (int64_t)row * a.row_stride[rank] + c0;
  T* dx = reinterpret_cast<T*>(a.dlogits[rank]) + (int64_t)row * a.drow_stride[rank] + c0;
  const float lse = a.lse[row];
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.f;
  const int64_t token = a.tokens[row];
  const bool asked = token >= 0 && token < a.first[a.nranks];
  const float g = asked ? a.grad_logprob[row] : 0.f;
  const float base = g + h * a.entropy[row];
  const int64_t at = token - a.first[rank] - c0;
  const int mine = asked && at >= 0 && at < n ? (int)at : -1;
  auto grad = [&](float v) {
    const float y = max_nan(v - lse, kFloorT);
    return -exp2_fast(y * kLog2e) * fmaf(h, y, base);
  };
  // rows that share a 16-byte phase go in packs, the ends one by one; others one by one altogether
  const bool together = (((uintptr_t)x ^ (uintptr_t)dx) & 15) == 0;
  const int head = together ? min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T)) : n;
  const int packs = (n - head) / 8, done = head + packs * 8;
  constexpr int kAhead = kLpBytesAhead / (8 * (int)sizeof(T));
  for (int p0 = 0; p0 < packs; p0 += kLpThreads * kAhead) {
    Pack8<T> u[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const int p = p0 + i * kLpThreads + tid;
      if (p < packs) u[i].load_stream(x + head + (int64_t)p * 8);
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const int p = p0 + i * kLpThreads + tid;
      if (p >= packs) break;
      float v[8];
      u[i].widen(v);
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = grad(v[j]);
      const int k = mine - head - p * 8;
      if ((unsigned)k < 8u) {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (j == k) v[j] += g;
      }
      u[i].narrow(v);
      u[i].store(dx + head + (int64_t)p * 8);
    }
  }
  for (int i = tid; i < head + n - done; i += kLpThreads) {
    const int e = i < head ? i : done + i - head;
    from_float(dx + e, grad(to_float(x[e])) + (e == mine ? g : 0.f));
  }
}

int64_t token_logprobs_scratch_bytes(int, int) { return 2ll * kLpMaxBlocks * kLpPartFloats * (int64_t)sizeof(float); }

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  const void* fn = a.dtype == kF32 ? (a.top > 0 ? (const void*)token_logprobs_kernel<float, true>
                                                : (const void*)token_logprobs_kernel<float, false>)
                                   : (a.top > 0 ? (const void*)token_logprobs_kernel<uint16_t, true>
                                                : (const void*)token_logprobs_kernel<uint16_t, false>);
  int device = 0, sms = 0, per_sm = 0;
  cudaError_t e = current_device_sms(&device, &sms);
  if (e != cudaSuccess) return e;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kLpThreads, 0);
  if (e != cudaSuccess) return e;
  int64_t tiles = 0;
  for (int r = 0; r < a.nranks; r++) tiles += div_up(a.first[r + 1] - a.first[r], kLpTile);
  const int64_t grid = imin(imin((int64_t)sms * per_sm, kLpMaxBlocks), tiles * a.rows);
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs nranks=%d rows=%d vocab=%lld top=%d grid=%lld\n", a.nranks, a.rows,
                 (long long)a.first[a.nranks], a.top, (long long)grid);
  void* params[] = {const_cast<LogprobArgs*>(&a)};
  return cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(kLpThreads), params, 0, stream);
}

cudaError_t launch_token_logprobs_bwd(const LogprobBwdArgs& a, cudaStream_t stream) {
  int64_t widest = 0;
  for (int r = 0; r < a.nranks; r++) widest = imax(widest, a.first[r + 1] - a.first[r]);
  int tiles = (int)div_up(widest, kLpBwdTile);
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs_backward nranks=%d rows=%d vocab=%lld tiles=%d\n", a.nranks, a.rows,
                 (long long)a.first[a.nranks], tiles);
  dim3 grid((unsigned)((int64_t)a.rows * tiles), (unsigned)a.nranks);
  const void* fn = a.dtype == kF32 ? (const void*)token_logprobs_bwd_kernel<float>
                                   : (const void*)token_logprobs_bwd_kernel<uint16_t>;
  void* params[] = {const_cast<LogprobBwdArgs*>(&a), &tiles};
  return cudaLaunchKernel(fn, grid, dim3(kLpThreads), params, 0, stream);
}

}  // namespace rar
