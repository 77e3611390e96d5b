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
// The bytes of the logits bound it; instructions come close, so they are
// counted: about 7 a word, packed binary32 operations where there are any.
// Tiles of 1024 columns of all rows are cut into about one equal range per
// resident warp, so few rows use all SMs and many rows leave none idle, and no
// warp waits for another (blocks that joined their warps' results at the end of
// every row spent a fifth of the time at barriers). A row that a cut divides is
// joined by the warp that arrives last at it.
//
// Alternatives. Value and index make one 64-bit key. A warp holds its 32 best
// keys sorted over its lanes and a bound below which nothing can matter: first
// the top-th largest of the lanes' own maxima, then the list's top-th key. A
// word at or above the bound is rare after the first tile (about top / (words
// read) of them), and is read again and inserted where it belongs.
// Measured: 2048 rows of 8 shards of 16003 words in bf16, 524 MB: 87 us without
// alternatives (6.0 TB/s, 0.90 of the measured copy), 107 us with 5, 133 with 20:
// the list's instructions. 3 rows of 131072 words: 6.7 us without alternatives,
// 11 with 8, 14 with 20: a launch, a tile and a join of 128 parts. The
// gradient, 2048 rows of 131072 words read and written: 157 us, 6.8 TB/s (1.0 of
// the measured copy).
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxWorkers = 4864;       // most warps of a forward launch: a counter and two partial results each
// Alternatives are inserted one by one, and lanes' words looked at by the whole warp, where there are few; more are
// sorted, and found by each lane on its own (3 rows of 24848 words in f32, top 20: 14 us against 22; 704 rows of
// 80688 words in bf16, top 20: 53 against 66, top 5 no different).
constexpr int kLpFewKeys = 6, kLpFewLanes = 4;
// A row of few parts merges their lists, others pick from them (12 rows of 3381 words, top 20: 11.4 us against 15.5).
constexpr int kLpFewParts = 8;
constexpr int kLpPartFloats = 4 + 2 * 32;  // m, s, w, then 32 keys
static_assert(kLpMaxWorkers <= kOpCounters, "one arrival counter per warp");

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

__device__ __forceinline__ float sum_of(F2 a) {
  const float2 p = unpack(a);
  return p.x + p.y;
}

// A value's bits made monotonic, a NaN above all, -0 as 0 (-0 + 0 is 0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
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

// 32 values without NaN sorted over the lanes of a warp, largest in lane 0.
__device__ __forceinline__ float exchange(float k, int d, bool keep_large) {
  const float o = __shfl_xor_sync(~0u, k, d);
  return keep_large ? fmaxf(k, o) : fminf(k, o);
}
__device__ __forceinline__ float sort32(float k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) k = exchange(k, d, ((lane & d) == 0) == ((lane & size) == 0 || size == 32));
  return k;
}
// 32 keys sorted over the lanes, largest in lane 0: with one more, without the last.
__device__ __forceinline__ uint64_t insert32(uint64_t list, uint64_t key) {
  const int lane = threadIdx.x & 31, at = __popc(__ballot_sync(~0u, list > key));
  const uint64_t up = __shfl_up_sync(~0u, list, 1);
  return lane < at ? list : lane == at ? key : up;
}

// Sorts 32 keys over the lanes, largest in lane 0, from the stage whose runs have FROM lanes on (2: any keys;
// 32: two runs, one falling and one rising).
template <int FROM>
__device__ __forceinline__ uint64_t sort32(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = FROM; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const uint64_t o = __shfl_xor_sync(~0u, k, d);
      const bool large = ((lane & d) == 0) == ((lane & size) == 0 || size == 32);
      k = (o > k) == large ? o : k;
    }
  return k;
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

// A warp's alternatives.
struct TopList {
  uint64_t list = 0, bound = 0;  // sorted over the lanes; keys not above the bound cannot be among the top
  float bound_value = -INFINITY;  // value of the bound, for quick tests: !(value < bound_value) lets a NaN in

  // Another list, sorted likewise.
  __device__ __forceinline__ void merge(uint64_t sorted) {
    const uint64_t other = __shfl_xor_sync(~0u, sorted, 31);
    list = sort32<32>(other > list ? other : list);
  }
  // Every lane's key, 0 for none: those above the bound are inserted one after another, or where MANY are expected and
  // there are many, sorted and merged.
  template <bool MANY>
  __device__ __forceinline__ void offer(uint64_t key, int top) {
    uint32_t votes = __ballot_sync(~0u, key > bound);
    if (votes == 0) return;
    if (MANY && __popc(votes) > kLpFewKeys) {
      merge(sort32<2>(key > bound ? key : 0));
      votes = 0;
    }
    for (; votes != 0; votes &= votes - 1) list = insert32(list, __shfl_sync(~0u, key, __ffs(votes) - 1));
    const uint64_t last = __shfl_sync(~0u, list, top - 1);
    bound = last > bound ? last : bound;
    bound_value = bound == 0 ? -INFINITY : key_value(bound);
  }
  // `value` is in the top-th place of some values: no key of a smaller value matters.
  __device__ __forceinline__ void start(float value) {
    bound_value = value;
    if (value != -INFINITY) bound = ((uint64_t)ordered(value) << 32) - 1;
  }
};

// NARROW: rows of few rounds, where it pays to look how much of a round there is.
template <typename T, bool TOP, bool NARROW>
__global__ void __launch_bounds__(kLpThreads, 4) token_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  constexpr int kAhead = 64 / (8 * (int)sizeof(T));  // packs of a lane in flight
  __shared__ __align__(16) T s_words[TOP ? kLpWarps : 1][kAhead][32][8];
  const uint32_t magic = op_start(a.ws);
  const int lane = threadIdx.x & 31;
  // neighbouring ranges go to different blocks, so that few workers still spread over the SMs
  const uint32_t worker = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  if (worker >= a.workers) return;
  const uint32_t per_row = a.first_tile[a.nranks];
  // rows in a.cuts equal parts each, or (a.cuts 0) all tiles in one equal range a worker: w's start at w * each + min(w, more)
  auto start_of = [&](uint32_t w) {
    return a.cuts > 0 ? w / a.cuts * per_row + (uint32_t)((uint64_t)(w % a.cuts) * per_row / a.cuts)
                      : (w * a.each + min(w, a.more)) * a.unit;
  };
  auto worker_of = [&](uint32_t row, bool last) {  // the one with the row's first or last tile
    if (a.cuts > 0) return row * a.cuts + (last ? a.cuts - 1 : 0);
    const uint32_t at = (row * per_row + (last ? per_row - 1 : 0)) / a.unit, split = a.more * (a.each + 1);
    return at < split ? at / (a.each + 1) : a.more + (at - split) / a.each;
  };
  const uint32_t end = start_of(worker + 1);

  for (uint32_t at = start_of(worker); at < end;) {
    const uint32_t row = at / per_row, row_first = row * per_row;
    const int t0 = (int)(at - row_first), t1 = (int)(min(end, row_first + per_row) - row_first);
    float m = -INFINITY;                           // near the largest of the lane's words
    F2 s2 = f2(0.f, 0.f), w2 = s2;            // its sums in two halves
    TopList tops;

    for (int t = t0; t < t1;) {
      // the part's words of one shard
      int rank = 0;
      while (t >= a.first_tile[rank + 1]) rank++;
      const int ts = t - a.first_tile[rank], te = min(t1, a.first_tile[rank + 1]) - a.first_tile[rank];
      const int64_t width = a.first[rank + 1] - a.first[rank];
      const int64_t c0 = (int64_t)ts * kLpTile, c1 = imin((int64_t)te * kLpTile, width);
      const T* x = reinterpret_cast<const T*>(a.logits[rank]) + (int64_t)row * a.row_stride[rank] + c0;
      const int n = (int)(c1 - c0);
      const bool begins = t == t0;
      t = te + a.first_tile[rank];
      // up to the first and from the last 16-byte boundary one by one, 16-byte packs between
      const int head = min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T));
      const int packs = (n - head) / 8, tail = n - head - packs * 8;
      const T* body = x + head;
      const uint32_t word = (uint32_t)(a.first[rank] + c0) + head;

      // a round is kAhead packs a lane, 32 apart
      Pack8<T> u[kAhead];
      auto fetch = [&](int p) {
        if (p - lane + 32 * kAhead <= packs) {
#pragma unroll
          for (int i = 0; i < kAhead; i++) u[i].load_stream(body + (int64_t)(p + i * 32) * 8);
        } else {
#pragma unroll
          for (int i = 0; i < kAhead; i++) {
            if (p + i * 32 < packs) u[i].load_stream(body + (int64_t)(p + i * 32) * 8);
            else u[i].absent();
          }
        }
      };
      if (packs > 0) fetch(lane);
      for (int p = lane; p - lane < packs; p += 32 * kAhead) {
        float best = largest(u[0]);
#pragma unroll
        for (int i = 1; i < kAhead; i++) best = fmaxf(best, largest(u[i]));
        if (best > m + 8.f) {
          if (m != -INFINITY) {
            const float d = (m - best) * kLog2e, e = exp2_fast(d);
            w2 = e > 0.f ? mul2(f2(e, e), fma2(f2(d, d), s2, w2)) : f2(0.f, 0.f);
            s2 = mul2(s2, f2(e, e));
          }
          m = best;
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const F2 off = f2(neg, neg), log2e = f2(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          if (NARROW && i > 0 && p - lane + i * 32 >= packs) break;
          float v[8];
          u[i].widen(v);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float2 t = unpack(mul2(add2(f2(v[j], v[j + 1]), off), log2e));
            t = make_float2(max_nan(t.x, kFloorT), max_nan(t.y, kFloorT));
            const F2 e = f2(exp2_fast(t.x), exp2_fast(t.y));
            s2 = add2(s2, e);
            w2 = fma2(e, f2(t.x, t.y), w2);
          }
        }
        uint32_t lanes = 0;
        if constexpr (TOP) {
          if (begins && p == lane) tops.start(__shfl_sync(~0u, sort32(best), a.top - 1));
          // lanes with a word that may matter (a NaN, which the maxima leave out, shows in the sum): the warp looks at
          // their words together, a word to a lane, with the next round's loads on their way
          lanes = __ballot_sync(~0u, !(best < tops.bound_value) || sum_of(s2) != sum_of(s2));
          if (lanes != 0) {
#pragma unroll
            for (int i = 0; i < kAhead; i++) u[i].store(s_words[threadIdx.x >> 5][i][lane]);
          }
        }
        if (p - lane + 32 * kAhead < packs) fetch(p + 32 * kAhead);
        if constexpr (TOP) {
          if (lanes != 0) {
            T(*words)[32][8] = s_words[threadIdx.x >> 5];
            __syncwarp();
            if (__popc(lanes) > kLpFewLanes) {
              // many, as in the first rounds: each lane walks through its own words
              uint32_t mine = 0;
#pragma unroll
              for (int i = 0; i < kAhead; i++) {
                Pack8<T> own;
                own.load(words[i][lane]);
                float v[8];
                own.widen(v);
#pragma unroll
                for (int j = 0; j < 8; j++)
                  if (p + i * 32 < packs && !(v[j] < tops.bound_value)) mine |= 1u << (i * 8 + j);
              }
              while (__any_sync(~0u, mine != 0)) {
                const int b = __ffs(mine) - 1, i = b >> 3, j = b & 7;  // -1 when there are no more
                tops.offer<true>(mine != 0 ? top_key(to_float(words[i][lane][j]), word + (p + i * 32) * 8 + j) : 0, a.top);
                mine &= mine - 1;
              }
              lanes = 0;
            }
            for (; lanes != 0; lanes &= lanes - 1) {
              const int l = __ffs(lanes) - 1, pack = p - lane + l + (lane >> 3) * 32;
              const bool there = lane < 8 * kAhead && pack < packs;
              const int i = there ? lane >> 3 : 0;
              tops.offer<false>(there ? top_key(to_float(words[i][l][lane & 7]), word + pack * 8 + (lane & 7)) : 0, a.top);
            }
            __syncwarp();
          }
        }
      }
      if (head + tail > 0) {
        const bool mine = lane < head + tail;
        const int e = lane < head ? lane - head : packs * 8 + lane - head;
        const float v = mine ? to_float(body[e]) : -INFINITY;
        Stat one = {v, v == -INFINITY ? 0.f : 1.f, 0.f};
        if (v != v) one = {-INFINITY, v, 0.f};
        one = join(Stat{m, sum_of(s2), sum_of(w2)}, one);
        m = one.m;
        s2 = f2(one.s, 0.f);
        w2 = f2(one.w, 0.f);
        if constexpr (TOP) tops.offer<false>(mine ? top_key(v, word + e) : 0, a.top);
      }
    }
    // the token's word, needed last, is on its way during the joins
    const int64_t token = a.tokens[row];
    float word_of_token = 0.f;
    bool asked = false;
    for (int r = 0; r < a.nranks; r++)
      if (token >= a.first[r] && token < a.first[r + 1]) {
        asked = true;
        word_of_token = to_float(reinterpret_cast<const T*>(a.logits[r])[(int64_t)row * a.row_stride[r] + token - a.first[r]]);
      }
    Stat st = warp_join(Stat{m, sum_of(s2), sum_of(w2)});
    if (!op_ready(a.ws, magic)) return;

    bool whole = t0 == 0 && t1 == (int)per_row;  // this warp has the row's result
    if (!whole) {
      const uint32_t wf = worker_of(row, false), wl = worker_of(row, true);
      const bool starts_at_wf = start_of(wf) == row_first;
      float* parts = reinterpret_cast<float*>(a.ws + kOpScratchOffset);
      auto part_of = [&](uint32_t w) {  // of its first row, or of the row that starts in it and goes on
        return parts + (2 * w + (w == wf && !starts_at_wf)) * kLpPartFloats;
      };
      float* part = part_of(worker);
      if (lane == 0) {
        part[0] = st.m;
        part[1] = st.s;
        part[2] = st.w;
      }
      if (TOP && lane < a.top) reinterpret_cast<uint64_t*>(part + 4)[lane] = tops.list;
      __syncwarp();
      uint32_t arrived = 0;
      if (lane == 0) {
        // releases the warp's part, and acquires the others' if it is the last
        uint32_t* counter = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes) + wf;
        arrived = atom_add_acq_rel_u32(counter, 1u);
        if (arrived == wl - wf) *counter = 0;
      }
      whole = __shfl_sync(~0u, arrived, 0) == wl - wf;
      __syncwarp();  // what lane 0 acquired is there for all lanes
      if (whole) {
        // in the workers' order, whoever joins: a lane's share first, then over the lanes
        st = {-INFINITY, 0.f, 0.f};
        float head = -INFINITY;  // largest of the lane's parts' first alternatives
        constexpr int kAt = 4;   // parts of a lane at a time
        auto pair_of = [&](uint32_t w, int i) {
          ulonglong2 v = make_ulonglong2(0, 0);
          if (w <= wl) v = __ldcg(reinterpret_cast<const ulonglong2*>(part_of(w) + 4) + i / 2);
          if (i + 1 >= a.top) v.y = 0;
          return v;
        };
        for (uint32_t w0 = wf; w0 <= wl; w0 += 32 * kAt) {
          Stat q[kAt];
          uint64_t k[kAt];
#pragma unroll
          for (int j = 0; j < kAt; j++) {
            const uint32_t w = w0 + lane + 32 * j;
            q[j] = {-INFINITY, 0.f, 0.f};
            if (w <= wl) {
              const float* from = part_of(w);
              q[j] = {__ldcg(from), __ldcg(from + 1), __ldcg(from + 2)};
            }
            k[j] = 0;
            if (TOP && w <= wl) k[j] = __ldcg(reinterpret_cast<const unsigned long long*>(part_of(w) + 4));
          }
#pragma unroll
          for (int j = 0; j < kAt; j++) {
            st = join(st, q[j]);
            if (TOP && k[j] != 0) head = fmaxf(head, key_value(k[j]));
          }
        }
        st = warp_join(st);
        if constexpr (TOP) {
          // few parts: their lists one after another; many: a lane offers its parts' alternatives in turn, until they
          // fall below the bound
          tops = TopList();
          const bool few = wl - wf < (uint32_t)min(kLpFewParts, a.top);
          for (uint32_t w0 = wf; few && w0 <= wl; w0 += kAt) {
            uint64_t k[kAt];
#pragma unroll
            for (int j = 0; j < kAt; j++)
              k[j] = w0 + j <= wl && lane < a.top
                         ? __ldcg(reinterpret_cast<const unsigned long long*>(part_of(w0 + j) + 4) + lane) : 0;
#pragma unroll 1
            for (int j = 0; j < kAt; j++) {
              tops.merge(k[0]);
#pragma unroll
              for (int i = 1; i < kAt; i++) k[i - 1] = k[i];
            }
          }
          if (!few) tops.start(__shfl_sync(~0u, sort32(head), a.top - 1));
          for (uint32_t w0 = wf; !few && w0 <= wl; w0 += 32 * kAt) {
            ulonglong2 k[kAt];  // two alternatives of each
#pragma unroll
            for (int j = 0; j < kAt; j++) k[j] = pair_of(w0 + lane + 32 * j, 0);
#pragma unroll 1
            for (int j = 0; j < kAt; j++) {
              ulonglong2 now = k[0];
#pragma unroll
              for (int i = 1; i < kAt; i++) k[i - 1] = k[i];
              for (int i = 2;; i += 2) {
                tops.offer<true>(now.x, a.top);
                tops.offer<false>(now.y, a.top);
                const bool more = i < a.top && now.y > tops.bound;
                if (!__any_sync(~0u, more)) break;
                now = more ? pair_of(w0 + lane + 32 * j, i) : make_ulonglong2(0, 0);
              }
            }
          }
        }
      }
    }
    if (whole) {
      if (st.m == INFINITY) st.s = NAN;  // exp(inf - inf)
      const float log2_s = log2f(st.s), lse = st.m + kLn2 * log2_s;
      if (lane == 0) {
        a.logprob[row] = asked ? word_of_token - lse : 0.f;
        a.entropy[row] = kLn2 * (log2_s - st.w / st.s);
        a.lse[row] = lse;
      }
      if (TOP && lane < a.top) {
        a.top_values[(int64_t)row * a.top + lane] = key_value(tops.list) - lse;
        a.top_ids[(int64_t)row * a.top + lane] = key_index(tops.list);
      }
    }
    at = row_first + t1;
  }
}

// dx = g ([i == token] - p) - h p (y + entropy), y = x - lse, p = exp(y); g counts
// only if a token was asked for, and without it and h dx is 0 even where p is not
// a number. One pass, read and written once; SPAN threads (a block, or a warp) take
// SPAN * 8 * kLpBwdPacks columns of a row of a shard.
constexpr int kLpBwdPacks = 8;  // of a thread

template <typename T, int SPAN>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_bwd_kernel(const __grid_constant__ LogprobBwdArgs a,
                                                                       int tiles) {
  const uint32_t magic = op_start(a.ws);
  constexpr int kLpBwdTile = SPAN * 8 * kLpBwdPacks;
  const unsigned unit = blockIdx.x * (kLpThreads / SPAN) + threadIdx.x / SPAN;
  const unsigned row = unit / (unsigned)tiles, tile = unit % (unsigned)tiles;
  const int rank = blockIdx.y, tid = threadIdx.x % SPAN;
  const int64_t width = a.first[rank + 1] - a.first[rank], c0 = (int64_t)tile * kLpBwdTile;
  if (row >= (unsigned)a.rows || c0 >= width) return;
  const int n = (int)imin(kLpBwdTile, width - c0);
  const T* x = reinterpret_cast<const T*>(a.logits[rank]) + (int64_t)row * a.row_stride[rank] + c0;
  T* dx = reinterpret_cast<T*>(a.dlogits[rank]) + (int64_t)row * a.drow_stride[rank] + c0;
  const float lse = a.lse[row];
  const float h = a.grad_entropy != nullptr ? a.grad_entropy[row] : 0.f;
  const int64_t token = a.tokens[row];
  const bool asked = token >= 0 && token < a.first[a.nranks];
  const float g = asked ? a.grad_logprob[row] : 0.f;
  const bool nothing = !asked && h == 0.f;  // the row's terms are constants: gradient 0, whatever its logits are
  const float base = g + h * a.entropy[row];
  const int64_t at = token - a.first[rank] - c0;
  const int mine = asked && at >= 0 && at < n ? (int)at : -1;
  auto grad = [&](float v) {
    const float y = max_nan(v - lse, kFloorT), d = -exp2_fast(y * kLog2e) * fmaf(h, y, base);
    return nothing ? 0.f : d;
  };
  // rows that share a 16-byte phase go in packs, the ends one by one; others one by one altogether
  const bool together = (((uintptr_t)x ^ (uintptr_t)dx) & 15) == 0;
  const int head = together ? min(n, (int)((16 - ((uintptr_t)x & 15)) & 15) / (int)sizeof(T)) : n;
  if (!op_ready(a.ws, magic)) return;
  const int packs = (n - head) / 8, done = head + packs * 8;
  constexpr int kAhead = 64 / (8 * (int)sizeof(T));
  for (int p0 = 0; p0 < packs; p0 += SPAN * kAhead) {
    Pack8<T> u[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const int p = p0 + i * SPAN + tid;
      if (p < packs) u[i].load_stream(x + head + (int64_t)p * 8);
    }
#pragma unroll
    for (int i = 0; i < kAhead; i++) {
      const int p = p0 + i * SPAN + tid;
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
  for (int i = tid; i < head + n - done; i += SPAN) {
    const int e = i < head ? i : done + i - head;
    from_float(dx + e, grad(to_float(x[e])) + (e == mine ? g : 0.f));
  }
}

// Two partial results of each warp that a launch may have, whatever the rows are.
int64_t token_logprobs_scratch_bytes() { return 2ll * kLpMaxWorkers * kLpPartFloats * (int64_t)sizeof(float); }

cudaError_t launch_token_logprobs(const LogprobArgs& args, cudaStream_t stream) {
  LogprobArgs a = args;
  int64_t widest = 0;
  for (int r = 0; r < a.nranks; r++) widest = imax(widest, a.first[r + 1] - a.first[r]);
  // bf16 (27691 rows of 2 shards of 1224 words: 45 us against 51; shards of 16003 words: 90 against 88). A round of f32 is
  // half as many words and gained nothing.
  const bool narrow = widest <= 8 * kLpTile;
  const void* fn = a.dtype == kF32 ? (a.top > 0 ? (const void*)token_logprobs_kernel<float, true, false>
                                                : (const void*)token_logprobs_kernel<float, false, false>)
                   : narrow        ? (a.top > 0 ? (const void*)token_logprobs_kernel<uint16_t, true, true>
                                                : (const void*)token_logprobs_kernel<uint16_t, false, true>)
                                   : (a.top > 0 ? (const void*)token_logprobs_kernel<uint16_t, true, false>
                                                : (const void*)token_logprobs_kernel<uint16_t, false, false>);
  int resident = 0;
  const cudaError_t e = resident_blocks(fn, kLpThreads, 0, &resident);
  if (e != cudaSuccess) return e;
  for (int r = 0; r < a.nranks; r++)
    a.first_tile[r + 1] = a.first_tile[r] + (int)div_up(a.first[r + 1] - a.first[r], kLpTile);
  const int64_t tiles = (int64_t)a.rows * a.first_tile[a.nranks];
  int64_t grid = imin((int64_t)resident, kLpMaxWorkers / kLpWarps);
  // With alternatives, rows in whole numbers of equal parts where that leaves few warps idle: a cut costs its row
  // another start of the list (2048 rows of 131072 words, in 2 parts each against 2.4: top 20 147 against 175 us, top 5
  // 106 against 109, none 90 against 87).
  const int64_t most = grid * kLpWarps, cuts = imin(most / a.rows, a.first_tile[a.nranks]);
  a.cuts = a.top > 0 && (a.rows * cuts * 5 >= most * 4 || cuts == a.first_tile[a.nranks]) ? (uint32_t)cuts : 0;
  a.workers = a.cuts > 0 ? (uint32_t)(a.rows * cuts) : (uint32_t)imin(most, tiles);
  // More rows than warps stay whole if that leaves the warps few tiles apart, which cost less than the joins of two cut
  // rows a warp (top 5, in us: 10046 rows of 8 tiles 52 against 64, 9000 of 30 112 against 122, 25000 of 16 equal, 16000
  // of 30 205 against 201; none: 27691 of 4 41 against 45, 9000 of 30 equal, 5000 of 10 25 against 23).
  const int64_t idle = (div_up(a.rows, most) * most - a.rows) * a.first_tile[a.nranks];
  a.unit = a.rows >= most && idle <= most * (a.top > 0 ? 12 : 4) ? a.first_tile[a.nranks] : 1;
  a.each = (uint32_t)(tiles / a.unit / a.workers);
  a.more = (uint32_t)(tiles / a.unit % a.workers);
  grid = imin(grid, a.workers);
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs nranks=%d rows=%d vocab=%lld top=%d grid=%lld workers=%u\n", a.nranks,
                 a.rows, (long long)a.first[a.nranks], a.top, (long long)grid, a.workers);
  void* params[] = {&a};
  return launch_op(fn, dim3((unsigned)grid), kLpThreads, 0, stream, params);
}

cudaError_t launch_token_logprobs_bwd(const LogprobBwdArgs& a, cudaStream_t stream) {
  int64_t widest = 0;
  for (int r = 0; r < a.nranks; r++) widest = imax(widest, a.first[r + 1] - a.first[r]);
  // Narrow rows go a warp each, if there are more of them than the SMs hold blocks: 16777 rows of 8 shards of 500 words
  // in bf16 60 us against 242, of 2048 42 against 74, of 6007 44 against 45; wider ones the other way (8192: 42, 41), and
  // so 12 rows of 1500 (2.9, 2.3).
  int device = 0, sms = 0;
  const cudaError_t e = current_device_sms(&device, &sms);
  if (e != cudaSuccess) return e;
  const bool narrow = widest * (a.dtype == kF32 ? 4 : 2) <= 12288 && (int64_t)a.rows * a.nranks > 8 * sms;
  const int span = narrow ? 32 : kLpThreads;
  int tiles = (int)div_up(widest, span * 8 * kLpBwdPacks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: token_logprobs_backward nranks=%d rows=%d vocab=%lld tiles=%d span=%d\n", a.nranks,
                 a.rows, (long long)a.first[a.nranks], tiles, span);
  dim3 grid((unsigned)div_up((int64_t)a.rows * tiles, kLpThreads / span), (unsigned)a.nranks);
  const void* fn = a.dtype == kF32 ? (narrow ? (const void*)token_logprobs_bwd_kernel<float, 32>
                                             : (const void*)token_logprobs_bwd_kernel<float, kLpThreads>)
                                   : (narrow ? (const void*)token_logprobs_bwd_kernel<uint16_t, 32>
                                             : (const void*)token_logprobs_bwd_kernel<uint16_t, kLpThreads>);
  void* params[] = {const_cast<LogprobBwdArgs*>(&a), &tiles};
  return launch_op(fn, grid, kLpThreads, 0, stream, params);
}

}  // namespace rar
