// decode_attention.cu -- attention of one new token per request over a paged
// key-value cache, all virtual ranks in one launch.
//
//   s_t = scale * (q . k_t),  o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
// over the t < len cached tokens of the request, with the running maximum m and
// sum l of the softmax in binary32; lse = m + log l. A request of length 0
// gives o = 0 and lse = -inf. Results over parts of the cache (m, l, o
// unnormalised) join by o = sum_i 2^(m_i - M) o_i, l likewise, M = max m_i.
//
// Every cached element is read once for up to 16 query heads, so the bytes of
// the cache bound the kernel: about 4 flops a byte for 8 query heads in bf16
// against the 250 at which the tensor cores would. So the warp-wide matrix
// instruction does (the tensor pipe is 14% busy at the bound); the fifth
// generation's would want K, V and P staged in shared memory and tensor memory
// for a product of 8 columns.
//
// Split. An item is one (request, rank, key head, group of 8 NT H query heads);
// its tokens form tiles of 64. An item's units are its tiles and, ahead of them, one
// or two for what it costs beside; the units of all items in a row are cut into one
// equal range per resident block, whatever the lengths are, so a block may
// finish one item, do whole ones and start another; the next item's first tile
// and queries are loaded before the last one's results are joined (without the
// queries 159 requests of 8 tokens, 4 key heads of 256 on 2 ranks, f32, took 41 us
// instead of 34.5, 232 of up to 448 as below 148 instead of 143). An item that a cut divides
// is joined by the blocks that arrive last at it, in two levels and in block
// order. A block's four warps take 16 tokens of a tile each with a softmax of
// their own, and join in shared memory at the end of an item.
//
// Registers instead of shared memory. With tokens (not query heads, of which
// there are few) as the rows of the matrix instruction, S^T = K Q^T and
// O^T = V^T P^T take their left operands straight from 16-byte loads: the order
// of the contraction index of S^T and of the rows of O^T is free, so a lane's
// chunk of consecutive elements supplies what its fragments need (for bf16
// V^T one byte permute pairs two tokens). K of the next tile is loaded as soon
// as S^T is done with its registers and V as soon as O^T is, so a warp always
// has about a tile in flight and waits on no barrier.
//
// Measured: 64 requests of up to 16384 tokens, 8 query heads and one key head of
// 128 on each of 8 ranks, bf16, 2.15 GB: 317 us, 6.8 TB/s (1.0 of the measured
// copy). One request of 262145 tokens, 2 key heads: 55 us, 4.9 TB/s; 40 us are the
// bytes, the rest the launch, the chain of lengths, tables and first tiles, and
// two joins. 33 requests of up to 3001 tokens of 80 elements of f32: 33 us, 3.8
// TB/s: the same chain, and three products for one.
#include <cstdio>

#include "op_common.cuh"
#include "rar_launch.h"

namespace rar {

constexpr int kDaWarps = 4;        // warps that share a tile
constexpr int kDaTile = 16 * kDaWarps;  // tokens of a tile
constexpr int kDaMaxBlocks = 912;  // most blocks of a launch: partial results and counters for each
constexpr int kDaJoin = 16;        // partial results that one block joins before it hands on
static_assert(2 * kDaMaxBlocks <= kOpCounters, "two arrival counters per block");

namespace {

// 16 bytes of the cache, or zeros where `live` is false. Volatile, as the matrix
// instructions are: the order in which the loop asks for loads and uses them is
// what keeps a tile in flight.
__device__ __forceinline__ uint4 ldg_cache(const void* p, bool live) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)live));
  return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t tf32_of(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
// x = hi + lo + an error of at most 2^-22 |x|
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = tf32_of(x);
  lo = tf32_of(x - __uint_as_float(hi));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The running softmax of 8 NT query heads over a warp's tokens: query
// 8 nt + 2c + j of the lane (g, c) = (lane / 4, lane % 4) at [nt][j]. l is the
// lane's own part of the sum until the end.
template <int NT>
struct Softmax {
  float m[NT][2], l[NT][2];
};

// Scores (C fragment of S^T: tokens g, g + 8 by queries 2c, 2c + 1) to weights
// 2^(scale2 s - m), scale2 = scale log2(e). The maximum moves only if a score is
// more than 8 above it: weights up to 2^8 lose nothing in binary32, and the
// rescaling of o and the reduction over the lanes are skipped for almost every
// tile. The exponent is one fused operation, rounded once by its own size and
// not by the score's: m's rounding is in every weight alike and cancels.
template <int NT, int MT>
__device__ __forceinline__ void softmax_step(float (&s)[NT][4], float scale2, bool live0, bool live1, Softmax<NT>& st,
                                             float (&o)[MT][NT][4]) {
  auto larger = [&](int nt, int j) {
    return fmaxf(live0 ? s[nt][j] * scale2 : -INFINITY, live1 ? s[nt][2 + j] * scale2 : -INFINITY);
  };
  bool rise = false;
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int j = 0; j < 2; j++) rise |= larger(nt, j) > st.m[nt][j] + 8.f;
  if (__any_sync(~0u, rise)) {
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        float top = larger(nt, j);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        top = fmaxf(top, st.m[nt][j]);
        const float keep = top == -INFINITY ? 1.f : exp2_fast(st.m[nt][j] - top);
        st.m[nt][j] = top;
        st.l[nt][j] *= keep;
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          o[mt][nt][j] *= keep;
          o[mt][nt][2 + j] *= keep;
        }
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const float m = st.m[nt][j] == -INFINITY ? 0.f : st.m[nt][j];  // scores of -inf alone so far: their weights are 0
      s[nt][j] = live0 ? exp2_fast(fmaf(s[nt][j], scale2, -m)) : 0.f;
      s[nt][2 + j] = live1 ? exp2_fast(fmaf(s[nt][2 + j], scale2, -m)) : 0.f;
      st.l[nt][j] += s[nt][j] + s[nt][2 + j];
    }
}

// What a tile needs per type. DP: head_dim rounded up, to 64, 128, 192 or 256,
// binary32 to 96 as well (the chunks past head_dim are zero). Rows are cache rows, -1 for no token.
template <typename T, int DP, int NT>
struct Tile;

template <int DP, int NT>
struct Tile<uint16_t, DP, NT> {
  static constexpr int KC = DP / 32, VC = DP / 64, MT = DP / 16;
  static constexpr int kQueryBytes = NT * KC * 32 * 16;  // B fragments of Q^T in shared memory
  uint4 k[2][KC];  // tokens g, g + 8; elements 32 i + 8 c
  uint4 v[4][VC];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9; elements 64 h + 8 g

  // Piece i of the fragments, 16 bytes of shared memory, from the memory of the query heads.
  using Piece = uint4;
  __device__ __forceinline__ static Piece fetch_queries(int i, const uint16_t* q, int queries, int D) {
    const int lane = i & 31, chunk = (i >> 5) % KC, nt = (i >> 5) / KC;
    const int row = nt * 8 + (lane >> 2), d = chunk * 32 + (lane & 3) * 8;
    return row < queries && d < D ? *reinterpret_cast<const uint4*>(q + (int64_t)row * D + d) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ static uint4 fragment(Piece u) { return u; }
  __device__ __forceinline__ void load_k(const uint16_t* base, int row, int D) {
    const int lane = threadIdx.x & 31, c8 = (lane & 3) * 8;
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int r = __shfl_sync(~0u, row, (lane >> 2) + 8 * t);
      const uint16_t* p = base + (int64_t)r * D + c8;
#pragma unroll
      for (int i = 0; i < KC; i++)
        k[t][i] = ldg_cache(p + 32 * i, r >= 0 && 32 * i + c8 < D);
    }
  }
  __device__ __forceinline__ void load_v(const uint16_t* base, int row, int D) {
    const int lane = threadIdx.x & 31, g8 = (lane >> 2) * 8;
#pragma unroll
    for (int t = 0; t < 4; t++) {
      const int r = __shfl_sync(~0u, row, 2 * (lane & 3) + (t & 1) + 8 * (t >> 1));
      const uint16_t* p = base + (int64_t)r * D + g8;
#pragma unroll
      for (int h = 0; h < VC; h++)
        v[t][h] = ldg_cache(p + 64 * h, r >= 0 && 64 * h + g8 < D);
    }
  }
  __device__ __forceinline__ void scores(const char* smem, float (&s)[NT][4]) const {
    const uint4* q = reinterpret_cast<const uint4*>(smem) + (threadIdx.x & 31);
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KC; i++) {
        const uint4 b = q[(nt * KC + i) * 32];
        mma_bf16(x, k[0][i].x, k[1][i].x, k[0][i].y, k[1][i].y, b.x, b.y);
        mma_bf16(y, k[0][i].z, k[1][i].z, k[0][i].w, k[1][i].w, b.z, b.w);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) s[nt][j] = x[j] + y[j];
    }
  }
  // O^T += V^T P^T. P goes in as a bf16 and the bf16 of its remainder, two
  // instructions: P's own rounding (2^-9) would be as large as the result's. The
  // instruction truncates its sum, by about 2^-23 of it each time: 3e-5 after the
  // 144 tiles that a warp has of 64 requests up to 16384 tokens, where the result's
  // rounding takes up to 2e-3, so here the sum runs on, as the binary32 form's does
  // not. 0.2 to 0.3 % of the results are rounded otherwise than in 64 bits.
  __device__ __forceinline__ void accumulate(const float (&p)[NT][4], float (&o)[MT][NT][4]) const {
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const float a = p[nt][2 * t], b = p[nt][2 * t + 1];
        const uint32_t h = bf16_pair(a, b);
        hi[nt][t] = transpose8x8(h);
        lo[nt][t] = transpose8x8(bf16_pair(a - bf16_lo(h), b - bf16_hi(h)));
      }
#pragma unroll
    for (int h = 0; h < VC; h++) {
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&v[0][h]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&v[1][h]);
      const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&v[2][h]);
      const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&v[3][h]);
#pragma unroll
      for (int jj = 0; jj < 4; jj++) {
        const uint32_t a0 = __byte_perm(w0[jj], w1[jj], 0x5410), a1 = __byte_perm(w0[jj], w1[jj], 0x7632);
        const uint32_t a2 = __byte_perm(w2[jj], w3[jj], 0x5410), a3 = __byte_perm(w2[jj], w3[jj], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          mma_bf16(o[h * 4 + jj][nt], a0, a1, a2, a3, hi[nt][0], hi[nt][1]);
          mma_bf16(o[h * 4 + jj][nt], a0, a1, a2, a3, lo[nt][0], lo[nt][1]);
        }
      }
    }
  }
  // Element of row g (or g + 8) of o's tile mt.
  __device__ __forceinline__ static int dim_of(int mt, int g) { return (mt >> 2) * 64 + g * 8 + (mt & 3) * 2; }
};

// binary32: every operand as the sum of two tf32 values, three products
// (hi hi, hi lo, lo hi); what is left out is below 2^-21 of a product. The
// instruction truncates its sum, which over a chain of them adds up to a bias
// (5.7e-6 of the result after 36 tiles, where the operation in binary32 is
// 1.7e-6 off): so chains are short, and their ends are added with rounding.
template <int DP, int NT>
struct Tile<float, DP, NT> {
  static constexpr int KC = DP / 16, VC = DP / 32, MT = DP / 16;
  static constexpr int kQueryBytes = NT * 2 * KC * 32 * 16;
  float4 k[2][KC];  // tokens g, g + 8; elements 16 i + 4 c
  float4 v[4][VC];  // tokens c, c + 4, c + 8, c + 12; elements 32 h + 4 g

  using Piece = float2;
  __device__ __forceinline__ static Piece fetch_queries(int i, const float* q, int queries, int D) {
    const int lane = i & 31, step = (i >> 5) % (2 * KC), nt = (i >> 5) / (2 * KC);
    const int row = nt * 8 + (lane >> 2), d = (step >> 1) * 16 + (lane & 3) * 4 + (step & 1) * 2;
    return row < queries && d < D ? *reinterpret_cast<const float2*>(q + (int64_t)row * D + d) : make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ static uint4 fragment(Piece x) {
    uint4 u;
    split_tf32(x.x, u.x, u.z);
    split_tf32(x.y, u.y, u.w);
    return u;
  }
  __device__ __forceinline__ static float4 load4(const float* p, bool live) {
    const uint4 u = ldg_cache(p, live);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ __forceinline__ void load_k(const float* base, int row, int D) {
    const int lane = threadIdx.x & 31, c4 = (lane & 3) * 4;
#pragma unroll
    for (int t = 0; t < 2; t++) {
      const int r = __shfl_sync(~0u, row, (lane >> 2) + 8 * t);
      const float* p = base + (int64_t)r * D + c4;
#pragma unroll
      for (int i = 0; i < KC; i++) k[t][i] = load4(p + 16 * i, r >= 0 && 16 * i + c4 < D);
    }
  }
  __device__ __forceinline__ void load_v(const float* base, int row, int D) {
    const int lane = threadIdx.x & 31, g4 = (lane >> 2) * 4;
#pragma unroll
    for (int t = 0; t < 4; t++) {
      const int r = __shfl_sync(~0u, row, (lane & 3) + 4 * t);
      const float* p = base + (int64_t)r * D + g4;
#pragma unroll
      for (int h = 0; h < VC; h++) v[t][h] = load4(p + 32 * h, r >= 0 && 32 * h + g4 < D);
    }
  }
  __device__ __forceinline__ static void fold(float (&x)[NT][4], float (&s)[NT][4]) {
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        s[nt][j] += x[nt][j];
        x[nt][j] = 0.f;
      }
  }
  __device__ __forceinline__ void scores(const char* smem, float (&s)[NT][4]) const {
    const uint4* q = reinterpret_cast<const uint4*>(smem) + (threadIdx.x & 31);
    float x[NT][4] = {}, y[NT][4] = {}, z[NT][4] = {};  // three chains of dependent instructions, not one
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int j = 0; j < 4; j++) s[nt][j] = 0.f;
#pragma unroll
    for (int i = 0; i < KC; i++) {
      if (i % 2 == 0 && i > 0) fold(x, s);
      const float* f0 = reinterpret_cast<const float*>(&k[0][i]);
      const float* f1 = reinterpret_cast<const float*>(&k[1][i]);
#pragma unroll
      for (int e = 0; e < 2; e++) {
        uint32_t h[4], l[4];
        split_tf32(f0[2 * e], h[0], l[0]);
        split_tf32(f1[2 * e], h[1], l[1]);
        split_tf32(f0[2 * e + 1], h[2], l[2]);
        split_tf32(f1[2 * e + 1], h[3], l[3]);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
          const uint4 b = q[(nt * 2 * KC + 2 * i + e) * 32];
          mma_tf32(x[nt], h[0], h[1], h[2], h[3], b.x, b.y);
          mma_tf32(y[nt], h[0], h[1], h[2], h[3], b.z, b.w);
          mma_tf32(z[nt], l[0], l[1], l[2], l[3], b.x, b.y);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int j = 0; j < 4; j++) s[nt][j] += x[nt][j] + (y[nt][j] + z[nt][j]);
  }
  __device__ __forceinline__ void accumulate(const float (&p)[NT][4], float (&o)[MT][NT][4]) const {
    const int lane = threadIdx.x & 31, from = (lane & 3) * 4 + (lane >> 3);
    const bool odd = (lane >> 2) & 1;
    uint32_t ph[NT][2][2], pl[NT][2][2];  // [step of 8 tokens][token c, c + 4] of query g
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float a = __shfl_sync(~0u, p[nt][2 * t], from + 16 * e);
          const float b = __shfl_sync(~0u, p[nt][2 * t + 1], from + 16 * e);
          split_tf32(odd ? b : a, ph[nt][t][e], pl[nt][t][e]);
        }
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int h = 0; h < VC; h++) {
        const float* f0 = reinterpret_cast<const float*>(&v[2 * t][h]);
        const float* f1 = reinterpret_cast<const float*>(&v[2 * t + 1][h]);
#pragma unroll
        for (int jj = 0; jj < 2; jj++) {
          uint32_t a[4], b[4];
          split_tf32(f0[2 * jj], a[0], b[0]);
          split_tf32(f0[2 * jj + 1], a[1], b[1]);
          split_tf32(f1[2 * jj], a[2], b[2]);
          split_tf32(f1[2 * jj + 1], a[3], b[3]);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            float acc[4] = {};
            mma_tf32(acc, b[0], b[1], b[2], b[3], ph[nt][t][0], ph[nt][t][1]);
            mma_tf32(acc, a[0], a[1], a[2], a[3], pl[nt][t][0], pl[nt][t][1]);
            mma_tf32(acc, a[0], a[1], a[2], a[3], ph[nt][t][0], ph[nt][t][1]);
#pragma unroll
            for (int j = 0; j < 4; j++) o[h * 2 + jj][nt][j] += acc[j];
          }
        }
      }
  }
  __device__ __forceinline__ static int dim_of(int mt, int g) { return (mt >> 1) * 32 + g * 4 + (mt & 1) * 2; }
};

}  // namespace

// Whether K and V of a tile (DP elements of T, 16 tokens a warp) fit the
// registers together; else V is loaded when K has been used.
template <typename T, int DP>
constexpr bool kDaAhead = DP * sizeof(T) <= 512;

// Where a block's walk over the tiles stands: kept in shared memory so that the
// loop over tiles has the registers.
struct Part {
  int64_t tile_first;  // unit of the item's first tile
  int request, t0, t1, tiles, len;  // tiles t0..t1 of the item's `tiles`
  int rank, kvh, qg, queries;
};

// The shapes of a kernel. Four warps take 16 tokens of a tile each, H times for
// H groups of 8 NT query heads that read the same tiles at the same time (the
// second from L2).
template <typename T, int DP_, int NT, int H>
struct Shape {
  using Type = T;
  static constexpr int DP = DP_;
  using Tl = Tile<T, DP, NT>;
  static constexpr int kThreads = 32 * kDaWarps * H;
  // Resident blocks that the registers have to leave room for: as many as K, V and the accumulators let, where the rest
  // are temporaries that can wait (left to itself the compiler takes 215 registers at 128 elements of bf16: 329 us
  // against 318 for 64 requests up to 16384 tokens; binary32 at 80: 43 us against 36 for 33 requests).
  static constexpr int kBytes = DP * (int)sizeof(T);  // of a row of K, padded
  static constexpr int kBlocks = H > 1                        ? 1
                                 : kBytes * NT <= 128         ? 4
                                 : kBytes == 256 && DP == 128 ? (NT == 1 ? 3 : 2)
                                 : kBytes <= 256              ? 3
                                 : DP == 96 && NT == 1        ? 3
                                                              : 2;
  static constexpr int Q = NT * 8 * H;           // query heads of an item
  // What an item costs beside its tiles, in tiles: the start and the join of 8 query heads about one (232 requests of up to
  // 448 tokens, 4 key heads of 128 on 8 ranks, bf16: 8 query heads a key head 147 us with one, 150 with 2, 201 with
  // none; 16: 251, 211 and 377).
  static constexpr int kStart = Q / 8;
  static constexpr int kRow = DP + 4;
  static constexpr int kPartial = Q * (DP + 2);  // floats of a partial result: DP values a query, m, l
  static constexpr int kMergeBytes = kDaWarps * Q * kRow * 4, kQueryBytes = H * Tl::kQueryBytes;
  struct Shared {
    alignas(16) char buf[kMergeBytes];
    uint4 queries[kQueryBytes / 16];
    float m[kDaWarps][Q], l[kDaWarps][Q];
    float top[Q], total[Q];
    int64_t tiles[kDaWarps * H];
    Part part[2];  // the one worked on and the one after it
    int last;
  };
};

// Where an item's results go.
template <typename T>
struct Output {
  T* out;
  float* lse;  // null: not wanted
  // four values of a query head, not yet divided by the sum l of the weights 2^(s - m)
  __device__ __forceinline__ void write(int q, int d, int D, float4 x, float m, float l) const {
    const float f = l == 0.f ? 0.f : 1.f / l;  // no token with a weight: 0
    store4(out + (int64_t)q * D + d, x.x * f, x.y * f, x.z * f, x.w * f);
    if (d == 0 && lse != nullptr) lse[q] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
};
template <typename T>
__device__ __forceinline__ Output<T> output_of(const DecodeArgs& a, const Part& p, int q0) {
  Output<T> o;
  o.out = reinterpret_cast<T*>(a.out[p.rank]) + (int64_t)p.request * a.out_stride + (int64_t)q0 * a.head_dim;
  o.lse = a.lse[p.rank] == nullptr ? nullptr : a.lse[p.rank] + (int64_t)p.request * a.q_heads + q0;
  return o;
}

template <typename T, int DP, int NT, int H>
__global__ void __launch_bounds__(Shape<T, DP, NT, H>::kThreads, Shape<T, DP, NT, H>::kBlocks) decode_attention_kernel(
    const __grid_constant__ DecodeArgs a) {
  using S = Shape<T, DP, NT, H>;
  using Tl = Tile<T, DP, NT>;
  constexpr int MT = Tl::MT, Q = S::Q, kRow = S::kRow, kThreads = S::kThreads;
  extern __shared__ __align__(16) char smem[];
  typename S::Shared& sh = *reinterpret_cast<typename S::Shared*>(smem);

  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int warp = tid / 32 % kDaWarps, half = tid / 32 / kDaWarps, block = blockIdx.x;
  const int D = a.head_dim;
  const int longest = a.max_blocks << a.page_shift;
  bool bad = false;
  const uint32_t magic = op_start(a.ws);

  // Tiles of all requests: a segment of requests per thread, then a scan.
  auto length = [&](int b) {
    const int n = a.lens[b];
    return n < 0 ? 0 : n > longest ? longest : n;
  };
  auto tiles_of = [](int n) { return (n + kDaTile - 1) / kDaTile; };
  auto units_of = [&](int n) { return n == 0 ? 0 : S::kStart + tiles_of(n); };
  const int group = a.q_heads / a.kv_heads, qgroups = (group + Q - 1) / Q;
  const int per_request = a.nranks * a.kv_heads * qgroups;  // items of a request
  const int seg = (a.batch + kThreads - 1) / kThreads;
  int64_t before = 0, mine = 0, total = 0;  // units of the requests before the thread's, its own, all
  {
    const int b0 = min(tid * seg, a.batch), b1 = min(b0 + seg, a.batch);
    for (int b = b0; b < b1; b++) {
      const int n = a.lens[b];
      if (n < 0 || n > longest) bad = true;
      mine += units_of(length(b));
    }
    if (!op_ready(a.ws, magic)) return;
    int64_t scan = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, scan, d);
      if (lane >= d) scan += x;
    }
    if (lane == 31) sh.tiles[tid >> 5] = scan;
    __syncthreads();
    before = scan - mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
      if (w < tid >> 5) before += sh.tiles[w];
      total += sh.tiles[w];
    }
    total *= per_request;
  }
  // the first `more` of the blocks with work have each + 1 units, the others each
  const int64_t blocks = total < gridDim.x ? total : gridDim.x, each = blocks == 0 ? 0 : total / blocks;
  const int64_t more = total - each * blocks;
  auto start_of = [&](int64_t w) { return w * each + (w < more ? w : more); };
  auto block_of = [&](int64_t unit) {
    const int64_t split = more * (each + 1);
    return (int)(unit < split ? unit / (each + 1) : more + (unit - split) / each);
  };
  auto place = [&](Part& p, int64_t item_first, int64_t at) {  // tiles of the item that are the block's, from unit `at` on
    const int64_t end = start_of(block + 1);
    p.tile_first = item_first + S::kStart;
    p.t0 = p.t1 = 0;
    if (at >= end || end <= p.tile_first) return;
    p.t0 = (int)(at > p.tile_first ? at - p.tile_first : 0);
    p.t1 = (int)(end - p.tile_first < p.tiles ? end - p.tile_first : p.tiles);
    p.queries = min(Q, group - p.qg * Q);
  };
  if (block < blocks) {
    const int64_t t = start_of(block) / per_request;  // lies in the same request, units counted once per item
    if (t >= before && t < before + mine) {
      int b = tid * seg;
      for (int n; t >= before + (n = units_of(length(b))); b++) before += n;
      Part& p = sh.part[0];
      const int64_t first = before * per_request, at = start_of(block);
      const int n = units_of(length(b)), item = (int)((at - first) / n);
      p.request = b;
      p.len = length(b);
      p.tiles = n - S::kStart;
      p.qg = item % qgroups;
      p.kvh = item / qgroups % a.kv_heads;
      p.rank = item / qgroups / a.kv_heads;
      place(p, first + (int64_t)item * n, at);
    }
  }

  // Requests of length 0, shared out over the blocks.
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (length(b) != 0) continue;
    for (int r = 0; r < a.nranks; r++) {
      T* out = reinterpret_cast<T*>(a.out[r]) + (int64_t)b * a.out_stride;
      for (int i = tid; i < a.q_heads * D; i += kThreads) from_float(out + i, 0.f);
      if (a.lse[r] != nullptr)
        for (int i = tid; i < a.q_heads; i += kThreads) a.lse[r][(int64_t)b * a.q_heads + i] = -INFINITY;
    }
  }
  if (block >= blocks) {
    if (bad) op_report(a.ws, kErrCapacity);
    return;
  }

  // The part that follows `from`: of the next group of query heads, key head, rank or request.
  auto describe_next = [&](Part& p, const Part& from) {
    p.t0 = p.t1 = 0;
    if (from.t1 < from.tiles) return;  // the block's range ends in it
    const int64_t at = from.tile_first + from.tiles;
    if (at >= start_of(block + 1)) return;
    p.request = from.request;
    p.tiles = from.tiles;
    p.len = from.len;
    p.rank = from.rank;
    p.kvh = from.kvh;
    p.qg = from.qg + 1;
    if (p.qg == qgroups) {
      p.qg = 0;
      if (++p.kvh == a.kv_heads) {
        p.kvh = 0;
        if (++p.rank == a.nranks) {
          p.rank = 0;
          do {
            if (++p.request >= a.batch) return;
            p.len = length(p.request);
          } while (p.len == 0);
          p.tiles = tiles_of(p.len);
        }
      }
    }
    place(p, at, at);
  };
  // the lane's token of the warp's 16 in a tile of a part -> cache row
  auto row_of = [&](const Part& p, int tile) {
    const int t = tile * kDaTile + warp * 16 + (lane & 15);
    if (tile >= p.t1 || t >= p.len) return -1;
    const int page = a.table[(int64_t)p.request * a.table_stride + (t >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) {
      bad = true;
      return -1;
    }
    return ((page * a.kv_heads + p.kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
  };
  __syncthreads();
  if (sh.part[0].t1 == 0) {  // the range ends in an item's start
    if (bad) op_report(a.ws, kErrCapacity);
    return;
  }
  Tl tile;
  int row = row_of(sh.part[0], sh.part[0].t0);
  tile.load_k(reinterpret_cast<const T*>(a.k_cache[sh.part[0].rank]), row, D);
  if (kDaAhead<T, DP>) tile.load_v(reinterpret_cast<const T*>(a.v_cache[sh.part[0].rank]), row, D);

  // queries of a part into registers, and from there into shared memory
  constexpr int kPieces = S::kQueryBytes / 16, kEach = (kPieces + kThreads - 1) / kThreads;
  typename Tl::Piece pieces[kEach];
  auto fetch_queries = [&](const Part& p) {
    const T* q = reinterpret_cast<const T*>(a.q[p.rank]) + (int64_t)p.request * a.q_stride + (int64_t)(p.kvh * group + p.qg * Q) * D;
#pragma unroll
    for (int j = 0; j < kEach; j++)
      if (j * kThreads + tid < kPieces) pieces[j] = Tl::fetch_queries(j * kThreads + tid, q, p.queries, D);
  };
  auto put_queries = [&] {
#pragma unroll
    for (int j = 0; j < kEach; j++)
      if (j * kThreads + tid < kPieces) sh.queries[j * kThreads + tid] = Tl::fragment(pieces[j]);
  };
  fetch_queries(sh.part[0]);
  put_queries();

  // At the end of a part the first tile of the next one is on its way already, and so are its queries.
  for (int i = 0;; i ^= 1) {
    const Part& part = sh.part[i];
    Part& after = sh.part[i ^ 1];
    if (tid == 0) describe_next(after, part);
    __syncthreads();
    const int rank = part.rank, t1 = part.t1;
    const T* kc = reinterpret_cast<const T*>(a.k_cache[rank]);
    const T* vc = reinterpret_cast<const T*>(a.v_cache[rank]);
    auto row_at = [&](int t) { return t < t1 ? row_of(part, t) : row_of(after, after.t0 + t - t1); };
    float o[MT][NT][4];
    Softmax<NT> st;
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
#pragma unroll
      for (int j = 0; j < 2; j++) {
        st.m[nt][j] = -INFINITY;
        st.l[nt][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int j = 0; j < 4; j++) o[mt][nt][j] = 0.f;
    }
    {
      int next = row_at(part.t0 + 1);
      const char* queries = reinterpret_cast<const char*>(sh.queries) + half * Tl::kQueryBytes;
      const float scale2 = a.scale * 1.4426950408889634f;
      for (int t = part.t0; t < t1; t++) {
        float s[NT][4];
        // A tile may have no token in the warp's 16. Binary32 has products to save there, and does better with them
        // behind a test altogether (head size 256: 544 us against 595, 128: 142 against 153); bf16 loses 2 %.
        const bool any = sizeof(T) == 2 || __any_sync(~0u, row >= 0);
        if (any) tile.scores(queries, s);
        const bool live0 = __shfl_sync(~0u, row, g) >= 0, live1 = __shfl_sync(~0u, row, g + 8) >= 0;
        if (!kDaAhead<T, DP>) tile.load_v(vc, row, D);
        if (t + 1 == t1 && after.t1 > 0) {
          kc = reinterpret_cast<const T*>(a.k_cache[after.rank]);
          vc = reinterpret_cast<const T*>(a.v_cache[after.rank]);
        }
        if (kDaAhead<T, DP>) tile.load_k(kc, next, D);
        if (any) {
          softmax_step<NT, MT>(s, scale2, live0, live1, st, o);
          tile.accumulate(s, o);
        }
        if (kDaAhead<T, DP>) tile.load_v(vc, next, D);
        else tile.load_k(kc, next, D);
        row = next;
        next = row_at(t + 2);
      }
    }

    // the warps' results of this part of the item join in shared memory
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) st.l[nt][j] += __shfl_xor_sync(~0u, st.l[nt][j], d);
        if (g == 0) {
          sh.m[warp][half * NT * 8 + nt * 8 + 2 * c + j] = st.m[nt][j];
          sh.l[warp][half * NT * 8 + nt * 8 + 2 * c + j] = st.l[nt][j];
        }
      }
    __syncthreads();  // every warp is past the queries, and sh.m is there
    float* s_o = reinterpret_cast<float*>(sh.buf);
#pragma unroll
    for (int nt = 0; nt < NT; nt++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int q = half * NT * 8 + nt * 8 + 2 * c + j;
        float top = sh.m[0][q];
#pragma unroll
        for (int w = 1; w < kDaWarps; w++) top = fmaxf(top, sh.m[w][q]);
        const float f = st.m[nt][j] == -INFINITY ? 0.f : exp2_fast(st.m[nt][j] - top);
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
          float2* p = reinterpret_cast<float2*>(s_o + (warp * Q + q) * kRow + Tl::dim_of(mt, g));
          *p = make_float2(o[mt][nt][j] * f, o[mt][nt][2 + j] * f);
        }
      }
    if (tid < Q) {
      float m = sh.m[0][tid], l = 0.f;
#pragma unroll
      for (int w = 1; w < kDaWarps; w++) m = fmaxf(m, sh.m[w][tid]);
#pragma unroll
      for (int w = 0; w < kDaWarps; w++)  // without a maximum the sum is 0, or NaN if scores are, which shows in the total
        l += sh.m[w][tid] == -INFINITY ? sh.l[w][tid] : sh.l[w][tid] * exp2_fast(sh.m[w][tid] - m);
      sh.top[tid] = m;
      sh.total[tid] = l;
    }
    __syncthreads();
    const int values = part.queries * (DP / 4);
    auto sum4 = [&](int q, int d) {
      float4 x = *reinterpret_cast<const float4*>(s_o + q * kRow + d);
#pragma unroll
      for (int w = 1; w < kDaWarps; w++) {
        const float4 y = *reinterpret_cast<const float4*>(s_o + (w * Q + q) * kRow + d);
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      return x;
    };
    const Output<T> out = output_of<T>(a, part, part.kvh * group + part.qg * Q);
    if (part.t0 == 0 && t1 == part.tiles) {
      if (after.t1 > 0) fetch_queries(after);
      for (int i = tid; i < values; i += kThreads) {
        const int q = i / (DP / 4), d = i % (DP / 4) * 4;
        if (d < D) out.write(q, d, D, sum4(q, d), sh.top[q], sh.total[q]);
      }
    } else {
      // The item is cut: its blocks cf..cl leave partial results, each run of kDaJoin blocks is joined by the one
      // of them that arrives last, and the runs by the last of those, in block order both times.
      float* parts = reinterpret_cast<float*>(a.ws + kOpScratchOffset);
      const int cf = block_of(part.tile_first), cl = block_of(part.tile_first + part.tiles - 1);
      auto part_of = [&](int b) {  // a block leaves up to two: of the item that it goes on with, and of one that it starts
        return parts + (2 * (int64_t)b + (b == cf)) * S::kPartial;
      };
      float* mine_out = part_of(block);
      for (int i = tid; i < values; i += kThreads) {
        const int q = i / (DP / 4), d = i % (DP / 4) * 4;
        *reinterpret_cast<float4*>(mine_out + q * DP + d) = sum4(q, d);
      }
      if (tid < Q) {
        mine_out[Q * DP + tid] = sh.top[tid];
        mine_out[Q * DP + Q + tid] = sh.total[tid];
      }
      uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + kHeaderBytes);
      // a run's counter is that of its last block, which no other item's run ends with
      int from = cf + (block - cf) / kDaJoin * kDaJoin, count = min(kDaJoin, cl + 1 - from), step = 1;
      int counter = from + count - 1;
      for (;;) {
        __syncthreads();
        if (tid == 0) {
          // releases the block's partial result, and acquires the others' if it is the last
          sh.last = atom_add_acq_rel_u32(counters + counter, 1u) == (uint32_t)(count - 1);
          if (sh.last) counters[counter] = 0;
        }
        __syncthreads();
        if (!sh.last) break;
        const bool whole = step > 1 || count == cl + 1 - cf;  // nothing of the item is missing
        float* to = part_of(from);
        // Every thread weighs the partial results of its query head itself, so that all loads of kAt of them are under way
        // at once (4 requests of up to 5000 tokens, 7 query heads of 192: 17 us; 20.6 with the weights shared out first).
        constexpr int kAt = 8;
        for (int i = tid; i < values; i += kThreads) {
          const int q = i / (DP / 4), d = i % (DP / 4) * 4;
          if (d >= D) continue;
          float m = -INFINITY, l = 0.f;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p0 = 0; p0 < count; p0 += kAt) {
            float pm[kAt], pl[kAt];
            float4 y[kAt];
#pragma unroll
            for (int j = 0; j < kAt; j++) {
              pm[j] = -INFINITY;
              pl[j] = 0.f;
              y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (p0 + j < count) {
                const float* src = part_of(from + (p0 + j) * step);
                pm[j] = __ldcg(src + Q * DP + q);
                pl[j] = __ldcg(src + Q * DP + Q + q);
                y[j] = __ldcg(reinterpret_cast<const float4*>(src + q * DP + d));
              }
            }
            float top = m;
#pragma unroll
            for (int j = 0; j < kAt; j++) top = fmaxf(top, pm[j]);
            const float keep = m == -INFINITY ? 0.f : exp2_fast(m - top);
            l *= keep;
            x.x *= keep; x.y *= keep; x.z *= keep; x.w *= keep;
#pragma unroll
            for (int j = 0; j < kAt; j++) {
              const float f = pm[j] == -INFINITY ? 0.f : exp2_fast(pm[j] - top);
              l += f * pl[j];
              x.x += f * y[j].x; x.y += f * y[j].y; x.z += f * y[j].z; x.w += f * y[j].w;
            }
            m = top;
          }
          if (whole) {
            out.write(q, d, D, x, m, l);
          } else {
            *reinterpret_cast<float4*>(to + q * DP + d) = x;
            if (d == 0) {
              sh.top[q] = m;
              sh.total[q] = l;
            }
          }
        }
        if (whole) break;
        __syncthreads();  // every thread has read the weights that are overwritten now
        if (tid < Q) {
          to[Q * DP + tid] = sh.top[tid];
          to[Q * DP + Q + tid] = sh.total[tid];
        }
        step = kDaJoin;
        count = (cl - cf) / kDaJoin + 1;
        from = cf;
        counter = kDaMaxBlocks + cf;  // one item at most starts in a block's range and leaves it
      }
      if (after.t1 > 0) fetch_queries(after);
    }
    if (after.t1 == 0) break;
    put_queries();
    __syncthreads();  // the part's shared values have been read
  }
  if (bad) op_report(a.ws, kErrCapacity);
}

namespace {

struct DecodeKernel {
  const void* fn;
  int threads, shared, partial;  // bytes of shared memory, floats of a partial result
};

template <typename T, int DP, int NT, int H>
DecodeKernel kernel_of() {
  using S = Shape<T, DP, NT, H>;
  return {(const void*)decode_attention_kernel<T, DP, NT, H>, S::kThreads, (int)sizeof(typename S::Shared), S::kPartial};
}

// More than 8 query heads a key head (wide): two accumulators a tile where they
// fit the registers beside K and V. Where they do not, bf16 takes two groups of
// warps (head size 192, 16 heads on 8 ranks, 32 requests of 8192 tokens: 323 us
// against 461 of two passes over the cache; 256: 461 against 614); binary32 is
// bound by its instructions then: two groups take 1025 us against 1011, 1342
// against 1471, and a tenth more for short requests.
template <typename T>
DecodeKernel kernel_for(int head_dim, bool wide) {
  constexpr bool half = sizeof(T) == 2;
  if (head_dim <= 64) return wide ? kernel_of<T, 64, 2, 1>() : kernel_of<T, 64, 1, 1>();
  // the padding that a rounder size brings costs binary32 instructions, of which it has few to spare
  if (!half && head_dim <= 96) return wide ? kernel_of<float, 96, 2, 1>() : kernel_of<float, 96, 1, 1>();
  if (head_dim <= 128) return half && wide ? kernel_of<T, 128, half ? 2 : 1, 1>() : kernel_of<T, 128, 1, 1>();
  if (head_dim <= 192) return half && wide ? kernel_of<T, 192, 1, half ? 2 : 1>() : kernel_of<T, 192, 1, 1>();
  return half && wide ? kernel_of<T, 256, 1, half ? 2 : 1>() : kernel_of<T, 256, 1, 1>();
}
DecodeKernel kernel_for(int dtype, int head_dim, int group) {
  return dtype == kF32 ? kernel_for<float>(head_dim, group > 8) : kernel_for<uint16_t>(head_dim, group > 8);
}

}  // namespace

// Two partial results of each block that a launch may have, whatever the batch is.
int64_t decode_attention_scratch_bytes(int q_heads, int kv_heads, int head_dim) {
  const int group = q_heads / kv_heads;
  return 2ll * kDaMaxBlocks * imax(kernel_for(kF32, head_dim, group).partial, kernel_for(kBF16, head_dim, group).partial) *
         (int64_t)sizeof(float);
}

cudaError_t launch_decode_attention(const DecodeArgs& a, cudaStream_t stream) {
  const DecodeKernel k = kernel_for(a.dtype, a.head_dim, a.q_heads / a.kv_heads);
  int resident = 0;
  const cudaError_t e = resident_blocks(k.fn, k.threads, k.shared, &resident);
  if (e != cudaSuccess) return e;
  const int64_t grid = imin((int64_t)resident, kDaMaxBlocks);
  if (trace_on())
    std::fprintf(stderr, "rar trace: decode_attention nranks=%d batch=%d heads=%d/%d dim=%d grid=%lld threads=%d\n",
                 a.nranks, a.batch, a.q_heads, a.kv_heads, a.head_dim, (long long)grid, k.threads);
  void* params[] = {const_cast<DecodeArgs*>(&a)};
  return launch_op(k.fn, dim3((unsigned)grid), k.threads, k.shared, stream, params);
}

}  // namespace rar
