// mk_paged.cu -- the paged key/value cache: new rows rotated, rounded or
// quantised and written into pages (append), positions read back (gather), and
// attention of the newest rows over the pages.
//
// A pool is [page][KV head][slot][head_dim]; position p of sequence b is slot
// p % page_size of page table[b][p / page_size].  A row of head_dim values is
// handled by head_dim / 8 lanes of 8 consecutive values each: 16 bytes of a bf16
// row, 8 of an e4m3 row, so that a row's bytes are read and written by
// neighbouring lanes in whole sectors.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "mk_internal.h"

namespace mk {
namespace {

constexpr int kRowThreads = 256;       // threads per block of append and gather
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126, the smallest scale of a row

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The pool row of position p of sequence b, head h, or -1 where it has none
// (negative, past the table, unmapped page).
__device__ __forceinline__ int pool_row(const mk_paged_kv &kv, int b, int h, long long p) {
  if (p < 0) return -1;
  const long long e = p / kv.page_size;
  if (e >= kv.max_pages) return -1;
  const int page = kv.page_table[static_cast<long long>(b) * kv.max_pages + e];
  if (page < 0 || page >= kv.n_pages) return -1;
  return (page * kv.n_kv_heads + h) * kv.page_size + static_cast<int>(p - e * kv.page_size);
}

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// Eight consecutive values as fp32: 16-byte loads where the operand allows them.
__device__ __forceinline__ void load8(const float *p, int vec, float (&x)[8]) {
  if (vec) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
  }
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int vec, float (&x)[8]) {
  if (vec) {
    unpack8(*reinterpret_cast<const uint4 *>(p), x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(p[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&t);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(float *p, int vec, const float (&x)[8]) {
  if (vec) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = x[i];
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, int vec, const float (&x)[8]) {
  if (vec) {
    *reinterpret_cast<uint4 *>(p) = pack8(x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(x[i]);
  }
}

// Eight e4m3 codes as fp32.
__device__ __forceinline__ void decode8(const uint2 &u, float (&x)[8]) {
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Rotate-half of a row held 8 values a lane: value i pairs with i + HD / 2, which
// the lane HD / 16 away holds.  cs: the position's (cos, sin) of the HD / 2 angles.
template <int HD>
__device__ __forceinline__ void rotate8(float (&x)[8], const float2 *cs, int lane8) {
  constexpr int kLanes = HD / 8;
  const bool low = lane8 < kLanes / 2;
  const float2 *c = cs + 8 * (lane8 % (kLanes / 2));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, x[i], kLanes / 2, kLanes);
    const float2 w = c[i];
    x[i] = low ? x[i] * w.x - other * w.y : x[i] * w.x + other * w.y;
  }
}

// ---------------------------------------------------------------------------
// Append.  Items are (t, head, key or value) rows of sequence blockIdx.y, the
// heads fastest, one group of HD / 8 lanes each.  A key row is rotated in fp32;
// then each value is rounded once: to bf16, or to the e4m3 code of x / scale with
// scale = max(amax / 448, 2^-126) over the row's finite values (half a step of
// e4m3, 2^-4 relative; the division keeps x = amax on the largest code).  Every
// lane of a warp stays in the shuffles; rows without a place are not written.
// Bound by memory: each input byte is read once, each cache byte written once.
// ---------------------------------------------------------------------------
template <int HD, typename TIn, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) kv_append(const __grid_constant__ KvAppend a) {
  pdl_wait();
  pdl_launch();
  constexpr int kLanes = HD / 8;
  const int lane8 = threadIdx.x % kLanes;
  const int rows = a.T * a.kv.n_kv_heads * 2;
  const int item = blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes;
  const int is_v = item < rows ? item % 2 : 0;
  const int h = item / 2 % a.kv.n_kv_heads, t = item / 2 / a.kv.n_kv_heads;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const long long p = static_cast<long long>(a.positions[b]) + t;
    bool on = item < rows && (!a.counts || t < a.counts[b]) && (!a.rope || p < a.rope_len);
    const int row = on ? pool_row(a.kv, b, h, p) : -1;
    on = row >= 0;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (on) {
      const mk_strides &s = is_v ? a.vs : a.ks;
      const TIn *src = static_cast<const TIn *>(is_v ? a.v : a.k) + b * s.seq + t * s.token + h * s.head;
      load8(src + 8 * lane8, a.vec, x);
    }
    if (a.rope) {  // the shuffles run in every lane
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = x[i];
      rotate8<HD>(r, a.rope + (on ? p * (HD / 2) : 0), lane8);
      if (!is_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = r[i];
      }
    }
    void *pool = is_v ? a.kv.v : a.kv.k;
    const long long at = static_cast<long long>(row) * HD + 8 * lane8;
    if constexpr (E4M3) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float m = fabsf(x[i]);
        amax = m < INFINITY ? fmaxf(amax, m) : amax;  // NaN compares false
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o, kLanes));
      const float scale = fmaxf(amax / kE4m3Max, kTinyScale);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] / scale, x[2 * i + 1] / scale),
                                                                __NV_SATFINITE, __NV_E4M3);
        w[i / 2] |= static_cast<uint32_t>(c) << (16 * (i & 1));
      }
      if (on) {
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pool) + at) = make_uint2(w[0], w[1]);
        if (lane8 == 0) (is_v ? a.kv.v_scale : a.kv.k_scale)[row] = scale;
      }
    } else if (on) {
      store8(static_cast<__nv_bfloat16 *>(pool) + at, 1, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Gather.  Items as in append; value = code * scale in fp32, rounded once to the
// output's type; zeros for positions without a place.
// ---------------------------------------------------------------------------
template <int HD, typename TOut, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) kv_gather(const __grid_constant__ KvGather a) {
  pdl_wait();
  pdl_launch();
  constexpr int kLanes = HD / 8;
  const int lane8 = threadIdx.x % kLanes;
  const int rows = a.T * a.kv.n_kv_heads * 2;
  const int item = blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes;
  if (item >= rows) return;
  const int is_v = item % 2, h = item / 2 % a.kv.n_kv_heads, t = item / 2 / a.kv.n_kv_heads;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    if (a.counts && t >= a.counts[b]) continue;
    const int row = pool_row(a.kv, b, h, static_cast<long long>(a.starts[b]) + t);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (row >= 0) {
      const void *pool = is_v ? a.kv.v : a.kv.k;
      const long long at = static_cast<long long>(row) * HD + 8 * lane8;
      if constexpr (E4M3) {
        decode8(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pool) + at), x);
        const float s = (is_v ? a.kv.v_scale : a.kv.k_scale)[row];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= s;
      } else {
        load8(static_cast<const __nv_bfloat16 *>(pool) + at, 1, x);
      }
    }
    const mk_strides &s = is_v ? a.vs : a.ks;
    TOut *dst = static_cast<TOut *>(is_v ? a.v : a.k) + b * s.seq + t * s.token + h * s.head;
    store8(dst + 8 * lane8, a.vec, x);
  }
}

// ---------------------------------------------------------------------------
// Attention of the newest rows, split over the cache and joined.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(s_rj - m_r),
//   s_rj = (q_r . k_j) scale log2(e)   (times the key's scale in an 8-bit cache)
//
// with m_r a running reference of the row's scores: sums taken under an older
// one are multiplied by 2^(old - new), so one pass over the cache is enough.
//
// Work.  An item is (sequence, KV head, group of up to 8 NT query rows r = t G + g
// of that head); its cache is cut into units of 16 positions.  The units of all
// items are numbered in one line, and each block takes an equal share of it
// (the lengths live on the device, so every block counts them itself): ragged
// batches and single long sequences load all SMs alike.  An item that lies in
// one block is finished there; of one that does not, each block leaves its
// unnormalised sums and their reference, and the last to arrive (a counter per
// item) joins them in the order of the blocks, so that the result does not
// depend on who was last.
//
// A unit is one warp's: S^T = K Q^T and O^T += V^T P^T on mma.sync, positions and
// then head dimensions as M = 16, query rows as N = 8.  Decoding has few rows, so a
// product that put them at M = 16 or 128 would mostly multiply padding; the
// operands need no shared memory, since the sums over k may run in any order:
// each lane takes 16-byte pieces of the K rows that it owns in the fragment
// (64 contiguous bytes of a row a load) and of V rows (128 bytes a load), two
// positions' values are interleaved by byte permutes, and P^T is turned from the
// first product's layout into the second's by movmatrix.  Loads go straight from
// memory into registers, a whole unit (8 KB of a bf16 cache) at a time per warp.
//
// Exactness.  bf16 rows and codes are exact operands.  A query value enters as
// NQ pieces (bf16 cache: 3 truncated bf16 pieces are the fp32 value itself; codes:
// 2 fp16 pieces of the row divided by a power of two, 2^-24 of the value), a
// weight as 3 truncated bf16 pieces, again the value itself; with bf16 rows in and
// out two pieces (2^-16 of it) are well under the output's rounding of 2^-8.
// Everything else is fp32.
// ---------------------------------------------------------------------------
constexpr int kAtWarps = 4;
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kUnit = 16;          // positions per unit
constexpr float kLazy = 8.0f;      // a score may pass its row's reference by 2^8 before it is moved
constexpr int kAtMaxBlocks = 3;    // resident blocks per SM, at most
constexpr int kMinUnits = 8;       // units per block, at least: two a warp
constexpr int kJoin = 16;          // blocks of an item joined by one; more are joined in two levels

template <int HD, bool E4M3>
struct Geo {
  static constexpr int kBytes = E4M3 ? 1 : 2;
  static constexpr int KS = HD / 16;                    // k steps of S^T, m tiles of O^T
  static constexpr int KW = HD * kBytes / 16;           // 32-bit words of a K row per lane (4 lanes a row)
  static constexpr int VW = HD * kBytes / 32;           // of a V row (8 lanes a row)
  static constexpr int EC = E4M3 ? (HD == 128 ? 16 : 8) : 8;  // dims of a V piece
  // head dimension of element e of the V pieces of lane group g
  static __device__ __forceinline__ int dim(int g, int e) { return (e / EC * 8 + g) * EC + e % EC; }
  // first of the four head dimensions that lane column c holds in k step ks
  static __device__ __forceinline__ int kdim(int ks, int c) {
    return E4M3 ? 64 * (ks / 4) + 16 * c + 4 * (ks % 4) : 32 * (ks / 2) + 8 * c + 4 * (ks % 2);
  }
};

// TIO: the rows' type; NT: query rows of a block / 8.
template <int HD, typename TIO, bool E4M3, int NT>
struct AtShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int NQ = E4M3 ? 2 : sizeof(TIO) == 4 ? 3 : 2;
  static constexpr int NP = sizeof(TIO) == 4 ? 3 : 2;
  static constexpr int kQBytes = Geo<HD, E4M3>::KS * NQ * NT * 32 * 8;      // fragments of Q^T
  static constexpr int kStage = kRows * HD * 4;                             // rotated q, fp32
  static constexpr int kLd = HD + 2;                                        // row stride of the warps' sums
  static constexpr int kMerge = kAtWarps * kRows * kLd * 4;
  static constexpr int kSmem = kMerge > kQBytes + kStage ? kMerge : kQBytes + kStage;
  static constexpr int kBlocks = NT == 1 ? 3 : 2;                           // resident per SM
};

struct AttnArgs {
  PagedAttn a;
  int G, R, n_rg;            // query heads of a KV head, rows of a KV head, row groups
  uint32_t magic, shift;     // p / page_size = (p * magic) >> shift for 0 <= p < 2^31
  int cap;                   // positions of a page table's row
  float qscale;              // scale * log2(e)
  float *part;               // [2 * blocks][kRows][HD] sums
  float2 *part_ml;           // [2 * blocks][kRows] (reference, sum of weights)
  uint32_t *count;           // [blocks] per item, then [2 * blocks] per group of the first level
};

__device__ __forceinline__ uint4 ld_cache(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_cache(const uint2 *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes (low 16 bits) to fp16x2, and that to bf16x2 (both exact).
__device__ __forceinline__ uint32_t codes_f16(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t f16_bf16(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// The pair (x, y) as N bf16x2 words whose values add up to it: truncated pieces for
// N = 3 (all 24 bits), a rounded and a rounded rest for N = 2 (2^-17).
template <int N>
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t (&w)[N]) {
  if constexpr (N == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      w[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
      x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
      y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    }
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w[0] = *reinterpret_cast<const uint32_t *>(&h);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
    w[1] = *reinterpret_cast<const uint32_t *>(&l);
  }
}

__device__ __forceinline__ void split_f16(float x, float y, uint32_t (&w)[2]) {
  const __half2 h = __floats2half2_rn(x, y);
  w[0] = *reinterpret_cast<const uint32_t *>(&h);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  w[1] = *reinterpret_cast<const uint32_t *>(&l);
}

struct Item {
  int b, rg, h;      // sequence, row group, KV head
  int len, cost;     // positions to visit, units
};

__device__ __forceinline__ int seq_rows(const PagedAttn &a, int b) {
  return a.counts ? max(0, min(a.counts[b], a.T)) : a.T;
}

// Positions that row group rg of sequence b visits (-1: it has no rows).
__device__ __forceinline__ int group_len(const AttnArgs &p, int rows, int b, int rg) {
  const int n = seq_rows(p.a, b), t0 = rg * rows / p.G;
  if (t0 >= n) return -1;
  const int t1 = min((min(p.R, (rg + 1) * rows) - 1) / p.G, n - 1);
  const long long len = static_cast<long long>(p.a.positions[b]) + t1 + 1;
  return static_cast<int>(max(0ll, min(len, static_cast<long long>(p.cap))));
}

__device__ __forceinline__ int units_of(int len) { return len < 0 ? 0 : max(1, (len + kUnit - 1) / kUnit); }

__device__ __forceinline__ long long seq_units(const AttnArgs &p, int rows, int b) {
  long long n = 0;
  for (int rg = 0; rg < p.n_rg; ++rg) n += units_of(group_len(p, rows, b, rg));
  return n * p.a.kv.n_kv_heads;
}

template <int HD, typename TIO, bool E4M3, int NT>
__global__ void __launch_bounds__(kAtThreads, (AtShape<HD, TIO, E4M3, NT>::kBlocks))
paged_attn(const __grid_constant__ AttnArgs p) {
  using S = AtShape<HD, TIO, E4M3, NT>;
  using X = Geo<HD, E4M3>;
  constexpr int kRows = S::kRows, NQ = S::NQ, NP = S::NP, KS = X::KS, KW = X::KW, VW = X::VW, kLd = S::kLd;
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ long long s_scan[kAtWarps];
  __shared__ long long s_at;
  __shared__ int s_b;
  __shared__ float s_f[kRows];                  // factor of a row's scores
  __shared__ int s_lim[kRows];                  // last position a row sees, -1: none
  __shared__ float s_m[kAtWarps][kRows], s_l[kAtWarps][kRows];
  __shared__ float s_M[kRows], s_L[kRows];
  __shared__ uint32_t s_last;
  uint2 *qfrag = reinterpret_cast<uint2 *>(dyn);
  float *stage = reinterpret_cast<float *>(dyn + S::kQBytes);
  float *merge = reinterpret_cast<float *>(dyn);
  const PagedAttn &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch();

  // ---- this block's share of the units, and the sequence that holds its first ------------
  // inclusive sum of n over the block's threads, and over all of them
  auto block_scan = [&](long long n, long long &all) {
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) {
      if (w < warp) incl += s_scan[w];
      all += s_scan[w];
    }
    return incl;
  };
  long long total = 0, n = 0, incl = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAtThreads) {
    long long all;
    n = b0 + tid < a.B ? seq_units(p, kRows, b0 + tid) : 0;
    incl = block_scan(n, all);
    total += all;
  }
  if (total == 0) return;
  const long long nb = min(static_cast<long long>(gridDim.x), (total + kMinUnits - 1) / kMinUnits);
  if (blockIdx.x >= nb) return;
  const long long u0 = blockIdx.x * total / nb, u1 = (blockIdx.x + 1) * total / nb;
  auto block_of = [&](long long u) { return static_cast<int>(((u + 1) * nb - 1) / total); };
  if (tid == 0) s_b = -1;
  __syncthreads();
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kAtThreads) {
    if (a.B > kAtThreads) {  // else n and incl are still those of the only pass
      long long all;
      n = b0 + tid < a.B ? seq_units(p, kRows, b0 + tid) : 0;
      incl = block_scan(n, all) + base;
      base += all;
    }
    if (n > 0 && incl - n <= u0 && u0 < incl) {
      s_b = b0 + tid;
      s_at = incl - n;
    }
    __syncthreads();
    if (s_b >= 0) break;
  }
  int b = s_b, rg = 0, h = 0;
  long long at = s_at;  // first unit of item (b, rg, h)

  for (long long u = u0; u < u1;) {
    // the item that holds unit u: row groups in order, each with all KV heads
    int len = group_len(p, kRows, b, rg);
    int cost = units_of(len);
    while (at + cost <= u) {
      at += cost;
      if (cost == 0 || ++h == a.kv.n_kv_heads) {
        h = 0;
        if (++rg == p.n_rg) {
          rg = 0;
          ++b;
        }
        len = group_len(p, kRows, b, rg);
        cost = units_of(len);
      }
    }
    const int seg0 = static_cast<int>(u - at), seg1 = static_cast<int>(min(u1 - at, static_cast<long long>(cost)));
    const bool whole = seg0 == 0 && seg1 == cost;
    const int pos = a.positions[b], n_rows = seq_rows(a, b), r0 = rg * kRows;

    // ---- loads of a unit, a whole one ahead of its products ------------------------------
    const int32_t *table = a.kv.page_table + static_cast<long long>(b) * a.kv.max_pages;
    const long long all_see = static_cast<long long>(pos) + r0 / p.G;  // last position that every row sees
    // pool row of position 16 unit + lane % 16, or -1
    auto row_at = [&](int unit) {
      const int q = unit * kUnit + (lane & 15);
      if (unit >= seg1 || q >= len) return -1;
      const int e = static_cast<int>((static_cast<unsigned long long>(q) * p.magic) >> p.shift);
      const int page = table[e];
      if (page < 0 || page >= a.kv.n_pages) return -1;
      return (page * a.kv.n_kv_heads + h) * a.kv.page_size + (q - e * a.kv.page_size);
    };
    uint32_t kw[2][KW], vw[4][VW];
    float ksc = 0.f, vsc = 0.f;  // scales of position lane % 16
    auto load_k = [&](int row) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int r = __shfl_sync(0xffffffffu, row, g + 8 * s);
        const char *src = static_cast<const char *>(a.kv.k) + static_cast<long long>(r) * (HD * X::kBytes);
#pragma unroll
        for (int i = 0; i < KW / 4; ++i) {
          const uint4 x = r >= 0 ? ld_cache(reinterpret_cast<const uint4 *>(src) + i * 4 + c) : make_uint4(0, 0, 0, 0);
          kw[s][4 * i] = x.x; kw[s][4 * i + 1] = x.y; kw[s][4 * i + 2] = x.z; kw[s][4 * i + 3] = x.w;
        }
      }
      if constexpr (E4M3) {
        ksc = row >= 0 ? a.kv.k_scale[row] : 0.f;
        vsc = row >= 0 ? a.kv.v_scale[row] : 0.f;
      }
    };
    auto load_v = [&](int row) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * c + (s & 1) + 8 * (s >> 1));
        const char *src = static_cast<const char *>(a.kv.v) + static_cast<long long>(r) * (HD * X::kBytes);
        if constexpr (VW >= 4) {
#pragma unroll
          for (int i = 0; i < VW / 4; ++i) {
            const uint4 x = r >= 0 ? ld_cache(reinterpret_cast<const uint4 *>(src) + i * 8 + g) : make_uint4(0, 0, 0, 0);
            vw[s][4 * i] = x.x; vw[s][4 * i + 1] = x.y; vw[s][4 * i + 2] = x.z; vw[s][4 * i + 3] = x.w;
          }
        } else {
          const uint2 x = r >= 0 ? ld_cache(reinterpret_cast<const uint2 *>(src) + g) : make_uint2(0, 0);
          vw[s][0] = x.x; vw[s][1] = x.y;
        }
      }
    };
    int row = row_at(seg0 + warp), next = row_at(seg0 + warp + kAtWarps);
    load_k(row);
    load_v(row);

    // ---- Q: rotated, in pieces, in the layout of the product's B operand -----------------
    __syncthreads();  // the last item's shared memory is free
    {
      constexpr int kPerRow = kAtThreads / kRows, kPairs = HD / 2 / kPerRow;
      const int r = tid / kPerRow, part = tid % kPerRow;  // pairs part, part + kPerRow, .. of row r
      const int t = (r0 + r) / p.G, hq = h * p.G + (r0 + r) % p.G;
      const long long at_p = static_cast<long long>(pos) + t;
      const bool on = r0 + r < p.R && t < n_rows && at_p >= 0 && (!a.rope || at_p < a.rope_len);
      const TIO *q = static_cast<const TIO *>(a.q) + b * a.qs.seq + t * a.qs.token + hq * a.qs.head;
      float x[kPairs], y[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        x[i] = on ? to_f(q[part + kPerRow * i]) : 0.f;
        y[i] = on ? to_f(q[part + kPerRow * i + HD / 2]) : 0.f;
      }
      if (a.rope && on) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 w = a.rope[at_p * (HD / 2) + part + kPerRow * i];
          const float lo = x[i], hi = y[i];
          x[i] = lo * w.x - hi * w.y;
          y[i] = hi * w.x + lo * w.y;
        }
      }
      float f = p.qscale;
      if constexpr (E4M3) {  // a power of two takes the row's largest value to [2^10, 2^11)
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) m = fmaxf(m, fmaxf(fabsf(x[i]), fabsf(y[i])));
#pragma unroll
        for (int o = kPerRow / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = m < INFINITY ? max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100) : 0;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          x[i] = ldexpf(x[i], 10 - e);
          y[i] = ldexpf(y[i], 10 - e);
        }
        f = ldexpf(f, e - 10);
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        stage[r * HD + part + kPerRow * i] = x[i];
        stage[r * HD + part + kPerRow * i + HD / 2] = y[i];
      }
      if (part == 0) {
        s_f[r] = f;
        s_lim[r] = on ? static_cast<int>(min(at_p, 0x7fffffffll)) : -1;
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < KS * NT * 32; i += kAtThreads) {
      const int l = i % 32, n = i / 32 % NT, ks = i / 32 / NT;
      const float4 s = *reinterpret_cast<const float4 *>(stage + (8 * n + l / 4) * HD + X::kdim(ks, l % 4));
      uint32_t w0[NQ], w1[NQ];
      if constexpr (E4M3) {
        split_f16(s.x, s.y, w0);
        split_f16(s.z, s.w, w1);
      } else {
        split_bf16<NQ>(s.x, s.y, w0);
        split_bf16<NQ>(s.z, s.w, w1);
      }
#pragma unroll
      for (int k = 0; k < NQ; ++k) qfrag[((ks * NT + n) * NQ + k) * 32 + l] = make_uint2(w0[k], w1[k]);
    }
    __syncthreads();

    // ---- the warp's units ---------------------------------------------------------------
    float acc[KS][NT][4], m[NT][2], l[NT][2], f[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[n][j] = -INFINITY;
        l[n][j] = 0.f;
        f[n][j] = s_f[8 * n + 2 * c + j];
      }
#pragma unroll
      for (int t = 0; t < KS; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][n][j] = 0.f;
    }
    for (int unit = seg0 + warp; unit < seg1; unit += kAtWarps) {
      const int after = row_at(unit + 2 * kAtWarps);
      const int p0 = unit * kUnit;
      // S^T = K Q^T, one sum per piece of q while there are few tiles: the chains of
      // dependent products are shorter
      constexpr int kSums = NT <= 2 ? NQ : 1;
      float sp[kSums][NT][4];
#pragma unroll
      for (int i = 0; i < kSums; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) sp[i][n][j] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a0, a1, a2, a3;
        if constexpr (E4M3) {
          a0 = codes_f16(kw[0][k] & 0xffffu);
          a1 = codes_f16(kw[1][k] & 0xffffu);
          a2 = codes_f16(kw[0][k] >> 16);
          a3 = codes_f16(kw[1][k] >> 16);
        } else {
          a0 = kw[0][2 * k];
          a1 = kw[1][2 * k];
          a2 = kw[0][2 * k + 1];
          a3 = kw[1][2 * k + 1];
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 q = qfrag[((k * NT + n) * NQ + i) * 32 + lane];
            mma<E4M3>(sp[i % kSums][n], a0, a1, a2, a3, q.x, q.y);
          }
      }
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[n][j] = sp[kSums - 1][n][j];
#pragma unroll
          for (int i = kSums - 2; i >= 0; --i) s[n][j] += sp[i][n][j];
        }
      float ks_[2] = {1.f, 1.f}, vs_[2] = {1.f, 1.f};
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ks_[i] = __shfl_sync(0xffffffffu, ksc, g + 8 * i);
          vs_[i] = __shfl_sync(0xffffffffu, vsc, g + 8 * i);
        }
      }
      load_k(next);  // in flight through the softmax and the second product

      // scores (element j: position g + 8 (j / 2), row 2 c + j % 2 of tile n); masks
      const bool held = __all_sync(0xffffffffu, row >= 0);
      const bool full = held && p0 + kUnit - 1 <= all_see;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] *= E4M3 ? f[n][j & 1] * ks_[j >> 1] : f[n][j & 1];
      if (!full) {
        const int rj[2] = {__shfl_sync(0xffffffffu, row, g), __shfl_sync(0xffffffffu, row, g + 8)};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (rj[j >> 1] < 0 || p0 + g + 8 * (j >> 1) > s_lim[8 * n + 2 * c + (j & 1)]) s[n][j] = -INFINITY;
      }
      // the rows' references, moved where a score passes one by more than kLazy
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) over = over || s[n][j] > m[n][j & 1] + kLazy;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[n][j], s[n][j + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float to = fmaxf(m[n][j], x);
            const float by = to == -INFINITY ? 1.f : ex2(m[n][j] - to);
            m[n][j] = to;
            l[n][j] *= by;
#pragma unroll
            for (int t = 0; t < KS; ++t) {
              acc[t][n][j] *= by;
              acc[t][n][j + 2] *= by;
            }
          }
      }
      // weights; a masked one is zero whatever its value's scale holds
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = s[n][j];
          const float w = x == -INFINITY ? 0.f : ex2(x - m[n][j & 1]);
          l[n][j & 1] += w;
          s[n][j] = !E4M3 || x == -INFINITY ? w : w * vs_[j >> 1];
        }
      if (!full) {
        // V values that only some rows see are multiplied by the others' zero weights:
        // where one is not finite, those positions are added value by value instead.
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const uint32_t x = vw[i][w];
            if (E4M3)
              bad = bad || (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);
            else
              bad = bad || (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
          }
        if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p0 + 2 * c + (i & 1) + 8 * (i >> 1) > all_see)
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[i][w] = 0;
          for (int i = 0; i < kUnit; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, i);
            if (r < 0 || p0 + i <= all_see) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float w[2];
              bool sees[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                w[j] = __shfl_sync(0xffffffffu, i < 8 ? s[n][j] : s[n][j + 2], (i & 7) * 4 + c);
                sees[j] = p0 + i <= s_lim[8 * n + 2 * c + j];
              }
#pragma unroll
              for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const long long o = static_cast<long long>(r) * HD + X::dim(g, 2 * t + e);
                  float v;
                  if constexpr (E4M3) {
                    const uint32_t hv = codes_f16(static_cast<const uint8_t *>(a.kv.v)[o]);
                    v = __half2float(__ushort_as_half(static_cast<unsigned short>(hv)));
                  } else {
                    v = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.kv.v)[o]);
                  }
#pragma unroll
                  for (int j = 0; j < 2; ++j)
                    if (sees[j]) acc[t][n][2 * e + j] = fmaf(w[j], v, acc[t][n][2 * e + j]);
                }
            }
          }
        }
      }

      // O^T += V^T P^T
      uint32_t pb[NT][NP][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[NP];
          split_bf16<NP>(s[n][2 * i], s[n][2 * i + 1], w);
#pragma unroll
          for (int k = 0; k < NP; ++k) pb[n][k][i] = turn8x8(w[k]);
        }
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        uint32_t a0, a1, a2, a3;
        if constexpr (E4M3) {
          const uint32_t sel = t & 1 ? 0x7362 : 0x5140;  // codes 2 t, 2 t + 1 of both positions
          const uint32_t x = __byte_perm(vw[0][t / 2], vw[1][t / 2], sel), y = __byte_perm(vw[2][t / 2], vw[3][t / 2], sel);
          a0 = f16_bf16(codes_f16(x & 0xffffu));
          a1 = f16_bf16(codes_f16(x >> 16));
          a2 = f16_bf16(codes_f16(y & 0xffffu));
          a3 = f16_bf16(codes_f16(y >> 16));
        } else {
          a0 = __byte_perm(vw[0][t], vw[1][t], 0x5410);
          a1 = __byte_perm(vw[0][t], vw[1][t], 0x7632);
          a2 = __byte_perm(vw[2][t], vw[3][t], 0x5410);
          a3 = __byte_perm(vw[2][t], vw[3][t], 0x7632);
        }
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<false>(acc[t][n], a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
      }
      load_v(next);  // in flight through the next first product
      row = next;
      next = after;
    }

    // ---- the warps' sums under one reference, added in the warps' order --------------------
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[n][j];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          s_m[warp][8 * n + 2 * c + j] = m[n][j];
          s_l[warp][8 * n + 2 * c + j] = x;
        }
      }
    __syncthreads();
    if (tid < kRows) {
      float M = s_m[0][tid], L = 0.f;
#pragma unroll
      for (int w = 1; w < kAtWarps; ++w) M = fmaxf(M, s_m[w][tid]);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w)
        if (s_m[w][tid] > -INFINITY) L += s_l[w][tid] * ex2(s_m[w][tid] - M);
        else L += s_l[w][tid];  // zero, or NaN
      s_M[tid] = M;
      s_L[tid] = L;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * n + 2 * c + j;
        const float by = m[n][j] == -INFINITY ? 1.f : ex2(m[n][j] - s_M[r]);
#pragma unroll
        for (int t = 0; t < KS; ++t)  // elements 2 t and 2 t + 1 are neighbouring dimensions
          *reinterpret_cast<float2 *>(merge + (warp * kRows + r) * kLd + X::dim(g, 2 * t)) =
              make_float2(acc[t][n][j] * by, acc[t][n][2 + j] * by);
      }
    }
    __syncthreads();

    // From here on a thread holds pairs of dimensions: pair i of the item's kRows x HD.
    constexpr int kPairsAll = kRows * HD / 2, kPer = kPairsAll / kAtThreads;
    auto finish = [&](int i, float2 x, float L) {
      const int r = i / (HD / 2), d = 2 * (i % (HD / 2));
      const int t = (r0 + r) / p.G, hq = h * p.G + (r0 + r) % p.G;
      if (r0 + r >= p.R || t >= n_rows) return;
      const bool none = s_lim[r] < 0 || L == 0.f;
      const float2 y = none ? make_float2(0.f, 0.f) : make_float2(x.x / L, x.y / L);
      const long long o = ((static_cast<long long>(b) * a.T + t) * a.Hq + hq) * HD + d;
      if constexpr (sizeof(TIO) == 4) {  // a caller's out may start on any element
        static_cast<float *>(a.out)[o] = y.x;
        static_cast<float *>(a.out)[o + 1] = y.y;
      } else {
        static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(y.x);
        static_cast<__nv_bfloat16 *>(a.out)[o + 1] = __float2bfloat16_rn(y.y);
      }
    };
    auto summed = [&](int i) {
      const float *src = merge + i / (HD / 2) * kLd + 2 * (i % (HD / 2));
      float2 x = *reinterpret_cast<const float2 *>(src);
#pragma unroll
      for (int w = 1; w < kAtWarps; ++w) {
        const float2 y = *reinterpret_cast<const float2 *>(src + w * kRows * kLd);
        x.x += y.x;
        x.y += y.y;
      }
      return x;
    };
    if (whole) {
#pragma unroll
      for (int i = tid; i < kPairsAll; i += kAtThreads) finish(i, summed(i), s_L[i / (HD / 2)]);
    } else {
      // ---- this block's part of the item, and the join by the last to leave one ------------
      const int first = block_of(at), last = block_of(at + cost - 1), me = blockIdx.x;
      // slot 1: the item begins in this block; slot 0: it began before
      auto slot_of = [&](int blk) { return 2 * blk + (blk == first); };
      float2 *dst = reinterpret_cast<float2 *>(p.part) + static_cast<long long>(slot_of(me)) * kPairsAll;
#pragma unroll
      for (int i = 0; i < kPer; ++i) __stcg(dst + tid + i * kAtThreads, summed(tid + i * kAtThreads));
      if (tid < kRows) __stcg(p.part_ml + slot_of(me) * kRows + tid, make_float2(s_M[tid], s_L[tid]));
      // joins the parts of blocks b0, b0 + step, .. <= b1 (at most kJoin, or any number
      // on the second level); `out`: into the item's output, else back into b0's part
      auto join = [&](int b0, int b1, int step, bool out) {
        __syncthreads();
        const int parts = (b1 - b0) / step + 1;
        for (int i = tid; i < kRows; i += kAtThreads) {
          float M = -INFINITY, L = 0.f;
#pragma unroll 8
          for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(p.part_ml + slot_of(b0 + k * step) * kRows + i).x);
#pragma unroll 8
          for (int k = 0; k < parts; ++k) {
            const float2 ml = __ldcg(p.part_ml + slot_of(b0 + k * step) * kRows + i);
            L += ml.x == -INFINITY ? ml.y : ml.y * ex2(ml.x - M);
          }
          s_M[i] = M;
          s_L[i] = L;
        }
        __syncthreads();
        float2 x[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
          const int sl = slot_of(b0 + k * step);
          const float2 *src = reinterpret_cast<const float2 *>(p.part) + static_cast<long long>(sl) * kPairsAll;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int r = (tid + i * kAtThreads) / (HD / 2);
            const float mk = __ldcg(p.part_ml + sl * kRows + r).x;
            const float by = mk == -INFINITY ? 1.f : ex2(mk - s_M[r]);
            const float2 y = __ldcg(src + tid + i * kAtThreads);
            x[i].x = fmaf(y.x, by, x[i].x);
            x[i].y = fmaf(y.y, by, x[i].y);
          }
        }
        if (out) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) finish(tid + i * kAtThreads, x[i], s_L[(tid + i * kAtThreads) / (HD / 2)]);
        } else {
          float2 *o = reinterpret_cast<float2 *>(p.part) + static_cast<long long>(slot_of(b0)) * kPairsAll;
          __syncthreads();  // every thread has read b0's reference
#pragma unroll
          for (int i = 0; i < kPer; ++i) __stcg(o + tid + i * kAtThreads, x[i]);
          if (tid < kRows) __stcg(p.part_ml + slot_of(b0) * kRows + tid, make_float2(s_M[tid], s_L[tid]));
        }
      };
      // arrives at a counter of `n`; true in every thread of the block that is last
      auto arrive = [&](uint32_t *counter, uint32_t n) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const uint32_t old = atomicAdd(counter, 1u);
          s_last = old == n - 1;
          if (old == n - 1) *counter = 0;  // for the next call
          __threadfence();
        }
        __syncthreads();
        return s_last != 0;
      };
      const int n = last - first + 1;
      if (n <= kJoin) {
        if (arrive(p.count + first, n)) join(first, last, 1, true);
      } else {
        const int lead = first + (me - first) / kJoin * kJoin, end = min(last, lead + kJoin - 1);
        if (arrive(p.count + gridDim.x + slot_of(lead), end - lead + 1)) {
          join(lead, end, 1, false);
          if (arrive(p.count + first, (n + kJoin - 1) / kJoin)) join(first, last, kJoin, true);
        }
      }
    }
    u = at + seg1;
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args &&...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

dim3 row_grid(const mk_paged_kv &kv, int B, int T) {
  const int per = kRowThreads / (kv.head_dim / 8);
  const unsigned rows = static_cast<unsigned>(T) * kv.n_kv_heads * 2;  // checked to fit by the caller
  return dim3((rows + per - 1) / per, std::min(B, 65535));
}

}  // namespace

cudaError_t launch_kv_append(const KvAppend &a, int in_dtype, cudaStream_t st) {
  const dim3 grid = row_grid(a.kv, a.B, a.T), block(kRowThreads);
  const bool f32 = in_dtype == MK_F32, e4m3 = a.kv.dtype == MK_E4M3;
  if (a.kv.head_dim == 64) {
    if (f32) return e4m3 ? launch(kv_append<64, float, true>, grid, block, 0, st, a)
                         : launch(kv_append<64, float, false>, grid, block, 0, st, a);
    return e4m3 ? launch(kv_append<64, __nv_bfloat16, true>, grid, block, 0, st, a)
                : launch(kv_append<64, __nv_bfloat16, false>, grid, block, 0, st, a);
  }
  if (f32) return e4m3 ? launch(kv_append<128, float, true>, grid, block, 0, st, a)
                       : launch(kv_append<128, float, false>, grid, block, 0, st, a);
  return e4m3 ? launch(kv_append<128, __nv_bfloat16, true>, grid, block, 0, st, a)
              : launch(kv_append<128, __nv_bfloat16, false>, grid, block, 0, st, a);
}

cudaError_t launch_kv_gather(const KvGather &a, int out_dtype, cudaStream_t st) {
  const dim3 grid = row_grid(a.kv, a.B, a.T), block(kRowThreads);
  const bool f32 = out_dtype == MK_F32, e4m3 = a.kv.dtype == MK_E4M3;
  if (a.kv.head_dim == 64) {
    if (f32) return e4m3 ? launch(kv_gather<64, float, true>, grid, block, 0, st, a)
                         : launch(kv_gather<64, float, false>, grid, block, 0, st, a);
    return e4m3 ? launch(kv_gather<64, __nv_bfloat16, true>, grid, block, 0, st, a)
                : launch(kv_gather<64, __nv_bfloat16, false>, grid, block, 0, st, a);
  }
  if (f32) return e4m3 ? launch(kv_gather<128, float, true>, grid, block, 0, st, a)
                       : launch(kv_gather<128, float, false>, grid, block, 0, st, a);
  return e4m3 ? launch(kv_gather<128, __nv_bfloat16, true>, grid, block, 0, st, a)
              : launch(kv_gather<128, __nv_bfloat16, false>, grid, block, 0, st, a);
}

// Workspace: counters (three words per block), then the parts of at most two items per
// block; laid out for the largest grid and the most rows, whatever a call takes.
static size_t count_bytes(int n_sm) { return (sizeof(uint32_t) * 3 * kAtMaxBlocks * static_cast<size_t>(n_sm) + 255) / 256 * 256; }

size_t paged_attention_workspace(int n_sm) {
  // 2 blocks per SM x 2 parts x 32 rows are more than 3 x 2 x 8 and 2 x 2 x 16
  return count_bytes(n_sm) + sizeof(float) * 2 * 2 * static_cast<size_t>(n_sm) * 32 * (128 + 2);
}

template <int HD, typename TIO, bool E4M3, int NT>
static cudaError_t run_attention(AttnArgs &p, void *workspace, int n_sm, cudaStream_t st) {
  using S = AtShape<HD, TIO, E4M3, NT>;
  static_assert(S::kBlocks * S::kRows * 2 <= 2 * 2 * 32 && S::kBlocks <= kAtMaxBlocks, "workspace");
  const int blocks = n_sm * S::kBlocks;
  p.n_rg = (p.R + S::kRows - 1) / S::kRows;
  p.count = static_cast<uint32_t *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + count_bytes(n_sm));
  p.part_ml = reinterpret_cast<float2 *>(p.part + static_cast<size_t>(2) * blocks * S::kRows * HD);
  if (S::kSmem > 46 * 1024) {
    static std::atomic<uint64_t> done{0};  // devices on which the size is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
      e = cudaFuncSetAttribute(paged_attn<HD, TIO, E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    }
  }
  return launch(paged_attn<HD, TIO, E4M3, NT>, dim3(blocks), dim3(kAtThreads), S::kSmem, st, p);
}

template <int HD, typename TIO, bool E4M3>
static cudaError_t run_rows(AttnArgs &p, void *workspace, int n_sm, cudaStream_t st) {
  if (p.R <= 8) return run_attention<HD, TIO, E4M3, 1>(p, workspace, n_sm, st);
  if (p.R <= 16) return run_attention<HD, TIO, E4M3, 2>(p, workspace, n_sm, st);
  return run_attention<HD, TIO, E4M3, 4>(p, workspace, n_sm, st);
}

cudaError_t launch_paged_attention(const PagedAttn &a, int dtype, void *workspace, int n_sm, cudaStream_t st) {
  AttnArgs p{};
  p.a = a;
  p.G = a.Hq / a.kv.n_kv_heads;
  p.R = a.T * p.G;
  const uint32_t d = a.kv.page_size;
  uint32_t l = 0;
  while ((1u << l) < d) ++l;  // d < 2^31
  p.shift = 31 + l;
  p.magic = static_cast<uint32_t>(((1ull << p.shift) + d - 1) / d);
  p.cap = a.kv.max_pages * a.kv.page_size;
  p.qscale = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);  // log2(e)
  const bool f32 = dtype == MK_F32, e4m3 = a.kv.dtype == MK_E4M3;
  if (a.kv.head_dim == 64) {
    if (f32) return e4m3 ? run_rows<64, float, true>(p, workspace, n_sm, st) : run_rows<64, float, false>(p, workspace, n_sm, st);
    return e4m3 ? run_rows<64, __nv_bfloat16, true>(p, workspace, n_sm, st)
                : run_rows<64, __nv_bfloat16, false>(p, workspace, n_sm, st);
  }
  if (f32) return e4m3 ? run_rows<128, float, true>(p, workspace, n_sm, st) : run_rows<128, float, false>(p, workspace, n_sm, st);
  return e4m3 ? run_rows<128, __nv_bfloat16, true>(p, workspace, n_sm, st)
              : run_rows<128, __nv_bfloat16, false>(p, workspace, n_sm, st);
}

}  // namespace mk
