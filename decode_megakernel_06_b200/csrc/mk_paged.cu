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
// Attention, one block of HD threads per (query head, row): scores of HD
// positions at a time, one a thread, then the running maximum and sum of the
// softmax and thread d's output dimension.
// ---------------------------------------------------------------------------
template <int HD, typename TIO, bool E4M3>
__global__ void __launch_bounds__(HD) paged_attn(const __grid_constant__ PagedAttn a) {
  pdl_wait();
  pdl_launch();
  __shared__ float sq[HD], sp[HD], red[HD / 32];
  __shared__ int srow[HD];
  const int h = blockIdx.x, t = blockIdx.y, d = threadIdx.x, g = h / (a.Hq / a.kv.n_kv_heads);
  for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
    if (a.counts && t >= a.counts[b]) continue;
    const long long p = static_cast<long long>(a.positions[b]) + t;
    const bool on = !a.rope || p < a.rope_len;
    const TIO *q = static_cast<const TIO *>(a.q) + b * a.qs.seq + t * a.qs.token + h * a.qs.head;
    if (on && p >= 0) {
      float x = to_f(q[d]);
      if (a.rope) {
        const float y = to_f(q[d ^ (HD / 2)]);
        const float2 w = a.rope[p * (HD / 2) + d % (HD / 2)];
        x = d < HD / 2 ? x * w.x - y * w.y : x * w.x + y * w.y;
      }
      sq[d] = x * a.scale;
    }
    float m = -INFINITY, l = 0.f, o = 0.f;
    const long long len = on ? min(p + 1, static_cast<long long>(a.kv.max_pages) * a.kv.page_size) : 0;
    for (long long j0 = 0; j0 < len; j0 += HD) {
      __syncthreads();
      const int row = j0 + d < len ? pool_row(a.kv, b, g, j0 + d) : -1;
      float s = -INFINITY;
      if (row >= 0) {
        s = 0.f;
        for (int i = 0; i < HD; i += 8) {
          float x[8];
          if constexpr (E4M3)
            decode8(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.kv.k) + static_cast<long long>(row) * HD + i), x);
          else
            load8(static_cast<const __nv_bfloat16 *>(a.kv.k) + static_cast<long long>(row) * HD + i, 1, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) s = fmaf(sq[i + k], x[k], s);
        }
        if (E4M3) s *= a.kv.k_scale[row];
      }
      srow[d] = row;
      sp[d] = s;
      __syncthreads();
      float mt = m;
      bool any = false;
      for (int j = 0; j < HD; ++j)
        if (srow[j] >= 0) {
          any = true;
          // fmaxf drops NaN: a NaN score makes the row NaN through its p below
          mt = fmaxf(mt, sp[j]);
        }
      if (!any) continue;
      const float c = m == -INFINITY ? 0.f : expf(m - mt);
      o *= c;
      l *= c;
      m = mt;
      for (int j = 0; j < HD; ++j) {
        const int r = srow[j];
        if (r < 0) continue;
        const float pj = expf(sp[j] - m);
        float v;
        if constexpr (E4M3) {
          const __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(a.kv.v)[static_cast<long long>(r) * HD + d], __NV_E4M3);
          v = __half2float(*reinterpret_cast<const __half *>(&hr)) * a.kv.v_scale[r];
        } else {
          v = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.kv.v)[static_cast<long long>(r) * HD + d]);
        }
        l += pj;
        o = fmaf(pj, v, o);
      }
    }
    const float y = l == 0.f ? 0.f : o / l;
    const long long at = ((static_cast<long long>(b) * a.T + t) * a.Hq + h) * HD + d;
    if (sizeof(TIO) == 4) static_cast<float *>(a.out)[at] = y;
    else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
    __syncthreads();
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

size_t paged_attention_workspace(int n_sm) { return static_cast<size_t>(n_sm) * 256; }

cudaError_t launch_paged_attention(const PagedAttn &a, int dtype, void *workspace, cudaStream_t st) {
  (void)workspace;
  const dim3 grid(a.Hq, a.T, std::min(a.B, 65535)), block(a.kv.head_dim);
  const bool f32 = dtype == MK_F32, e4m3 = a.kv.dtype == MK_E4M3;
  if (a.kv.head_dim == 64) {
    if (f32) return e4m3 ? launch(paged_attn<64, float, true>, grid, block, 0, st, a)
                         : launch(paged_attn<64, float, false>, grid, block, 0, st, a);
    return e4m3 ? launch(paged_attn<64, __nv_bfloat16, true>, grid, block, 0, st, a)
                : launch(paged_attn<64, __nv_bfloat16, false>, grid, block, 0, st, a);
  }
  if (f32) return e4m3 ? launch(paged_attn<128, float, true>, grid, block, 0, st, a)
                       : launch(paged_attn<128, float, false>, grid, block, 0, st, a);
  return e4m3 ? launch(paged_attn<128, __nv_bfloat16, true>, grid, block, 0, st, a)
              : launch(paged_attn<128, __nv_bfloat16, false>, grid, block, 0, st, a);
}

}  // namespace mk
