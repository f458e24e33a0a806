// mk_paged.cu -- the paged key/value cache: new rows rotated, rounded or
// quantised and written into pages (append), positions read back (gather), and
// attention of the newest rows over the pages.
//
// A pool is [page][KV head][slot][head_dim]; position p of sequence b is slot
// p % page_size of page table[b][p / page_size].  A row of head_dim values is
// appended by head_dim / 16 lanes and gathered by head_dim / 8, neighbouring lanes
// reading and writing neighbouring bytes in whole sectors.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "mk_internal.h"

namespace mk {
namespace {

constexpr int kRowThreads = 256;       // threads per block of gather
constexpr int kAppendThreads = 128;    // and of append
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyScale = 1.17549435e-38f;  // 2^-126, the smallest scale of a row

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The pool row of position p of sequence b, head h, or -1 where it has none
// (negative, past the table, unmapped page).
__device__ __forceinline__ int pool_row(const mk_paged_kv &kv, int b, int h, long long p) {
  if (p < 0 || p >= static_cast<long long>(kv.max_pages) * kv.page_size) return -1;
  const int at = static_cast<int>(p), e = at / kv.page_size;  // below 2^31, as checked by the caller
  const int page = kv.page_table[static_cast<long long>(b) * kv.max_pages + e];
  if (page < 0 || page >= kv.n_pages) return -1;
  return (page * kv.n_kv_heads + h) * kv.page_size + (at - e * kv.page_size);
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
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

// Stores eight values, the last four of them at p + second (4 with bf16).
__device__ __forceinline__ void store8(float *p, int second, int vec, const float (&x)[8]) {
  if (vec) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + second) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i < 4 ? i : second + i - 4] = x[i];
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, int, int vec, const float (&x)[8]) {
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

// Four consecutive values of a row, kept in their own type until they are used.
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void clear() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p, int vec) {
    if (vec) v = *reinterpret_cast<const float4 *>(p);
    else v = make_float4(p[0], p[1], p[2], p[3]);
  }
  __device__ __forceinline__ float at(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void clear() { v = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int vec) {
    if (vec) {
      v = *reinterpret_cast<const uint2 *>(p);
    } else {
      const uint16_t *u = reinterpret_cast<const uint16_t *>(p);
      v = make_uint2(u[0] | static_cast<uint32_t>(u[1]) << 16, u[2] | static_cast<uint32_t>(u[3]) << 16);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};

// ---------------------------------------------------------------------------
// Append.  A group of HD / 16 lanes takes a token of sequence blockIdx.y and every
// `spread`-th of its KV heads: the place of the token is looked up once, its
// rotary angles are held in registers, and the next head's rows are in flight while
// one's are rounded.  Sixteen values a lane: what is done once per row and lane (the
// largest value, its scale, a reciprocal, addresses) is most of the instructions.  A key
// row is rotated in fp32; then each value is rounded once: to bf16, or to the e4m3 code
// of x / scale with scale = max(amax / 448, 2^-126) over the row's finite values (half a
// step of e4m3, 2^-4 relative; a true quotient keeps x = amax on the largest code).
// Every lane of a warp stays in the shuffles; rows without a place are not written.  Each input byte is read once, each cache byte
// written once: 30.1 us for 135 MB (4.5 TB/s), bound by the instructions of rounding
// and scaling beside the loads' latency.
// ---------------------------------------------------------------------------
constexpr int kHeadsAtOnce = 2;  // heads whose key and value rows a group of a gather loads together

// Eight values of a row in their own type: two fours.
template <typename T>
struct Eight {
  Four<T> lo, hi;
  __device__ __forceinline__ void clear() {
    lo.clear();
    hi.clear();
  }
  __device__ __forceinline__ void load(const T *p, int second, int vec) {  // the last four at p + second; bf16: 4
    if (sizeof(T) == 2 && vec) {  // one 16-byte load
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      set(u);
    } else {
      lo.load(p, vec);
      hi.load(p + second, vec);
    }
  }
  __device__ __forceinline__ void set(const uint4 &u) {
    if constexpr (sizeof(T) == 2) {
      lo.v = make_uint2(u.x, u.y);
      hi.v = make_uint2(u.z, u.w);
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i < 2 ? make_float2(lo.at(2 * i), lo.at(2 * i + 1)) : make_float2(hi.at(2 * i - 4), hi.at(2 * i - 3));
  }
};

// Two fp32 values in one instruction: appending an 8-bit cache is bound by issue slots.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long &>(d))
      : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)),
        "l"(reinterpret_cast<const unsigned long long &>(c)));
  return d;
}

// Rounds a row and writes it at dst (its scale at *scale_at): a lane holds eight
// dimensions of the lower half in x[0 .. 3], the second four kSecond behind the first,
// and those HD / 2 above them in x[4 .. 7].
template <int HD, bool E4M3, int kSecond>
__device__ __forceinline__ void put_row(char *dst, float *scale_at, bool on, float2 (&x)[8], int lane) {
  constexpr int kLanes = HD / 16;
  if constexpr (E4M3) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(fmaxf(amax, fabsf(x[i].x)), fabsf(x[i].y));  // NaN is passed over
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o, kLanes));
    if (__any_sync(0xffffffffu, amax == INFINITY)) {  // the largest finite value; infinities get its code
      float f = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f = fabsf(x[i].x) < INFINITY ? fmaxf(f, fabsf(x[i].x)) : f;
        f = fabsf(x[i].y) < INFINITY ? fmaxf(f, fabsf(x[i].y)) : f;
      }
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, o, kLanes));
      amax = f;
      const float most = fmaxf(f, kE4m3Max * kTinyScale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i].x = fabsf(x[i].x) == INFINITY ? copysignf(most, x[i].x) : x[i].x;
        x[i].y = fabsf(x[i].y) == INFINITY ? copysignf(most, x[i].y) : x[i].y;
      }
    }
    // Quotients a / b: y = a r with r = 1 / b, and its remainder once more, y + r (a - y b)
    // (Markstein, Computation of elementary functions on the IBM RISC System/6000
    // processor, 1990).  For scales of 2^-80 up and the values next to e4m3's midpoints that is
    // the correctly rounded quotient for every mantissa of the scale; below, remainders
    // leave fp32's range, so such a row is first multiplied by a power of two, as its
    // scale is.
    constexpr float k448 = 1.0f / kE4m3Max;
    const float s0 = amax * k448;
    const float scale = fmaxf(fmaf(fmaf(-s0, kE4m3Max, amax), k448, s0), kTinyScale);
    float by = scale;
    constexpr float kSmallRow = 8.2718061255e-25f, kUp = 1.2676506002e30f;  // 2^-80, 2^100
    const bool small = amax > 0.f && amax < kSmallRow;
    if (__any_sync(0xffffffffu, small)) {
      const float up = small ? kUp : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], make_float2(up, up));
      by *= up;
    }
    const float r = __frcp_rn(by);
    const float2 r2 = make_float2(r, r), s2 = make_float2(-by, -by);
    float2 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = mul2(x[i], r2);
      q[i] = fma2(fma2(y, s2, x[i]), r2, y);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(q[2 * i], __NV_SATFINITE, __NV_E4M3)) |
             static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(q[2 * i + 1], __NV_SATFINITE, __NV_E4M3)) << 16;
    if (on) {
      if constexpr (kSecond == 4) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(dst + HD / 2) = make_uint2(w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(dst + i / 2 * (HD / 2) + i % 2 * kSecond) = w[i];
      }
      if (lane == 0) *scale_at = scale;
    }
  } else if (on) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    if constexpr (kSecond == 4) {
      *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(dst + HD) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2 *>(dst + i / 2 * HD + i % 2 * (2 * kSecond)) = make_uint2(w[2 * i], w[2 * i + 1]);
    }
  }
}

// 5 blocks of 128 threads per SM: with bf16 rows 20 warps cover more of the loads' latency than 16
// (8 x up to 4096 rows: 34.8 us into an 8-bit cache and 38.8 into bf16, 30.2 and 33.7 here);
// at 24 registers spill (35.5 and 36.5).  fp32 rows spill at 20 already, 76 to 92 bytes,
// and would be faster at 16 (8 x 2000 rows of 4 heads, 8-bit: 17.9 us against 22.0).
template <int HD, typename TIn, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, 5) kv_append(const __grid_constant__ KvAppend a) {
  pdl_wait();
  pdl_launch();
  constexpr int kLanes = HD / 16;
  // fp32 rows of 128: a lane's dimensions in four quarters of a row, so that a load of 16
  // bytes a lane takes whole sectors (8 x 2000 rows of 4 heads, 8-bit: 22.0 us against
  // 24.5); rows of 64 lose by it, their stores then being of half sectors or of more
  // pieces (16 x up to 1000 rows of 8 heads, bf16: 20.4 against 17.9)
  constexpr bool kQuarters = sizeof(TIn) == 4 && HD == 128;
  constexpr int kAt = kQuarters ? 4 : 8, kSecond = kQuarters ? HD / 4 : 4;
  const int lane = threadIdx.x % kLanes, hkv = a.kv.n_kv_heads;
  const int group = blockIdx.x * (kAppendThreads / kLanes) + threadIdx.x / kLanes;
  const int t = group / a.spread, h0 = group - t * a.spread;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    bool on = t < a.T && (!a.counts || t < a.counts[b]);
    if (!__any_sync(0xffffffffu, on)) continue;
    const long long p = static_cast<long long>(a.positions[b]) + t;
    // this group's next rows to load; read before their place is known
    const long long k_step = a.ks.head * a.spread, v_step = a.vs.head * a.spread;
    const TIn *k = static_cast<const TIn *>(a.k) + b * a.ks.seq + t * a.ks.token + h0 * a.ks.head + kAt * lane;
    const TIn *v = static_cast<const TIn *>(a.v) + b * a.vs.seq + t * a.vs.token + h0 * a.vs.head + kAt * lane;
    const bool has_row = on;
    using Raw = Eight<TIn>[2][2];  // key and value, lower and upper half
    auto load = [&](Raw &raw, int h) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        raw[0][half].clear();
        raw[1][half].clear();
        if (has_row && h < hkv) {
          raw[0][half].load(k + half * (HD / 2), kSecond, a.vec);
          raw[1][half].load(v + half * (HD / 2), kSecond, a.vec);
        }
      }
      k += k_step;
      v += v_step;
    };
    Raw raw;
    load(raw, h0);
    on = on && (!a.rope || p < a.rope_len);
    const int first = on ? pool_row(a.kv, b, 0, p) : -1;  // the row of head 0
    // (cos, cos) and (sin, sin) of this lane's pairs of dimensions i, i + HD / 2
    float2 cos2[4], sin2[4];
    if (a.rope) {
      const float2 *src = a.rope + (on && p >= 0 ? p * (HD / 2) : 0) + kAt * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = i < 2 ? 2 * i : kSecond + 2 * i - 4;
        const float2 u = src[at], w = src[at + 1];
        cos2[i] = make_float2(u.x, w.x);
        sin2[i] = make_float2(u.y, w.y);
      }
    }
    on = first >= 0;
    // where this group's next row goes
    constexpr int kBytes = E4M3 ? 1 : 2;
    long long row = first + static_cast<long long>(h0) * a.kv.page_size;
    const long long row_step = static_cast<long long>(a.spread) * a.kv.page_size;
    char *kd = static_cast<char *>(a.kv.k) + (row * HD + kAt * lane) * kBytes;
    char *vd = static_cast<char *>(a.kv.v) + (row * HD + kAt * lane) * kBytes;
    for (int hb = 0; hb < hkv; hb += a.spread) {  // as often in every lane
      const int h = hb + h0;
      const bool put = on && h < hkv;
      Eight<TIn> kr[2] = {raw[0][0], raw[0][1]}, vr[2] = {raw[1][0], raw[1][1]};
      load(raw, h + a.spread);  // in flight through this turn's rounding
      float2 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = kr[j / 4].pair(j % 4);
      if (a.rope) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = x[j], hi = x[j + 4], minus = make_float2(-sin2[j].x, -sin2[j].y);
          x[j] = fma2(hi, minus, mul2(lo, cos2[j]));
          x[j + 4] = fma2(lo, sin2[j], mul2(hi, cos2[j]));
        }
      }
      put_row<HD, E4M3, kSecond>(kd, a.kv.k_scale + row, put, x, lane);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = vr[j / 4].pair(j % 4);
      put_row<HD, E4M3, kSecond>(vd, a.kv.v_scale + row, put, x, lane);
      row += row_step;
      kd += row_step * (HD * kBytes);
      vd += row_step * (HD * kBytes);
    }
  }
}

// ---------------------------------------------------------------------------
// Gather.  Groups of lanes and heads as in append; value = code * scale in fp32,
// rounded once to the output's type; zeros for positions without a place.  A lane has
// eight neighbouring values, or, where the output is fp32, four of the row's first
// half and four of its second: a store of 16 bytes a lane then covers whole sectors
// (10 x 4000 positions of 2 8-bit heads of 64: 11.5 us against 15.7).
// Bound by memory: 47 us for 271 MB (5.8 TB/s, 88% of the measured copy).
// ---------------------------------------------------------------------------
template <int HD, typename TOut, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) kv_gather(const __grid_constant__ KvGather a) {
  pdl_wait();
  pdl_launch();
  constexpr int kLanes = HD / 8, kWords = E4M3 ? 2 : 4;
  constexpr bool kHalves = sizeof(TOut) == 4;
  constexpr int kAt = kHalves ? 4 : 8, kSecond = kHalves ? HD / 2 : 4;
  const int lane8 = threadIdx.x % kLanes, hkv = a.kv.n_kv_heads;
  const int group = blockIdx.x * (kRowThreads / kLanes) + threadIdx.x / kLanes;
  const int t = group / a.spread, h0 = group - t * a.spread;
  if (t >= a.T) return;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    if (a.counts && t >= a.counts[b]) continue;
    const int first = pool_row(a.kv, b, 0, static_cast<long long>(a.starts[b]) + t);
    TOut *ko = static_cast<TOut *>(a.k) + b * a.ks.seq + t * a.ks.token + kAt * lane8;
    TOut *vo = static_cast<TOut *>(a.v) + b * a.vs.seq + t * a.vs.token + kAt * lane8;
    for (int hb = 0; hb < hkv; hb += kHeadsAtOnce * a.spread) {  // as often in every lane
      uint32_t raw[kHeadsAtOnce][2][kWords];
      float scale[kHeadsAtOnce][2];
#pragma unroll
      for (int i = 0; i < kHeadsAtOnce; ++i)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int h = hb + h0 + i * a.spread;
          const bool on = first >= 0 && h < hkv;
          const long long row = first + static_cast<long long>(h) * a.kv.page_size;
          const char *src = static_cast<const char *>(kv ? a.kv.v : a.kv.k) + (row * HD + kAt * lane8) * (kWords / 2);
          scale[i][kv] = 1.f;
          if constexpr (E4M3) {
            if constexpr (kHalves) {
              raw[i][kv][0] = on ? *reinterpret_cast<const uint32_t *>(src) : 0;
              raw[i][kv][1] = on ? *reinterpret_cast<const uint32_t *>(src + kSecond) : 0;
            } else {
              const uint2 u = on ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0, 0);
              raw[i][kv][0] = u.x; raw[i][kv][1] = u.y;
            }
            if (on) scale[i][kv] = (kv ? a.kv.v_scale : a.kv.k_scale)[row];
          } else if constexpr (kHalves) {
            const uint2 u = on ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0, 0);
            const uint2 w = on ? *reinterpret_cast<const uint2 *>(src + 2 * kSecond) : make_uint2(0, 0);
            raw[i][kv][0] = u.x; raw[i][kv][1] = u.y; raw[i][kv][2] = w.x; raw[i][kv][3] = w.y;
          } else {
            const uint4 u = on ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
            raw[i][kv][0] = u.x; raw[i][kv][1] = u.y; raw[i][kv][2] = u.z; raw[i][kv][3] = u.w;
          }
        }
#pragma unroll
      for (int i = 0; i < kHeadsAtOnce; ++i) {
        const int h = hb + h0 + i * a.spread;
        if (h >= hkv) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          float x[8];
          if constexpr (E4M3) {
            decode8(make_uint2(raw[i][kv][0], raw[i][kv][1]), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= scale[i][kv];
          } else {
            unpack8(make_uint4(raw[i][kv][0], raw[i][kv][1], raw[i][kv][2], raw[i][kv][3]), x);
          }
          store8((kv ? vo + h * a.vs.head : ko + h * a.ks.head), kSecond, a.vec, x);
        }
      }
    }
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
// unnormalised sums and their reference, and the last of eight neighbours to arrive
// (a counter per group) joins theirs in the order of the blocks, then the last of
// eight such groups, so that the result does not depend on who was last.
//
// Measured (B200, 6.56 TB/s copy): 4 caches of 131072, bf16, 32/8 heads of 128: 327 to 340 us,
// 6.3 to 6.6 TB/s; 8 of 4096: 33 us, of which the loads take 20 and the rest is the counting,
// the first pages' chain of loads, the merge and the join; 32 8-bit caches of 512 to 2048:
// 21 us, 8 blocks of 7 rows at 2048: 26 us.  Of these two the units take 9 and 12 us (products,
// conversions, exponentials at 12 warps per SM), the chain before them 6 and 8, the merge,
// the parts and the join after them 4 and 6.
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
// Exactness.  bf16 rows are exact operands, and so are codes in fp16.  With a bf16
// cache a query value and a weight enter as 3 truncated bf16 pieces, which are the
// fp32 value itself; with bf16 rows in and out as two (2^-17 of it), well under the
// output's rounding of 2^-8.  With codes they enter as 2 fp16 pieces, 2^-23 of the
// value or half of fp16's smallest step: queries of the row multiplied by a power of two
// that takes its largest to 2^10 or more, weights times their value's scale under a
// reference that takes the row's largest to 2^6 and keeps it below 2^14.  Everything else is
// fp32; what the tensor cores add, with truncation, is one unit's at most.
// ---------------------------------------------------------------------------
constexpr int kUnit = 16;          // positions per unit
// A score may pass its row's reference by 2^kLazy before the reference is moved (fewer
// moves, and no maximum to find in most units).  In an 8-bit cache the weights times
// their values' scales enter the second product in fp16, so the reference follows the
// scores plus log2(scale): a product is set to 2^kBase at most and may grow to 2^14.
template <bool E4M3>
struct Lazy {
  static constexpr float kLazy = E4M3 ? 14.0f : 8.0f, kBase = E4M3 ? 6.0f : 0.0f;
};
constexpr float kLeastScale = -80.0f;  // log2 of scales below it counts as this: the sums of weights stay finite
constexpr float kLeastValueScale = 8.2718061255e-25f;  // 2^kLeastScale
constexpr int kMinUnits = 8;       // units per block, at least
constexpr int kSecondItem = 32;    // what a second item costs a block, in units
constexpr int kJoinBits = 3;       // parts of an item that one block joins, all their loads in flight; more are
constexpr int kJoin = 1 << kJoinBits;  // joined in levels (one cache of 8192: 51.2 us by 32 at a time, 25.1 by 16, 18.2 by 8)
constexpr int kLevels = 3;
constexpr int kAtMaxBlocks = kJoin * kJoin * kJoin;  // blocks of a grid, at most

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
  // Small blocks leave fewer items cut and overlap one's prologue with another's loop:
  // 27 us against 34 in one block of 12 warps per SM for 32 ragged sequences, 27.8
  // against 29.4 in one of 8 warps with groups of 32 rows for 8 blocks of 7 rows.  As many are
  // resident as registers allow.
  static constexpr int kWarps = 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kBlocks = NT == 1 || E4M3 || HD == 64 ? 3 : 2;
  static constexpr int NQ = E4M3 ? 2 : sizeof(TIO) == 4 ? 3 : 2;
  static constexpr int NP = E4M3 ? 2 : sizeof(TIO) == 4 ? 3 : 2;
  static constexpr int kQBytes = Geo<HD, E4M3>::KS * NQ * NT * 32 * 8;      // fragments of Q^T
  static constexpr int kLdq = HD + 4;                                       // row stride of the rotated q
  static constexpr int kStage = kRows * kLdq * 4;
  static constexpr int kLd = HD + 4;                                        // row stride of the warps' sums
  static constexpr int kMerge = kWarps * kRows * kLd * 4;
  static constexpr int kSmem = kMerge > kQBytes + kStage ? kMerge : kQBytes + kStage;
};

struct Div {  // x / d = (x magic) >> shift for 0 <= x < 2^31
  uint32_t magic, shift;
  __device__ __forceinline__ int of(int x) const {
    return static_cast<int>((static_cast<unsigned long long>(x) * magic) >> shift);
  }
};

struct AttnArgs {
  PagedAttn a;
  int G, R, n_rg;            // query heads of a KV head, rows of a KV head, row groups
  int vec;                   // rows of q start on 16-byte boundaries
  int few;                   // up to 32 sequences of up to 8 row groups each, units below 2^30
  Div by_page, by_G;
  int cap;                   // positions of a page table's row
  float qscale;              // scale * log2(e)
  float4 *part;              // [2 * blocks][kRows][HD / 4] sums
  float2 *part_ml;           // [2 * blocks][kRows] (reference, sum of weights)
  uint32_t *count;           // [kLevels][2 * blocks]: arrivals at a group's first part
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

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes (low 16 bits) to fp16x2: exact.
__device__ __forceinline__ uint32_t codes_f16(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
  return *reinterpret_cast<const uint32_t *>(&h);
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

__device__ __forceinline__ int seq_rows(const PagedAttn &a, int b) {
  return a.counts ? max(0, min(a.counts[b], a.T)) : a.T;
}

// Positions that row group rg of sequence b visits (-1: it has no rows).
__device__ __forceinline__ int group_len(const AttnArgs &p, int rows, int b, int rg) {
  const int n = seq_rows(p.a, b);
  int t0 = 0, t1 = n - 1;
  if (p.n_rg > 1) {
    t0 = p.by_G.of(rg * rows);
    t1 = min(p.by_G.of(min(p.R, (rg + 1) * rows) - 1), t1);
  }
  if (t0 >= n) return -1;
  const long long len = static_cast<long long>(p.a.positions[b]) + t1 + 1;
  return static_cast<int>(max(0ll, min(len, static_cast<long long>(p.cap))));
}

__device__ __forceinline__ int units_of(int len) { return len < 0 ? 0 : max(1, (len + kUnit - 1) / kUnit); }

// Weight of an item of n units when parts hold up to `size`.
__device__ __forceinline__ int weight_of(int n, int size) { return size == 1 ? n : (n + size - 1) / size; }

// The size of the parts.  1: the line of units is cut into equal shares, an item
// wherever one ends, so that many blocks work on two items.  Else each item is cut
// into equal parts, one a block, of the smallest size for which the blocks suffice
// (parts <= units / size + items <= blocks): no block pays for a second prologue, merge
// and join, but the longest part (`longest`: the longest item) sets the time.  Parts
// are taken while that is at most 5/4 of a share and a second item.  Measured, parts
// against shares: 32 sequences of 512 to 2048 20.9 and 24.0 us; 8 x 4096 33.0 and 36.4;
// one of 8192 18.2 and 21.7; 24 of 3000 to 12000 (192 items) 167 and 132; 4 x 131072,
// where a prologue is little beside the loads, 340 and 333 (parts all the same).
template <typename I>
__device__ __forceinline__ int part_size(I units, I items, int longest, int grid) {
  if (items >= grid) return 1;
  const I size = max(static_cast<I>(kMinUnits), (units + grid - items - 1) / (grid - items));
  const I share = units / grid;
  return min(size, static_cast<I>(longest)) <= share + share / 4 + kSecondItem && size < (1 << 26) ? static_cast<int>(size) : 1;
}

// A block's place: weights [u0, u1) of the line, of which sequence b's first is `at`.
// Shares hold `share` weights, the first `more` of them one more.
struct Place {
  long long u0, u1, at, share, more;
  int size, b;  // b < 0: nothing
};

__device__ __forceinline__ void share_out(Place &w, long long line, int grid) {
  const long long nb = min(static_cast<long long>(grid), w.size > 1 ? line : (line + kMinUnits - 1) / kMinUnits);
  w.share = line / max(nb, 1ll);
  w.more = line - w.share * nb;
  w.u0 = blockIdx.x * w.share + min(static_cast<long long>(blockIdx.x), w.more);
  w.u1 = blockIdx.x < nb ? w.u0 + w.share + (blockIdx.x < w.more) : w.u0;
}

// Any number of sequences and row groups; s_scan: kWarps + 2 words of shared memory.
template <int THREADS>
__device__ __noinline__ Place place_of_many(const AttnArgs &p, int rows, long long *s_scan) {
  constexpr int kWarps = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.a.B;
  int longest = 0;
  auto seq_weight = [&](int b, int size) {
    long long n = 0;
#pragma unroll 1
    for (int rg = 0; rg < p.n_rg; ++rg) {
      const int units = units_of(group_len(p, rows, b, rg));
      longest = max(longest, units);
      n += weight_of(units, size);
    }
    return n * p.a.kv.n_kv_heads;
  };
  Place w{};
  w.size = 1;
  w.b = -1;
  long long line = 0;
  // pass 0: the units; 1: the weights, where parts are not single units; 2: the place
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    if (pass == 1) {
      longest = __reduce_max_sync(0xffffffffu, longest);
      __syncthreads();
      if (lane == 0) s_scan[warp] = longest;
      __syncthreads();
      for (int k = 0; k < kWarps; ++k) longest = max(longest, static_cast<int>(s_scan[k]));
      w.size = part_size(line, static_cast<long long>(B) * p.n_rg * p.a.kv.n_kv_heads, longest, gridDim.x);
      if (w.size == 1) continue;
    }
    if (pass == 2) {
      share_out(w, line, gridDim.x);
      if (w.u0 == w.u1) return w;
    }
    long long base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += THREADS) {
      const long long n = b0 + tid < B ? seq_weight(b0 + tid, w.size) : 0;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = incl;
      if (tid == 0) s_scan[kWarps] = -1;
      __syncthreads();
      incl += base;
      for (int k = 0; k < kWarps; ++k) {
        if (k < warp) incl += s_scan[k];
        base += s_scan[k];
      }
      if (pass == 2) {
        if (n > 0 && incl - n <= w.u0 && w.u0 < incl) {
          s_scan[kWarps] = b0 + tid;
          s_scan[kWarps + 1] = incl - n;
        }
        __syncthreads();
        if (s_scan[kWarps] >= 0) {
          w.b = static_cast<int>(s_scan[kWarps]);
          w.at = s_scan[kWarps + 1];
          break;
        }
      }
    }
    if (pass < 2) line = base;
  }
  return w;
}

// Up to 32 sequences of a few row groups each: every warp counts for itself.
__device__ __forceinline__ Place place_of_few(const AttnArgs &p, int rows) {
  const int lane = threadIdx.x & 31, hkv = p.a.kv.n_kv_heads, grid = gridDim.x;
  int longest = 0;
  auto seq_weight = [&](int size) {
    int n = 0;
    if (lane < p.a.B) {
#pragma unroll 1
      for (int rg = 0; rg < p.n_rg; ++rg) {
        const int units = units_of(group_len(p, rows, lane, rg));
        longest = max(longest, units);
        n += weight_of(units, size);
      }
    }
    return n * hkv;
  };
  int n = seq_weight(1);
  int line = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
  Place w{};
  longest = __reduce_max_sync(0xffffffffu, longest);
  w.size = part_size(line, p.a.B * p.n_rg * hkv, longest, grid);
  if (w.size > 1) n = seq_weight(w.size);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  line = __shfl_sync(0xffffffffu, incl, 31);
  const int nb = max(1, min(grid, w.size > 1 ? line : (line + kMinUnits - 1) / kMinUnits)), me = blockIdx.x;
  const int share = w.size > 1 ? 1 : line / nb, more = line - share * nb;
  const int u0 = me * share + min(me, more), u1 = me < nb ? u0 + share + (me < more) : u0;
  const unsigned hit = __ballot_sync(0xffffffffu, u0 < u1 && incl - n <= u0 && u0 < incl);
  w.share = share;
  w.more = more;
  w.u0 = u0;
  w.u1 = u1;
  w.b = hit ? __ffs(hit) - 1 : -1;
  w.at = __shfl_sync(0xffffffffu, incl - n, hit ? w.b : 0);
  return w;
}

// The block whose share holds weight u.
__device__ __noinline__ int block_of(long long u, long long share, long long more) {
  const long long cut = more * (share + 1);
  const bool low = u < cut;
  return static_cast<int>((low ? 0 : more) + (low ? u : u - cut) / (low ? share + 1 : share));
}

template <int HD, typename TIO, bool E4M3, int NT>
__global__ void __launch_bounds__((AtShape<HD, TIO, E4M3, NT>::kThreads), (AtShape<HD, TIO, E4M3, NT>::kBlocks))
paged_attn(const __grid_constant__ AttnArgs p) {
  using S = AtShape<HD, TIO, E4M3, NT>;
  using X = Geo<HD, E4M3>;
  constexpr int kRows = S::kRows, NQ = S::NQ, NP = S::NP, KS = X::KS, KW = X::KW, VW = X::VW, kLd = S::kLd, kLdq = S::kLdq,
                kAtWarps = S::kWarps, kAtThreads = S::kThreads;
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ long long s_scan[kAtWarps + 2];
  __shared__ float s_f[kRows];                  // factor of a row's scores
  __shared__ int s_lim[kRows];                  // last position a row sees, -1: none
  __shared__ float s_m[kAtWarps][kRows], s_l[kAtWarps][kRows];
  __shared__ float s_M[kRows], s_L[kRows];
  __shared__ float s_down[E4M3 ? kAtWarps : 1][kRows];  // of a unit with tiny value scales
  __shared__ long long s_out[kRows];            // first element of a row of the output, -1: no such row
  __shared__ uint32_t s_last;
  __shared__ int s_bad;
  uint2 *qfrag = reinterpret_cast<uint2 *>(dyn);
  float *stage = reinterpret_cast<float *>(dyn + S::kQBytes);
  float *merge = reinterpret_cast<float *>(dyn);
  const PagedAttn &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_launch();

  const Place place = p.few ? place_of_few(p, kRows) : place_of_many<kAtThreads>(p, kRows, s_scan);
  if (place.b < 0) return;
  int b = place.b, rg = 0, h = 0;
  long long at = place.at;  // first weight of item (b, rg, h)

  for (long long u = place.u0; u < place.u1;) {
    // the item that holds weight u: row groups in order, each with all KV heads
    int len = group_len(p, kRows, b, rg);
    int cost = units_of(len), weight = weight_of(cost, place.size);
#pragma unroll 1
    while (at + weight <= u) {
      at += weight;
      if (weight == 0 || ++h == a.kv.n_kv_heads) {
        h = 0;
        if (++rg == p.n_rg) {
          rg = 0;
          ++b;
        }
        len = group_len(p, kRows, b, rg);
        cost = units_of(len);
        weight = weight_of(cost, place.size);
      }
    }
    const int w0 = static_cast<int>(u - at), w1 = static_cast<int>(min(place.u1 - at, static_cast<long long>(weight)));
    // units [seg0, seg1) of the item; parts of equal size
    const bool cut_even = place.size > 1;
    const int seg0 = cut_even ? static_cast<int>(static_cast<long long>(w0) * cost / weight) : w0;
    const int seg1 = cut_even ? static_cast<int>(static_cast<long long>(w1) * cost / weight) : w1;
    const bool whole = seg0 == 0 && seg1 == cost;
    const int pos = a.positions[b], n_rows = seq_rows(a, b), r0 = rg * kRows;

    // ---- loads of a unit, a whole one ahead of its products ------------------------------
    const int32_t *table = a.kv.page_table + static_cast<long long>(b) * a.kv.max_pages;
    const long long all_see = static_cast<long long>(pos) + p.by_G.of(r0);  // last position that every row sees
    // A position's page (-1: none), and its pool row (-1: none) once that is known; the
    // position of a lane is 16 unit + lane % 16.  Selects, no branches: several pages'
    // numbers are then on their way at once.
    auto page_of = [&](int q, bool in) { return in ? table[p.by_page.of(q)] : -1; };
    auto row_of = [&](int q, int page) {
      const unsigned in_page = q - p.by_page.of(q) * a.kv.page_size;
      const unsigned row = (static_cast<unsigned>(page) * a.kv.n_kv_heads + h) * a.kv.page_size + in_page;
      return static_cast<unsigned>(page) < static_cast<unsigned>(a.kv.n_pages) ? static_cast<int>(row) : -1;
    };
    auto page_at = [&](int unit) {
      const int q = unit * kUnit + (lane & 15);
      return page_of(q, unit < seg1 && q < len);
    };
    auto row_at = [&](int unit, int page) { return row_of(unit * kUnit + (lane & 15), page); };
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
    // a unit's rows on their way into L2: lanes 0 .. 15 a key row each, the others a value row
    auto prefetch = [&](int row) {
      if (row < 0) return;
      const char *src = static_cast<const char *>(lane < 16 ? a.kv.k : a.kv.v) + static_cast<long long>(row) * (HD * X::kBytes);
#pragma unroll
      for (int i = 0; i < HD * X::kBytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i));
    };
    const int page0 = page_at(seg0 + warp), page1 = page_at(seg0 + warp + kAtWarps);
    int row, next;

    // ---- Q: rotated, in pieces, in the layout of the product's B operand -----------------
    {
      // lanes part, part + kPerRow, .. of a row hold four pairs of dimensions each
      constexpr int kPerRow = kAtThreads / kRows < HD / 8 ? kAtThreads / kRows : HD / 8, kQuads = HD / 8 / kPerRow;
      const int r = tid / kPerRow, part = tid % kPerRow;
      const bool lane_on = r < kRows;  // HD = 64 leaves half of the threads without a piece
      const int t = p.by_G.of(r0 + r), hq = h * p.G + (r0 + r) - t * p.G;
      const long long at_p = static_cast<long long>(pos) + t;
      const bool is_row = lane_on && r0 + r < p.R && t < n_rows;
      const bool on = is_row && at_p >= 0 && (!a.rope || at_p < a.rope_len);
      const TIO *q = static_cast<const TIO *>(a.q) + b * a.qs.seq + t * a.qs.token + hq * a.qs.head + 4 * part;
      const float2 *cs = a.rope + at_p * (HD / 2) + 4 * part;
      Four<TIO> lo[kQuads], hi[kQuads];
      float2 w[kQuads][4];
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        lo[i].clear();
        hi[i].clear();
        if (on) {
          lo[i].load(q + 4 * kPerRow * i, p.vec);
          hi[i].load(q + 4 * kPerRow * i + HD / 2, p.vec);
          if (a.rope) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = cs[4 * kPerRow * i + j];
          }
        }
      }
      row = row_at(seg0 + warp, page0);  // the queries are on their way
      next = row_at(seg0 + warp + kAtWarps, page1);
      load_k(row);
      load_v(row);
      prefetch(next);
      float x[kQuads][4], y[kQuads][4];
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = lo[i].at(j), v = hi[i].at(j);
          x[i][j] = a.rope && on ? u * w[i][j].x - v * w[i][j].y : u;
          y[i][j] = a.rope && on ? v * w[i][j].x + u * w[i][j].y : v;
        }
      float f = p.qscale;
      if constexpr (E4M3) {  // a power of two takes the row's largest value to [2^10, 2^11)
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(fabsf(x[i][j]), fabsf(y[i][j])));
#pragma unroll
        for (int o = kPerRow / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = m < INFINITY ? max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 10 - e) << 23);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i][j] *= up;
            y[i][j] *= up;
          }
        f *= __uint_as_float(static_cast<uint32_t>(127 + e - 10) << 23);
      }
      __syncthreads();  // the last item's shared memory is free
      if (lane_on) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          float *dst = stage + r * kLdq + 4 * (part + kPerRow * i);
          *reinterpret_cast<float4 *>(dst) = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
          *reinterpret_cast<float4 *>(dst + HD / 2) = make_float4(y[i][0], y[i][1], y[i][2], y[i][3]);
        }
        if (part == 0) {
          s_f[r] = f;
          s_lim[r] = on ? static_cast<int>(min(at_p, 0x7fffffffll)) : -1;
          s_out[r] = is_row ? ((static_cast<long long>(b) * a.T + t) * a.Hq + hq) * HD : -1;
        }
      }
      if (tid == 0) s_bad = 0;
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < KS * NT * 32; i += kAtThreads) {
      const int l = i % 32, n = i / 32 % NT, ks = i / 32 / NT;
      const float4 s = *reinterpret_cast<const float4 *>(stage + (8 * n + l / 4) * kLdq + X::kdim(ks, l % 4));
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
      const int after = row_at(unit + 2 * kAtWarps, page_at(unit + 2 * kAtWarps));
      prefetch(after);
      const int p0 = unit * kUnit;
      // S^T = K Q^T, one sum per piece of q: shorter chains of dependent products
      float sp[NQ][NT][4];
#pragma unroll
      for (int i = 0; i < NQ; ++i)
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
            mma<E4M3>(sp[i][n], a0, a1, a2, a3, q.x, q.y);
          }
      }
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[n][j] = sp[NQ - 1][n][j];
#pragma unroll
          for (int i = NQ - 2; i >= 0; --i) s[n][j] += sp[i][n][j];
        }
      float ks_[2] = {1.f, 1.f}, vs_[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
      const bool small = E4M3 && vsc != 0.f && fabsf(vsc) < kLeastValueScale;
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ks_[i] = __shfl_sync(0xffffffffu, ksc, g + 8 * i);
          vs_[i] = __shfl_sync(0xffffffffu, vsc, g + 8 * i);
          lv[i] = fmaxf(lg2(fabsf(vs_[i])), kLeastScale);
        }
      }
      load_k(next);  // in flight through the softmax and the second product

      // scores (element j: position g + 8 (j / 2), row 2 c + j % 2 of tile n); masks
      const bool full = __all_sync(0xffffffffu, row >= 0 && !small) && p0 + kUnit - 1 <= all_see;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] *= E4M3 ? f[n][j & 1] * ks_[j >> 1] : f[n][j & 1];
      // -inf is a masked score; one that is not masked comes of what is not finite, or lies outside
      // of fp32's range, and makes its row NaN
      const float none = full ? NAN : 0.f;  // the weight of -inf
      if (!full) {
        const int rj[2] = {__shfl_sync(0xffffffffu, row, g), __shfl_sync(0xffffffffu, row, g + 8)};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (s[n][j] == -INFINITY) s[n][j] = NAN;
            if (rj[j >> 1] < 0 || p0 + g + 8 * (j >> 1) > s_lim[8 * n + 2 * c + (j & 1)]) s[n][j] = -INFINITY;
          }
      }
      // the rows' references, moved where a score passes one by more than kLazy
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) over = over || s[n][j] > m[n][j & 1] + (Lazy<E4M3>::kLazy - lv[j >> 1]);
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // an infinite scale of a masked position gives NaN, which fmaxf passes over
            float x = fmaxf(s[n][j] + lv[0], s[n][j + 2] + lv[1]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float to = fmaxf(m[n][j], x - Lazy<E4M3>::kBase);
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
          const float w = x == -INFINITY ? none : ex2(x - m[n][j & 1]);
          l[n][j & 1] += w;
          s[n][j] = !E4M3 || x == -INFINITY ? w : w * vs_[j >> 1];
        }
      // Value scales too small for the reference's clamp: a row's products, and its sums so far,
      // are multiplied by a power of two that takes the unit's largest to 2^6, for the
      // time of the product.  2^46 is what the clamp takes at most; sums stay below 2^54.
      const bool tiny = E4M3 && !full && __any_sync(0xffffffffu, small);
      if (tiny) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(fabsf(s[n][j]), fabsf(s[n][j + 2]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const int bits = x > 0.f ? min(max(6 + 127 - static_cast<int>(__float_as_uint(x) >> 23), 0), 46) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(127 + bits) << 23);
            s[n][j] *= up;
            s[n][j + 2] *= up;
#pragma unroll
            for (int t = 0; t < KS; ++t) {
              acc[t][n][j] *= up;
              acc[t][n][j + 2] *= up;
            }
            if (g == 0) s_down[warp][8 * n + 2 * c + j] = __uint_as_float(static_cast<uint32_t>(127 - bits) << 23);
          }
        __syncwarp();
      }
      if (!full) {
        // V values that only some rows see meet the others' zero weights: one that is not
        // finite is taken out here, and put into the rows that see it below.
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p0 + 2 * c + (i & 1) + 8 * (i >> 1) > all_see)
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              const uint32_t x = vw[i][w];
              uint32_t keep = 0xffffffffu;
              if constexpr (E4M3) {
                const uint32_t nan = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                keep = ~((nan >> 7) * 255u);
              } else {
                if ((x & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                if ((x & 0x7f800000u) == 0x7f800000u) keep &= 0x0000ffffu;
              }
              vw[i][w] = x & keep;
              bad = bad || keep != 0xffffffffu;
            }
        if (bad) s_bad = 1;
      }

      // O^T += V^T P^T
      uint32_t pb[NT][NP][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[NP];
          if constexpr (E4M3) split_f16(s[n][2 * i], s[n][2 * i + 1], w);
          else split_bf16<NP>(s[n][2 * i], s[n][2 * i + 1], w);
#pragma unroll
          for (int k = 0; k < NP; ++k) pb[n][k][i] = turn8x8(w[k]);
        }
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        uint32_t a0, a1, a2, a3;
        if constexpr (E4M3) {
          const uint32_t sel = t & 1 ? 0x7362 : 0x5140;  // codes 2 t, 2 t + 1 of both positions
          const uint32_t x = __byte_perm(vw[0][t / 2], vw[1][t / 2], sel), y = __byte_perm(vw[2][t / 2], vw[3][t / 2], sel);
          a0 = codes_f16(x & 0xffffu);
          a1 = codes_f16(x >> 16);
          a2 = codes_f16(y & 0xffffu);
          a3 = codes_f16(y >> 16);
        } else {
          a0 = __byte_perm(vw[0][t], vw[1][t], 0x5410);
          a1 = __byte_perm(vw[0][t], vw[1][t], 0x7632);
          a2 = __byte_perm(vw[2][t], vw[3][t], 0x5410);
          a3 = __byte_perm(vw[2][t], vw[3][t], 0x7632);
        }
        // The tensor cores' fp32 sums truncate: kept in them over a long cache they fell
        // behind by 8e-8 of the output a unit (7e-6 where 128k positions are split over the
        // GPU, 1.3e-3 over a warp's share of a million).  So each unit's is its own, and added
        // with rounding; 0 to 4% of the time where rows are bf16.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = NP - 1; k >= 0; --k) mma<E4M3>(d, a0, a1, a2, a3, pb[n][k][0], pb[n][k][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[t][n][j] += d[j];
        }
      }
      load_v(next);  // in flight through the next first product
      if (tiny) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float down = s_down[warp][8 * n + 2 * c + (j & 1)];
#pragma unroll
            for (int t = 0; t < KS; ++t) acc[t][n][j] *= down;
          }
      }
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
        for (int t = 0; t < KS; t += 2)  // elements 2 t .. 2 t + 3 are neighbouring dimensions
          *reinterpret_cast<float4 *>(merge + (warp * kRows + r) * kLd + X::dim(g, 2 * t)) =
              make_float4(acc[t][n][j] * by, acc[t][n][2 + j] * by, acc[t + 1][n][j] * by, acc[t + 1][n][2 + j] * by);
      }
    }
    __syncthreads();

    // From here on a thread holds four neighbouring dimensions: piece i of the item's kRows x HD.
    constexpr int kPieces = kRows * HD / 4, kRowPieces = HD / 4;
    auto summed = [&](int i) {
      const float *src = merge + i / kRowPieces * kLd + 4 * (i % kRowPieces);
      float4 x = *reinterpret_cast<const float4 *>(src);
#pragma unroll
      for (int w = 1; w < kAtWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4 *>(src + w * kRows * kLd);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      return x;
    };
    if (s_bad) {  // values of this segment that are not finite and that only some rows see
      const int p1 = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(seg1) * kUnit));
#pragma unroll 1
      for (int q = max(static_cast<int>(max(all_see + 1, 0ll)), seg0 * kUnit); q < p1; ++q) {
        const int r = row_of(q, page_of(q, true));
        if (r < 0) continue;
#pragma unroll 1
        for (int i = tid; i < kRows * HD; i += kAtThreads) {
          const long long o = static_cast<long long>(r) * HD + i % HD;
          bool bad;
          if constexpr (E4M3) bad = (static_cast<const uint8_t *>(a.kv.v)[o] & 0x7f) == 0x7f;
          else bad = (static_cast<const uint16_t *>(a.kv.v)[o] & 0x7f80) == 0x7f80;
          if (bad && q <= s_lim[i / HD]) merge[i / HD * kLd + i % HD] = __uint_as_float(0x7fffffffu);
        }
      }
      __syncthreads();
    }
    auto finish = [&](int i, float4 x, float L) {
      const int r = i / kRowPieces;
      if (s_out[r] < 0) return;
      const bool none = s_lim[r] < 0 || L == 0.f;
      const float by = 1.0f / L;
      x = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * by, x.y * by, x.z * by, x.w * by);
      const long long o = s_out[r] + 4 * (i % kRowPieces);
      if constexpr (sizeof(TIO) == 4) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + o) = x;
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + o) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
      }
    };
    if (whole) {
#pragma unroll 1
      for (int i = tid; i < kPieces; i += kAtThreads) finish(i, summed(i), s_L[i / kRowPieces]);
    } else {
      // ---- this block's part of the item, and the join by the last to leave one ------------
      // block i of one-weight shares holds weight i
      const bool single = place.share == 1 && place.more == 0;
      const int first = single ? static_cast<int>(at) : block_of(at, place.share, place.more);
      const int last = single ? static_cast<int>(at) + weight - 1 : block_of(at + weight - 1, place.share, place.more);
      const int me = blockIdx.x;
      // slot 1: the item begins in this block; slot 0: it began before
      auto slot_of = [&](int blk) { return 2 * blk + (blk == first); };
#pragma unroll 1
      for (int i = tid; i < kPieces; i += kAtThreads) __stcg(p.part + static_cast<long long>(slot_of(me)) * kPieces + i, summed(i));
      if (tid < kRows) __stcg(p.part_ml + slot_of(me) * kRows + tid, make_float2(s_M[tid], s_L[tid]));
      // A tree of joins: the last of kJoin parts to arrive at their group's counter joins
      // them, in their order, into the output, or into the group's first part, which is one
      // of the next level's.
      const int n_parts = last - first + 1;
#pragma unroll 1
      for (int level = 0, bits = 0;; ++level, bits += kJoinBits) {
        const int step = 1 << bits, span = step << kJoinBits, b0 = first + ((me - first) & -span);
        const int parts = (min(last - b0 + 1, span) + step - 1) >> bits;
        uint32_t *counter = p.count + level * 2 * gridDim.x + slot_of(b0);
        const bool final = span >= n_parts;
        __syncthreads();  // the block's part is written; the release below makes it seen
        if (tid == 0) {
          uint32_t old;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
          s_last = old == static_cast<uint32_t>(parts - 1);
          if (s_last) *counter = 0;  // for the next call
        }
        __syncthreads();
        if (!s_last) break;
        // two pieces at a time
        static_assert(kPieces % (2 * kAtThreads) == 0 || kPieces == kAtThreads, "pieces per thread");
        constexpr int kAtOnce = kPieces == kAtThreads ? 1 : 2;
#pragma unroll 1
        for (int i0 = tid; i0 < kPieces; i0 += kAtOnce * kAtThreads) {
          float M[kAtOnce], L[kAtOnce];
          float4 x[kAtOnce];
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) {
            M[e] = -INFINITY;
            L[e] = 0.f;
            x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          float4 y[kAtOnce][kJoin];
          float2 ml[kAtOnce][kJoin];
#pragma unroll
          for (int k = 0; k < kJoin; ++k) {  // behind the last part: the last again, without weight
            const int slot = slot_of(b0 + (min(k, parts - 1) << bits));
            const float4 *src = p.part + static_cast<long long>(slot) * kPieces + i0;
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
              ml[e][k] = __ldcg(p.part_ml + slot * kRows + (i0 + e * kAtThreads) / kRowPieces);
              y[e][k] = __ldcg(src + e * kAtThreads);
            }
          }
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) {
#pragma unroll
            for (int k = 0; k < kJoin; ++k) M[e] = fmaxf(M[e], ml[e][k].x);
#pragma unroll
            for (int k = 0; k < kJoin; ++k)
              if (k < parts) {
                const float by = ml[e][k].x == -INFINITY ? 1.f : ex2(ml[e][k].x - M[e]);
                L[e] = fmaf(ml[e][k].y, by, L[e]);
                x[e].x = fmaf(y[e][k].x, by, x[e].x);
                x[e].y = fmaf(y[e][k].y, by, x[e].y);
                x[e].z = fmaf(y[e][k].z, by, x[e].z);
                x[e].w = fmaf(y[e][k].w, by, x[e].w);
              }
          }
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e) {
            const int i = i0 + e * kAtThreads, r = i / kRowPieces;
            if (final) {
              finish(i, x[e], L[e]);
            } else {
              __stcg(p.part + static_cast<long long>(slot_of(b0)) * kPieces + i, x[e]);  // read by this thread alone
              if (i % kRowPieces == 0) {
                s_M[r] = M[e];
                s_L[r] = L[e];
              }
            }
          }
        }
        if (final) break;
        __syncthreads();  // every thread has read b0's reference
        if (tid < kRows) __stcg(p.part_ml + slot_of(b0) * kRows + tid, make_float2(s_M[tid], s_L[tid]));
      }
    }
    u = at + w1;
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

// Groups per token and the grid: heads of a token are spread over groups while
// there are too few tokens to fill a B200's SMs (about 64 groups each).
constexpr int kSms = 148;
dim3 row_grid(const mk_paged_kv &kv, int threads, int lanes, int B, int T, int &spread) {
  const int per = threads / lanes;
  const long long tokens = static_cast<long long>(B) * T, want = kSms * 64;
  spread = static_cast<int>(std::max(1ll, std::min<long long>(kv.n_kv_heads, want / tokens)));
  const unsigned groups = static_cast<unsigned>(T) * spread;  // checked to fit by the caller
  return dim3((groups + per - 1) / per, std::min(B, 65535));
}

}  // namespace

cudaError_t launch_kv_append(const KvAppend &args, int in_dtype, cudaStream_t st) {
  KvAppend a = args;
  const dim3 grid = row_grid(a.kv, kAppendThreads, a.kv.head_dim / 16, a.B, a.T, a.spread), block(kAppendThreads);
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

cudaError_t launch_kv_gather(const KvGather &args, int out_dtype, cudaStream_t st) {
  KvGather a = args;
  const dim3 grid = row_grid(a.kv, kRowThreads, a.kv.head_dim / 8, a.B, a.T, a.spread), block(kRowThreads);
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

// Workspace: counters (of at most two items per block, for each level of a join), then
// the parts, laid out for the most rows.
constexpr size_t kCountBytes = sizeof(uint32_t) * kLevels * 2 * kAtMaxBlocks;

size_t paged_attention_workspace(int n_sm) {
  // two parts of 16 rows in 3 blocks per SM: more than of 8 rows
  return kCountBytes + sizeof(float) * 2 * static_cast<size_t>(n_sm) * 48 * (128 + 2);
}

template <int HD, typename TIO, bool E4M3, int NT>
static cudaError_t run_attention(AttnArgs &p, void *workspace, int n_sm, cudaStream_t st) {
  using S = AtShape<HD, TIO, E4M3, NT>;
  static_assert(S::kBlocks * S::kRows <= 48 && HD <= 128, "workspace");
  static_assert(S::kSmem <= 40 * 1024, "no opt-in needed beside the static shared memory");
  const int blocks = std::min(n_sm * S::kBlocks, kAtMaxBlocks);
  p.n_rg = (p.R + S::kRows - 1) / S::kRows;
  p.few = p.a.B <= 32 && p.n_rg <= 8 &&
          static_cast<long long>(p.a.B) * p.n_rg * p.a.kv.n_kv_heads * (p.cap / kUnit + 1) < (1ll << 30);
  p.count = static_cast<uint32_t *>(workspace);
  p.part = reinterpret_cast<float4 *>(static_cast<char *>(workspace) + kCountBytes);
  p.part_ml = reinterpret_cast<float2 *>(p.part + static_cast<size_t>(2) * blocks * S::kRows * HD / 4);
  return launch(paged_attn<HD, TIO, E4M3, NT>, dim3(blocks), dim3(S::kThreads), S::kSmem, st, p);
}

template <int HD, typename TIO, bool E4M3>
static cudaError_t run_rows(AttnArgs &p, void *workspace, int n_sm, cudaStream_t st) {
  if (p.R <= 8) return run_attention<HD, TIO, E4M3, 1>(p, workspace, n_sm, st);
  return run_attention<HD, TIO, E4M3, 2>(p, workspace, n_sm, st);
}

static Div div_by(uint32_t d) {  // d < 2^31: exact for dividends below 2^31 (Granlund and Montgomery 1994)
  uint32_t l = 0;
  while ((1u << l) < d) ++l;
  return {static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

cudaError_t launch_paged_attention(const PagedAttn &a, int dtype, void *workspace, int n_sm, cudaStream_t st) {
  AttnArgs p{};
  p.a = a;
  p.G = a.Hq / a.kv.n_kv_heads;
  p.R = a.T * p.G;
  p.vec = a.vec;
  p.by_page = div_by(a.kv.page_size);
  p.by_G = div_by(p.G);
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
