// kda_rows.cuh -- device helpers of the layer operators (convolution, scan, norms):
// loads and stores of activation rows in bf16 or fp32, the activations, and the
// sequence a token belongs to.  All arithmetic on rows is fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cfloat>
#include <cstdint>

#include "kda_ptx.cuh"

namespace kda {
namespace rows {

constexpr float kLog2e = 1.4426950408889634f, kLog2eRest = 1.925963033500e-8f;  // log2 e: fp32, and the rest
constexpr float kLn2 = 0.6931471805599453f, kLn2Rest = -1.904654e-9f;  // and ln 2

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }

// Raw bits of V consecutive elements, so that a thread can have several loads in
// flight in few registers.  V * sizeof(T) is 4, 8, 16 or 32 bytes (or one element).
template <typename T, int V>
struct Raw {
  static constexpr int kWords = (V * (int)sizeof(T) + 3) / 4;
  uint32_t w[kWords];
};

// INPLACE: an output of the kernel may be this buffer, so the read-only path is out.
template <bool INPLACE, typename W>
__device__ __forceinline__ W load_one(const W* p) {
  if constexpr (INPLACE) return *p;
  else return __ldg(p);
}
template <bool INPLACE = false, int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const void* p) {
  if constexpr (WORDS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = load_one<INPLACE>(static_cast<const uint4*>(p) + i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (WORDS == 2) {
    const uint2 v = load_one<INPLACE>(static_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = load_one<INPLACE>(static_cast<const uint32_t*>(p));
  }
}
template <int WORDS>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[WORDS]) {
  if constexpr (WORDS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i)
      static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else if constexpr (WORDS == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    *static_cast<uint32_t*>(p) = w[0];
  }
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(r.w[i]);
  } else if constexpr (V == 1) {
    f[0] = lo_bf16(r.w[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[2 * i] = lo_bf16(r.w[i]), f[2 * i + 1] = hi_bf16(r.w[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void pack(Raw<T, V>& r, const float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(f[i]);
  } else if constexpr (V == 1) {
    r.w[0] = pack_bf16(f[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  }
}

// V elements of a row that one thread holds: consecutive on the vector path (VEC),
// `step` elements apart on the scalar path (a warp's loads stay contiguous), where
// elements at or past `left` read as zero and are not written.
template <typename T, int V, bool VEC, bool INPLACE = false>
__device__ __forceinline__ void load_row(Raw<T, V>& r, const T* p, int step, int64_t left) {
  if constexpr (VEC) {
    load_words<INPLACE>(r.w, p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      r.w[i] = (int64_t)i * step < left
                   ? __float_as_uint(load_one<INPLACE>(reinterpret_cast<const float*>(p) + (int64_t)i * step))
                   : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t b = (int64_t)i * step < left
                             ? (uint32_t)load_one<INPLACE>(reinterpret_cast<const unsigned short*>(p) + (int64_t)i * step)
                             : 0u;
      if (i & 1) r.w[i / 2] |= b << 16;
      else r.w[i / 2] = b;
    }
  }
}
template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_row(T* p, const float (&f)[V], int step, int64_t left) {
  if constexpr (VEC) {
    Raw<T, V> r;
    pack(r, f);
    store_words(p, r.w);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((int64_t)i * step < left) p[(int64_t)i * step] = from_f<T>(f[i]);
  }
}

// Pairs of fp32 values in one 64-bit register: the packed operations run 128 values a clock
// on an SM, scalar ones 80 (measured, three-operand mix).  Kept as integers so that a pair
// loaded from memory is used as it is.
using pair = unsigned long long;
__device__ __forceinline__ pair pr(float a, float b) {
  pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ pair pr(float a) { return pr(a, a); }
__device__ __forceinline__ float2 un(pair v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ pair pmul(pair a, pair b) {
  pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair padd(pair a, pair b) {
  pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair pfma(pair a, pair b, pair c) {
  pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair pex2(pair v) {
  const float2 e = un(v);
  return pr(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
}

// exp(-x) = 2^-n, n = x log2 e, with the hardware exponential (2^-22).  Rounding n makes the
// error grow by 1.5 steps of 2^-24 for each unit of x: nothing to a step of bf16, but for rows
// of fp32 (T) the rounding is put back as exp(-x) = 2^-n (1 + (n ln 2 - x)).  That takes an x
// whose exponential is finite; at the ends sigmoid(x) is 0 and 1 as it is beyond them.
__device__ __forceinline__ float exp_range(float x) {  // what is no number stays none
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-88.5f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(128.f));
  return x;
}
template <typename T>
__device__ __forceinline__ float exp_minus(float x) {
  if constexpr (sizeof(T) < 4) return ptx::ex2_approx(-x * kLog2e);
  x = exp_range(x);
  const float n = x * kLog2e, e = ptx::ex2_approx(-n);
  return fmaf(e, fmaf(n, kLn2Rest, fmaf(n, kLn2, -x)), e);
}
template <typename T>
__device__ __forceinline__ pair exp_minus(pair x) {
  if constexpr (sizeof(T) < 4) return pex2(pmul(x, pr(-kLog2e)));
  const float2 v = un(x);
  x = pr(exp_range(v.x), exp_range(v.y));
  const pair n = pmul(x, pr(kLog2e));
  const pair e = pr(ptx::ex2_approx(-un(n).x), ptx::ex2_approx(-un(n).y));
  return pfma(e, pfma(n, pr(kLn2Rest), pfma(n, pr(kLn2), pmul(x, pr(-1.f)))), e);
}

// sigmoid(x) = 1 / (1 + exp(-x)) with the hardware reciprocal (2^-23): a clean zero where the
// exponential is infinite.  T: the rows' type.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  return ptx::rcp_approx(1.0f + exp_minus<T>(x));
}
template <typename T>
__device__ __forceinline__ pair sigmoid(pair x) {
  const float2 s = un(padd(exp_minus<T>(x), pr(1.0f)));
  return pr(ptx::rcp_approx(s.x), ptx::rcp_approx(s.y));
}
template <typename T>
__device__ __forceinline__ pair silu(pair x) { return pmul(x, sigmoid<T>(x)); }

// silu'(x) = s + x s (1 - s) from s = sigmoid(x).  1 - s is within 2^-23, and zero once s is 1
// (x = 17), so the slope is within 17 such steps of 1 however large x is; expanded to
// s + x s - x s^2 its error would grow with x.
__device__ __forceinline__ pair silu_slope(pair x, pair s) {
  return pfma(pmul(x, s), pfma(s, pr(-1.0f), pr(1.0f)), s);
}

// sigmoid(x) and its slope sigmoid(x) sigmoid(-x) = e s^2 with e = exp(-x).  As s - s^2 it would
// lose its digits where s nears 1: all of them from x = 17 on.  (An infinite e, which fp32 rows do
// not have, meets s = 0.)
template <typename T>
__device__ __forceinline__ float sigmoid(float x, float& slope) {
  const float e = exp_minus<T>(x), s = ptx::rcp_approx(1.0f + e);
  slope = (sizeof(T) < 4 ? fminf(e, FLT_MAX) : e) * s * s;
  return s;
}
template <typename T>
__device__ __forceinline__ pair sigmoid(pair x, pair& slope) {
  const pair e = exp_minus<T>(x);
  const float2 d = un(padd(e, pr(1.0f)));
  const pair s = pr(ptx::rcp_approx(d.x), ptx::rcp_approx(d.y));
  const pair f = sizeof(T) < 4 ? pr(fminf(un(e).x, FLT_MAX), fminf(un(e).y, FLT_MAX)) : e;
  slope = pmul(pmul(f, s), s);
  return s;
}

// V fp32 values that are computed with together: in pairs, or one alone.
template <int V>
struct Vals {
  pair v[V / 2];
};
template <>
struct Vals<1> {
  float v[1];
};
#define KDA_VALS_OP(NAME, PACKED, ONE)                                                     \
  template <int V>                                                                         \
  __device__ __forceinline__ Vals<V> NAME(const Vals<V>& a, const Vals<V>& b,              \
                                          const Vals<V>& c) {                              \
    Vals<V> r;                                                                             \
    if constexpr (V == 1) {                                                                \
      r.v[0] = ONE;                                                                        \
    } else {                                                                               \
      _Pragma("unroll") for (int i = 0; i < V / 2; ++i) r.v[i] = PACKED;                   \
    }                                                                                      \
    return r;                                                                              \
  }
KDA_VALS_OP(fma_of, pfma(a.v[i], b.v[i], c.v[i]), fmaf(a.v[0], b.v[0], c.v[0]))
KDA_VALS_OP(mul_first, pmul(a.v[i], b.v[i]), a.v[0] * b.v[0])
#undef KDA_VALS_OP
template <int V>
__device__ __forceinline__ Vals<V> mul_of(const Vals<V>& a, const Vals<V>& b) {
  return mul_first(a, b, b);
}
template <int V>
__device__ __forceinline__ Vals<V> splat(float f) {
  Vals<V> r;
  if constexpr (V == 1) {
    r.v[0] = f;
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = pr(f);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> sigmoid(const Vals<V>& x) {
  Vals<V> r;
  if constexpr (V == 1) {
    r.v[0] = sigmoid<T>(x.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = sigmoid<T>(x.v[i]);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> sigmoid(const Vals<V>& x, Vals<V>& slope) {
  Vals<V> r;
  if constexpr (V == 1) {
    r.v[0] = sigmoid<T>(x.v[0], slope.v[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = sigmoid<T>(x.v[i], slope.v[i]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ float sum_of(const Vals<V>& a) {
  if constexpr (V == 1) {
    return a.v[0];
  } else {
    pair s = a.v[0];
#pragma unroll
    for (int i = 1; i < V / 2; ++i) s = padd(s, a.v[i]);
    return un(s).x + un(s).y;
  }
}
template <int V>
__device__ __forceinline__ Vals<V> vals_from(const float (&f)[V]) {
  Vals<V> r;
  if constexpr (V == 1) {
    r.v[0] = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = pr(f[2 * i], f[2 * i + 1]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ void vals_to(const Vals<V>& a, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = a.v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[2 * i] = un(a.v[i]).x, f[2 * i + 1] = un(a.v[i]).y;
  }
}

// The sequence that holds token t: the largest n with cu[n] <= t (cu sorted), by a
// search of 32 pivots a step, all lanes of the warp together.  The result lies in
// [0, N - 1] whatever cu holds; the caller checks the token against its bounds.
__device__ __forceinline__ int find_sequence(const int64_t* cu, int N, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = N;  // cu[lo] <= t (or lo == 0), and cu[hi] > t (or hi == N)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && __ldg(cu + at) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le) | 1u;
    const int k = 31 - __clz(m);  // the last pivot that holds
    hi = min(hi, lo + (k + 1) * step);
    lo = lo + k * step;
  }
  return lo;
}

// Writes the status word of a workspace from a full check of cu_seqlens: one warp.
// cu[0] = 0, non-decreasing, cu[N] <= total.
__device__ __forceinline__ void check_seqlens(const int64_t* cu, int N, int64_t total,
                                              unsigned* status, unsigned bad_bit) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i <= N; i += 32) {
    const int64_t c = cu[i];
    bad |= c < 0 || c > total || (i == 0 && c != 0) || (i < N && cu[i + 1] < c);
  }
  bad = __any_sync(0xffffffffu, bad);
  if ((threadIdx.x & 31) == 0) *status = bad ? bad_bit : 0u;
}

}  // namespace rows

// out[e] = sum over r < rows of part[r * pitch + e] in a fixed order: the first n0 columns go to
// out0, the next n1 to out1, the rest to out2 (a null output drops its columns).
cudaError_t launch_column_sums(const float* part, int64_t rows, int64_t pitch, int64_t cols,
                               int64_t n0, int64_t n1, float* out0, float* out1, float* out2,
                               cudaStream_t stream);

}  // namespace kda
