// kda_norm.cu -- the norms before and after a block, forward and backward.
//
// Per row of D values: unit(h) = h rstd(h), rstd = (mean(h^2) + eps)^(-1/2).
//   before a block: h = residual + s x,  out = unit(h) w            (h is kept as well)
//   after a block:  out = residual + s (unit(x) w fn(gate))
// and backwards, with du = the gradient of unit(h) per value,
//   dh = rstd (du - unit(h) mean(du unit(h))),
// which needs the two row sums S1 = sum h^2 and S2 = sum du h in one reduction, since
// mean(du unit(h)) = rstd S2 / D.
//
// All of it is bound by HBM: each row is read once and written once, so a row stays in
// the registers of the threads that read it, between the reduction and the output.  Rows
// of up to 64 vectors belong to 16 or 32 lanes (no barrier, several rows per
// warp's loads in flight); longer ones to a block with one barrier per row.  Weight
// gradients are summed over a block's rows in registers, then over the blocks by a
// second launch, in a fixed order and in fp32: 2 to 3e-7 from their 64-bit values over 2^27
// values.  Sums of 16 rows at a time, added apart, and a second launch in 64 bits halve that
// and take 3 to 33 % longer.
//
// Device time, and bytes of the rows over it: forward before a block, 32,768 rows of 4,096
// bf16 values with an fp32 residual, 238 us (6.8 TB/s); forward after one, 1,048,576 rows of
// 128 bf16 with a gate, 136 us (5.9 TB/s); backward before a block, 32,768 x 4,096 bf16
// with a learned scale, 245 us (6.6 TB/s); backward after one, 74,097 rows of 1,001 fp32
// with gate and scale (no 16-byte alignment, so single values), 303 us (4.9 TB/s).  Backward
// over rows wider than 4,096, whose two vectors per thread and next rows in registers spill:
// 2^27 bf16 values with a learned scale in rows of 5,120 396, of 8,192 318 us before a block;
// after one, with a SiLU gate, 395 and 368.  Backward without a gate, bf16, where a row brings
// too few bytes to hide its two sums and the barrier: 2^27 values in rows of 1,024 169 us.
#include "kda_internal.h"
#include "kda_rows.cuh"
#include "../../include/kda_layer.h"

#include <cmath>
#include <type_traits>

namespace kda {
namespace {

using namespace rows;

struct NormParams {
  const void *a, *b, *c, *d;  // row inputs (see the kernels)
  void *o0, *o1;              // row outputs
  const float *weight, *scale;
  float scale_value, eps;
  int64_t n_rows, gate_stride;
  int heads, dim, fn;
  float* part;                // [blocks][1 or 2][dim] partial dweight (, dscale)
  int want_scale;
};

// A thread's values of a row come in vectors of V = 8 consecutive ones (16 bytes of bf16, 32
// of fp32), or singly (V = 1) where rows are not 16-byte aligned.  They are kept as they
// were read until they are needed, so that the next row's are on their way meanwhile.
template <typename T, int V>
__device__ __forceinline__ void load_vec(Raw<T, V>& r, const void* p, int64_t at) {
  if constexpr (V == 1) r.w[0] = __float_as_uint(to_f(static_cast<const T*>(p)[at]));
  else load_words<true>(r.w, static_cast<const T*>(p) + at);
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> values(const Raw<T, V>& r) {
  float f[V];
  if constexpr (V == 1) f[0] = __uint_as_float(r.w[0]);
  else unpack(r, f);
  return vals_from(f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(void* p, int64_t at, const Vals<V>& v) {
  float f[V];
  vals_to(v, f);
  store_row<T, V, (V > 1)>(static_cast<T*>(p) + at, f, 1, 1);
}

// Sums over the G threads of a row (G = 16, 32: lanes; G = 0: the whole block, one barrier,
// `red` alternates between two halves so that no second one is needed).  Every thread
// gets the same bits.  TWO: both sums are wanted.
template <int G, bool TWO>
__device__ __forceinline__ float2 row_sum(float2 v, float2* red, int turn) {
  constexpr int W = G == 16 ? 16 : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    if (TWO) v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (G != 0) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float2* r = red + (turn & 1) * 32;
  if (lane == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? r[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    if (TWO) v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// The gate's activation, and with its slope.
template <typename T, int V>
__device__ __forceinline__ Vals<V> gate_fn(const Vals<V>& p, int fn) {
  const Vals<V> s = sigmoid<T>(p);
  return fn == KDA_FN_SILU ? mul_of(p, s) : s;
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> gate_fn(const Vals<V>& p, int fn, Vals<V>& slope) {
  Vals<V> ds;
  const Vals<V> s = sigmoid<T>(p, ds);
  slope = ds;
  if (fn != KDA_FN_SILU) return s;
  slope = fma_of(p, ds, s);
  return mul_of(p, s);
}

// How far row's gate lies from where it would lie without a stride of its own.
__device__ __forceinline__ int64_t gate_shift(const NormParams& p, int64_t row) {
  const int64_t own = (int64_t)p.heads * p.dim;
  return p.gate_stride == own ? 0 : row / p.heads * (p.gate_stride - own);
}

// The rows of a block: group `grp` of the block's rows_per_block takes row
// blockIdx * rpb + grp, then every grid * rpb further.  Lanes of a warp run the same
// number of turns (the reductions are warp-wide); `live` masks the rows past the end.
#define KDA_NORM_ROWS(G)                                                                 \
  const int gsz = (G) ? (G) : (int)blockDim.x;                                           \
  const int rpb = (G) ? (int)blockDim.x / (G) : 1;                                       \
  const int g = (G) ? (int)threadIdx.x % (G) : (int)threadIdx.x;                         \
  const int grp = (G) ? (int)threadIdx.x / (G) : 0;                                      \
  __shared__ float2 red[64];                                                             \
  int turn = 0;                                                                          \
  const int D = p.dim, nv = (D + V - 1) / V;                                             \
  const float inv_d = 1.0f / (float)D;                                                   \
  const int64_t stride = (int64_t)gridDim.x * rpb;                                       \
  Vals<V> w[E], sc[E];                                                                   \
  _Pragma("unroll") for (int i = 0; i < E; ++i) {                                        \
    const int vi = i * gsz + g;                                                          \
    Raw<float, V> r;                                                                     \
    w[i] = splat<V>(0.f), sc[i] = splat<V>(p.scale_value);                               \
    if (vi < nv) load_vec(r, p.weight, (int64_t)vi * V), w[i] = values(r);               \
    if (vi < nv && p.scale) load_vec(r, p.scale, (int64_t)vi * V), sc[i] = values(r);    \
  }                                                                                      \
  /* f(i, offset) for the thread's vectors of a row that exists */                       \
  auto each = [&](int64_t row, auto f) {                                                 \
    _Pragma("unroll") for (int i = 0; i < E; ++i) {                                      \
      const int vi = i * gsz + g;                                                        \
      if (row < p.n_rows && vi < nv) f(i, row * D + (int64_t)vi * V);                    \
    }                                                                                    \
  };                                                                                     \
  int64_t row = (int64_t)blockIdx.x * rpb + grp;

// Rows on their way through shared memory: the backward over long rows (G = 0, one vector
// of 8 per thread) keeps the next ones there by asynchronous copies, since the weights and
// their gradients fill its registers.  Each thread reads back what it asked for, so no
// barrier is needed.  A slot has at most 128 bytes per thread, so that three fit with 512.
// Backward before a block over 2^27 bf16 values in rows of 1,024 and 4,096, with a learned
// scale: 270 and 246 us, against 726 and 319 with the next row in registers.
constexpr int kNormRing = 3;
__host__ __device__ constexpr bool norm_has_ring(int G, int E, int V) { return G == 0 && E == 1 && V == 8; }

template <typename T>
__device__ __forceinline__ void copy_vec(void* to, const void* from, int64_t at) {
#pragma unroll
  for (int b = 0; b < 8 * (int)sizeof(T); b += 16)
    ptx::cp_async16(static_cast<uint8_t*>(to) + b, static_cast<const uint8_t*>(from) + at * sizeof(T) + b, 16);
}

// Threads of a block, and the blocks per SM that a backward's registers leave room for: one of
// 512 threads with a ring (its rows in flight need no second block, and 64 registers spill).
constexpr int norm_threads(int G, int E, int V) { return G ? 256 : V == 1 && E == 8 ? 1024 : 512; }
constexpr int norm_bwd_blocks(int G, int E, int V) { return G || E > 1 || V == 8 ? 1 : 2; }

template <int G, int E, int V, typename T, typename TS>
__global__ void __launch_bounds__(norm_threads(G, E, V)) prenorm_fwd_kernel(const NormParams p) {
  KDA_NORM_ROWS(G)
  Raw<T, V> rx[E] = {};
  Raw<TS, V> rr[E] = {};
  auto fetch = [&](int64_t at_row) {
    each(at_row, [&](int i, int64_t at) {
      load_vec(rx[i], p.a, at);
      if (p.b) load_vec(rr[i], p.b, at);
    });
  };
  fetch(row);
  for (int64_t base = row - grp; base < p.n_rows; base += stride, row += stride, ++turn) {
    Vals<V> h[E], sq = splat<V>(0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      h[i] = fma_of(sc[i], values(rx[i]), values(rr[i]));
      sq = fma_of(h[i], h[i], sq);
    }
    fetch(row + stride);
    const float s = row_sum<G, false>(make_float2(sum_of(sq), 0.f), red, turn).x;
    const float rstd = rsqrtf(s * inv_d + p.eps);
    each(row, [&](int i, int64_t at) {
      if (p.o1) store_vec<TS, V>(p.o1, at, h[i]);
      store_vec<T, V>(p.o0, at, mul_of(mul_of(h[i], splat<V>(rstd)), w[i]));
    });
  }
}

template <int G, int E, int V, typename T, typename TS>
__global__ void __launch_bounds__(norm_threads(G, E, V)) postnorm_fwd_kernel(const NormParams p) {
  KDA_NORM_ROWS(G)
  Vals<V> sw[E];
#pragma unroll
  for (int i = 0; i < E; ++i) sw[i] = mul_of(w[i], sc[i]);
  Raw<T, V> rx[E] = {}, rg[E] = {}, rr[E] = {};
  auto fetch_x = [&](int64_t at_row) {
    each(at_row, [&](int i, int64_t at) { load_vec(rx[i], p.a, at); });
  };
  auto fetch_rest = [&](int64_t at_row) {
    const int64_t shift = gate_shift(p, at_row);
    each(at_row, [&](int i, int64_t at) {
      if (p.b) load_vec(rg[i], p.b, at + shift);
      if (p.c) load_vec(rr[i], p.c, at);
    });
  };
  fetch_x(row);
  fetch_rest(row);
  for (int64_t base = row - grp; base < p.n_rows; base += stride, row += stride, ++turn) {
    Vals<V> x[E], sq = splat<V>(0.f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] = values(rx[i]);
      sq = fma_of(x[i], x[i], sq);
    }
    fetch_x(row + stride);
    const float s = row_sum<G, false>(make_float2(sum_of(sq), 0.f), red, turn).x;
    const float rstd = rsqrtf(s * inv_d + p.eps);
    each(row, [&](int i, int64_t at) {
      Vals<V> n = mul_of(mul_of(x[i], splat<V>(rstd)), sw[i]);
      if (p.b) n = mul_of(n, gate_fn<T>(values(rg[i]), p.fn));
      if (p.c) n = fma_of(n, splat<V>(1.f), values(rr[i]));
      store_vec<T, V>(p.o0, at, n);
    });
    fetch_rest(row + stride);
  }
}

// Adds the block's row groups' dweight and dscale in the groups' order and writes the
// block's partial row.
template <int G, int E, int V>
__device__ __forceinline__ void write_partials(const NormParams& p, const Vals<V> (&dwv)[E],
                                               const Vals<V> (&dsv)[E], int g, int grp, int gsz,
                                               int rpb, int nv) {
  extern __shared__ __align__(16) uint8_t norm_ring[];
  float* const acc = reinterpret_cast<float*>(norm_ring);  // [2][dim], rows sharing a block
  float dw[E][V], ds[E][V];
#pragma unroll
  for (int i = 0; i < E; ++i) vals_to(dwv[i], dw[i]), vals_to(dsv[i], ds[i]);
  const int pitch = (p.want_scale ? 2 : 1) * p.dim;
  float* out = p.part + (int64_t)blockIdx.x * pitch;
  if constexpr (G == 0) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int vi = i * gsz + g;
      if (vi >= nv) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        out[vi * V + k] = dw[i][k];
        if (p.want_scale) out[p.dim + vi * V + k] = ds[i][k];
      }
    }
  } else {
    for (int r = 0; r < rpb; ++r) {
      if (grp == r) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int vi = i * gsz + g;
          if (vi >= nv) continue;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int e = vi * V + k;
            acc[e] = r ? acc[e] + dw[i][k] : dw[i][k];
            if (p.want_scale) acc[p.dim + e] = r ? acc[p.dim + e] + ds[i][k] : ds[i][k];
          }
        }
      }
      __syncthreads();
    }
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) out[e] = acc[e];
  }
}

// a = dout, b = dresidual_out or null, c = h, d = x or null (dscale)
template <int G, int E, int V, typename T, typename TS>
__global__ void __launch_bounds__(norm_threads(G, E, V), norm_bwd_blocks(G, E, V))
    prenorm_bwd_kernel(const NormParams p) {
  constexpr bool RING = norm_has_ring(G, E, V);
  extern __shared__ __align__(16) uint8_t norm_ring[];
  KDA_NORM_ROWS(G)
  Vals<V> dw[E], ds[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = ds[i] = splat<V>(0.f);
  Raw<TS, V> rh[E] = {}, rd[E] = {};
  Raw<T, V> ry[E] = {}, rx[E] = {};
  // a ring slot: h, dresidual_out, dout, x of all threads
  constexpr int SLOT = 16 * (int)(sizeof(TS) + sizeof(T));
  constexpr int AHEAD = kNormRing - 1;
  auto slot_of = [&](int k) { return norm_ring + k % kNormRing * (int)blockDim.x * SLOT; };
  auto issue = [&](int64_t at_row, int k) {
    if constexpr (RING) {
      uint8_t* const to = slot_of(k);
      const int n = blockDim.x;
      each(at_row, [&](int, int64_t at) {
        copy_vec<TS>(to + g * 8 * sizeof(TS), p.c, at);
        if (p.b) copy_vec<TS>(to + (n + g) * 8 * sizeof(TS), p.b, at);
        copy_vec<T>(to + 2 * n * 8 * sizeof(TS) + g * 8 * sizeof(T), p.a, at);
        if (p.want_scale) copy_vec<T>(to + 2 * n * 8 * sizeof(TS) + (n + g) * 8 * sizeof(T), p.d, at);
      });
      ptx::cp_async_commit();
    }
  };
  auto fetch_sums = [&](int64_t at_row) {
    if constexpr (!RING) {
      each(at_row, [&](int i, int64_t at) {
        load_vec(rh[i], p.c, at);
        load_vec(ry[i], p.a, at);
      });
    }
  };
  auto fetch_rest = [&](int64_t at_row) {
    if constexpr (!RING) {
      each(at_row, [&](int i, int64_t at) {
        if (p.b) load_vec(rd[i], p.b, at);
        if (p.want_scale) load_vec(rx[i], p.d, at);
      });
    }
  };
  for (int k = 0; k < AHEAD; ++k) issue(row + k * stride, k);
  fetch_sums(row);
  fetch_rest(row);
  for (int64_t base = row - grp; base < p.n_rows; base += stride, row += stride, ++turn) {
    if constexpr (RING) {
      issue(row + AHEAD * stride, turn + AHEAD);
      ptx::cp_async_wait<AHEAD>();
      const uint8_t* const from = slot_of(turn);
      const int n = blockDim.x;
      if (g < nv) {  // the others' part of a slot is never filled: their values stay zero
        load_words<true>(rh[0].w, from + g * 8 * sizeof(TS));
        if (p.b) load_words<true>(rd[0].w, from + (n + g) * 8 * sizeof(TS));
        load_words<true>(ry[0].w, from + 2 * n * 8 * sizeof(TS) + g * 8 * sizeof(T));
        if (p.want_scale)
          load_words<true>(rx[0].w, from + 2 * n * 8 * sizeof(TS) + (n + g) * 8 * sizeof(T));
      }
    }
    Vals<V> h[E], dy[E], s1 = splat<V>(0.f), s2 = s1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      h[i] = values(rh[i]);
      dy[i] = values(ry[i]);
      s1 = fma_of(h[i], h[i], s1);
      s2 = fma_of(mul_of(dy[i], w[i]), h[i], s2);
    }
    fetch_sums(row + stride);
    const float2 s = row_sum<G, true>(make_float2(sum_of(s1), sum_of(s2)), red, turn);
    const float rstd = rsqrtf(s.x * inv_d + p.eps);
    const float c = s.y * inv_d * rstd * rstd * rstd;
    each(row, [&](int i, int64_t at) {
      const Vals<V> dr = mul_of(dy[i], splat<V>(rstd));
      Vals<V> dh = fma_of(dr, w[i], values(rd[i]));
      dh = fma_of(h[i], splat<V>(-c), dh);
      dw[i] = fma_of(dr, h[i], dw[i]);
      ds[i] = fma_of(dh, values(rx[i]), ds[i]);
      if (p.o1) store_vec<TS, V>(p.o1, at, dh);
      if (p.o0) store_vec<T, V>(p.o0, at, mul_of(dh, sc[i]));
    });
    fetch_rest(row + stride);
  }
  write_partials<G, E, V>(p, dw, ds, g, grp, gsz, rpb, nv);
}

// a = dout, b = gate or null, c = x; o0 = dx, o1 = dgate.  With a = fn(gate), a' its slope:
// P = dout a and Q = dout a' are all that is kept of dout and the gate.
template <int G, int E, int V, typename T, typename TS>
__global__ void __launch_bounds__(norm_threads(G, E, V), norm_bwd_blocks(G, E, V))
    postnorm_bwd_kernel(const NormParams p) {
  constexpr bool RING = norm_has_ring(G, E, V);
  extern __shared__ __align__(16) uint8_t norm_ring[];
  KDA_NORM_ROWS(G)
  Vals<V> dw[E], ds[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = ds[i] = splat<V>(0.f);
  Raw<T, V> rx[E] = {}, ry[E] = {}, rg[E] = {};
  constexpr int SLOT = 8 * 3 * (int)sizeof(T);  // x, dout, gate of all threads
  constexpr int AHEAD = kNormRing - 1;
  auto slot_of = [&](int k) { return norm_ring + k % kNormRing * (int)blockDim.x * SLOT; };
  auto issue = [&](int64_t at_row, int k) {
    if constexpr (RING) {
      uint8_t* const to = slot_of(k);
      const int64_t shift = gate_shift(p, at_row);
      const int n = blockDim.x;
      each(at_row, [&](int, int64_t at) {
        copy_vec<T>(to + g * 8 * sizeof(T), p.c, at);
        copy_vec<T>(to + (n + g) * 8 * sizeof(T), p.a, at);
        if (p.b) copy_vec<T>(to + (2 * n + g) * 8 * sizeof(T), p.b, at + shift);
      });
      ptx::cp_async_commit();
    }
  };
  auto fetch = [&](int64_t at_row) {
    if constexpr (!RING) {
      const int64_t shift = gate_shift(p, at_row);
      each(at_row, [&](int i, int64_t at) {
        load_vec(rx[i], p.c, at);
        load_vec(ry[i], p.a, at);
        if (p.b) load_vec(rg[i], p.b, at + shift);
      });
    }
  };
  for (int k = 0; k < AHEAD; ++k) issue(row + k * stride, k);
  fetch(row);
  for (int64_t base = row - grp; base < p.n_rows; base += stride, row += stride, ++turn) {
    if constexpr (RING) {
      issue(row + AHEAD * stride, turn + AHEAD);
      ptx::cp_async_wait<AHEAD>();
      const uint8_t* const from = slot_of(turn);
      const int n = blockDim.x;
      if (g < nv) {  // the others' part of a slot is never filled: their values stay zero
        load_words<true>(rx[0].w, from + g * 8 * sizeof(T));
        load_words<true>(ry[0].w, from + (n + g) * 8 * sizeof(T));
        if (p.b) load_words<true>(rg[0].w, from + (2 * n + g) * 8 * sizeof(T));
      }
    }
    Vals<V> x[E], P[E], Q[E], s1 = splat<V>(0.f), s2 = s1;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] = values(rx[i]);
      P[i] = values(ry[i]);
      Q[i] = splat<V>(0.f);
      if (p.b) {
        Vals<V> slope;
        const Vals<V> act = gate_fn<T>(values(rg[i]), p.fn, slope);
        Q[i] = mul_of(P[i], slope);
        P[i] = mul_of(P[i], act);
      }
      s1 = fma_of(x[i], x[i], s1);
      s2 = fma_of(mul_of(mul_of(P[i], sc[i]), w[i]), x[i], s2);
    }
    fetch(row + stride);
    const float2 s = row_sum<G, true>(make_float2(sum_of(s1), sum_of(s2)), red, turn);
    const float rstd = rsqrtf(s.x * inv_d + p.eps);
    const float c = s.y * inv_d * rstd * rstd * rstd;
    each(row, [&](int i, int64_t at) {
      const Vals<V> u = mul_of(x[i], splat<V>(rstd)), su = mul_of(sc[i], u);
      const Vals<V> rws = mul_of(mul_of(w[i], sc[i]), splat<V>(rstd));
      store_vec<T, V>(p.o0, at, fma_of(rws, P[i], mul_of(x[i], splat<V>(-c))));
      if (p.o1) store_vec<T, V>(p.o1, at, mul_of(mul_of(w[i], su), Q[i]));
      dw[i] = fma_of(su, P[i], dw[i]);
      ds[i] = fma_of(mul_of(w[i], u), P[i], ds[i]);
    });
  }
  write_partials<G, E, V>(p, dw, ds, g, grp, gsz, rpb, nv);
}

// A block per 32 columns: 32 row groups add every 32nd row, then their sums are added
// in order.
__global__ void column_sums_kernel(const float* part, int64_t rows, int64_t pitch, int64_t cols,
                                   int64_t n0, int64_t n1, float* out0, float* out1, float* out2) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t e = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (e < cols) {
#pragma unroll 4
    for (int64_t r = grp; r < rows; r += 32) s += part[r * pitch + e];
  }
  sums[grp][lane] = s;
  __syncthreads();
  s = sums[lane][grp];  // lane: row group, grp: column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t c = (int64_t)blockIdx.x * 32 + grp;
  if (lane == 0 && c < cols) {
    float* const out = c < n0 ? out0 : c < n0 + n1 ? out1 : out2;
    if (out) out[c < n0 ? c : c < n0 + n1 ? c - n0 : c - n0 - n1] = s;
  }
}

// How a row is divided: G lanes (0: a block of `threads`), E vectors of V values each.
struct NormPlan {
  int G, E, V, threads, rpb;
};

NormPlan norm_plan(int dim, bool vec) {
  NormPlan n;
  n.V = vec ? 8 : 1;
  const int nv = (dim + n.V - 1) / n.V;
  n.threads = 256;
  if (nv <= 16) {
    n.G = 16, n.E = 1;
  } else if (nv <= 64) {
    n.G = 32, n.E = nv <= 32 ? 1 : 2;
  } else {
    n.G = 0;
    n.E = vec ? (nv <= 512 ? 1 : 2) : (nv <= 2048 ? 4 : 8);
    n.threads = ((nv + n.E - 1) / n.E + 31) / 32 * 32;
  }
  n.rpb = n.G ? n.threads / n.G : 1;
  return n;
}

constexpr int kMaxBlocks = 1216;  // 8 blocks on each of 152 SMs: partial rows of the sums

int64_t norm_grid(const NormPlan& n, int64_t rows, int num_sms, int per_sm) {
  const int64_t need = (rows + n.rpb - 1) / n.rpb;
  const int64_t most = (int64_t)num_sms * per_sm;
  return need < most ? need : most;
}

// A kernel, and on which devices its limit of dynamic shared memory has been raised.
struct NormKernel {
  void (*run)(NormParams);
  bool (*raised)[64];
};
template <void (*KERNEL)(NormParams)>
NormKernel norm_kernel() {
  static bool raised[64];
  return {KERNEL, &raised};
}

#define KDA_NORM_CASE(KERNEL, G_, E_, V_) \
  if (n.G == G_ && n.E == E_ && n.V == V_) return norm_kernel<KERNEL<G_, E_, V_, T, TS>>();
#define KDA_NORM_PICK(NAME, KERNEL)                                                \
  template <typename T, typename TS>                                               \
  NormKernel NAME##_of(const NormPlan& n) {                                        \
    KDA_NORM_CASE(KERNEL, 16, 1, 8)                                                \
    KDA_NORM_CASE(KERNEL, 32, 1, 8)                                                \
    KDA_NORM_CASE(KERNEL, 32, 2, 8)                                                \
    KDA_NORM_CASE(KERNEL, 0, 1, 8)                                                 \
    KDA_NORM_CASE(KERNEL, 0, 2, 8)                                                 \
    KDA_NORM_CASE(KERNEL, 16, 1, 1)                                                \
    KDA_NORM_CASE(KERNEL, 32, 1, 1)                                                \
    KDA_NORM_CASE(KERNEL, 32, 2, 1)                                                \
    KDA_NORM_CASE(KERNEL, 0, 4, 1)                                                 \
    KDA_NORM_CASE(KERNEL, 0, 8, 1)                                                 \
    return {};                                                                     \
  }                                                                                \
  NormKernel NAME(const NormPlan& n, int32_t dtype, int32_t stream_dtype) {        \
    if (dtype == KDA_ROW_FP32) return NAME##_of<float, float>(n);                  \
    return stream_dtype == KDA_ROW_FP32 && NORM_TWO_TYPES ? NAME##_of<bf16, std::conditional_t<NORM_TWO_TYPES, float, bf16>>(n) \
                                                          : NAME##_of<bf16, bf16>(n);  \
  }
#define NORM_TWO_TYPES true
KDA_NORM_PICK(pick_prenorm_fwd, prenorm_fwd_kernel)
KDA_NORM_PICK(pick_prenorm_bwd, prenorm_bwd_kernel)
#undef NORM_TWO_TYPES
#define NORM_TWO_TYPES false
KDA_NORM_PICK(pick_postnorm_fwd, postnorm_fwd_kernel)
KDA_NORM_PICK(pick_postnorm_bwd, postnorm_bwd_kernel)
#undef NORM_TWO_TYPES

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

kda_status check_norm(int64_t rows, int32_t dim, int32_t dtype, int32_t stream_dtype, float eps,
                      const float* scale, float scale_value) {
  if (rows < 0 || dim < 1 || dim > KDA_NORM_MAX_DIM || rows >= (int64_t(1) << 40) / dim)
    return KDA_ERR_INVALID_SHAPE;
  if ((dtype != KDA_ROW_BF16 && dtype != KDA_ROW_FP32) ||
      (stream_dtype != KDA_ROW_FP32 && stream_dtype != dtype) || !(eps >= 0.f) ||
      !std::isfinite(eps) || (!scale && !std::isfinite(scale_value)))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status run_norm(NormKernel kernel, const NormPlan& n, const NormParams& p,
                    int64_t grid, size_t smem, cudaStream_t stream) {
  if (!kernel.run) return KDA_ERR_INVALID_SHAPE;
  kernel.run<<<(unsigned)grid, n.threads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status run_norm_bwd(NormKernel kernel, const NormPlan& n, NormParams& p, int num_sms,
                        int ring_bytes, void* workspace, float* dweight, float* dscale,
                        cudaStream_t stream) {
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
  // as many blocks as run at once, so that the partial rows are few
  const bool ring = norm_has_ring(n.G, n.E, n.V);
  const int per_sm = n.G ? 4 : n.V == 8 ? 512 / n.threads : n.threads >= 512 ? 2 : 1024 / n.threads;
  int64_t grid = norm_grid(n, p.n_rows, num_sms, per_sm < 8 ? per_sm : 8);
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  const size_t smem = n.G ? 2 * (size_t)p.dim * sizeof(float)
                          : ring ? (size_t)kNormRing * n.threads * ring_bytes : 0;
  // The limit belongs to the kernel, for all threads of the host: raised once to the most that
  // a block of 512 threads takes, never to this call's own size.  (No instance but those with
  // a ring goes beyond what needs no request.)
  if (ring && kernel.run &&
      ensure_smem_attr(reinterpret_cast<const void*>(kernel.run), kNormRing * 512 * ring_bytes,
                       *kernel.raised) != cudaSuccess)
    return KDA_ERR_CUDA;
  if (grid > 0) {
    const kda_status st = run_norm(kernel, n, p, grid, smem, stream);
    if (st != KDA_OK) return st;
  }
  return launch_column_sums(p.part, grid, (p.want_scale ? 2 : 1) * (int64_t)p.dim,
                            (p.want_scale ? 2 : 1) * (int64_t)p.dim, p.dim, p.dim, dweight, dscale,
                            nullptr, stream) ==
                 cudaSuccess
             ? KDA_OK
             : KDA_ERR_CUDA;
}

}  // namespace

cudaError_t launch_column_sums(const float* part, int64_t rows, int64_t pitch, int64_t cols,
                               int64_t n0, int64_t n1, float* out0, float* out1, float* out2,
                               cudaStream_t stream) {
  if (cols <= 0) return cudaSuccess;
  column_sums_kernel<<<(unsigned)((cols + 31) / 32), 1024, 0, stream>>>(part, rows, pitch, cols, n0, n1,
                                                                       out0, out1, out2);
  return cudaGetLastError();
}

}  // namespace kda

extern "C" {

kda_status kda_norm_bwd_get_workspace_size(int64_t rows, int32_t dim, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  if (rows < 0 || dim < 1 || dim > KDA_NORM_MAX_DIM) return KDA_ERR_INVALID_SHAPE;
  const int64_t blocks = rows < kda::kMaxBlocks ? rows : kda::kMaxBlocks;
  *bytes = KDA_STATUS_BYTES + (size_t)blocks * 2 * dim * sizeof(float);
  return KDA_OK;
}

kda_status kda_prenorm_fwd(const void* x, const void* residual, const float* weight,
                           const float* res_scale, float res_scale_value, float eps, void* out,
                           void* residual_out, int64_t rows, int32_t dim, int32_t dtype,
                           int32_t stream_dtype, cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_norm(rows, dim, dtype, stream_dtype, eps, res_scale, res_scale_value);
  if (st != KDA_OK) return st;
  if (!weight || (rows > 0 && (!x || !out))) return KDA_ERR_NULL_POINTER;
  const size_t e = dtype == KDA_ROW_FP32 ? 4 : 2, se = stream_dtype == KDA_ROW_FP32 ? 4 : 2;
  if (!al_to(x, e) || !al_to(out, e) || !al_to(residual, se) || !al_to(residual_out, se) ||
      !al_to(weight, 4) || !al_to(res_scale, 4))
    return KDA_ERR_MISALIGNED;
  st = check_device();
  if (st != KDA_OK || rows == 0) return st;
  int num_sms = 0;
  if (sm_count(&num_sms) != KDA_OK) return KDA_ERR_CUDA;
  const NormPlan n = norm_plan(dim, dim % 8 == 0 && al16(x) && al16(out) && al16(residual) &&
                                        al16(residual_out) && al16(weight) && al16(res_scale));
  NormParams p = {};
  p.a = x, p.b = residual, p.o0 = out, p.o1 = residual_out;
  p.weight = weight, p.scale = res_scale, p.scale_value = res_scale_value, p.eps = eps;
  p.n_rows = rows, p.dim = dim;
  return run_norm(pick_prenorm_fwd(n, dtype, stream_dtype), n, p, norm_grid(n, rows, num_sms, 32), 0,
                  stream);
}

kda_status kda_prenorm_bwd(const void* dout, const void* dresidual_out, const void* h,
                           const float* weight, const void* x, const float* res_scale,
                           float res_scale_value, float eps, void* dx, void* dresidual,
                           float* dweight, float* dres_scale, int64_t rows, int32_t dim,
                           int32_t dtype, int32_t stream_dtype, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_norm(rows, dim, dtype, stream_dtype, eps, res_scale, res_scale_value);
  if (st != KDA_OK) return st;
  if (!weight || !dweight || !workspace ||
      (rows > 0 && (!dout || !h || (!dx && !dresidual) || (dres_scale && !x))))
    return KDA_ERR_NULL_POINTER;
  const size_t e = dtype == KDA_ROW_FP32 ? 4 : 2, se = stream_dtype == KDA_ROW_FP32 ? 4 : 2;
  if (!al_to(x, e) || !al_to(dout, e) || !al_to(dx, e) || !al_to(dresidual_out, se) ||
      !al_to(h, se) || !al_to(dresidual, se) || !al_to(weight, 4) || !al_to(res_scale, 4) ||
      !al_to(dweight, 4) || !al_to(dres_scale, 4) || !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  size_t need = 0;
  kda_norm_bwd_get_workspace_size(rows, dim, &need);
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  int num_sms = 0;
  if (sm_count(&num_sms) != KDA_OK) return KDA_ERR_CUDA;
  const NormPlan n =
      norm_plan(dim, dim % 8 == 0 && al16(dout) && al16(dresidual_out) && al16(h) &&
                         (!dres_scale || al16(x)) && al16(dx) && al16(dresidual) && al16(weight) &&
                         al16(res_scale));
  NormParams p = {};
  p.a = dout, p.b = dresidual_out, p.c = h, p.d = x, p.o0 = dx, p.o1 = dresidual;
  p.weight = weight, p.scale = res_scale, p.scale_value = res_scale_value, p.eps = eps;
  p.n_rows = rows, p.dim = dim, p.want_scale = dres_scale != nullptr;
  return run_norm_bwd(pick_prenorm_bwd(n, dtype, stream_dtype), n, p, num_sms, 16 * (int)(e + se),
                      workspace, dweight, dres_scale, stream);
}

kda_status kda_postnorm_fwd(const void* x, const float* weight, const void* gate,
                            int64_t gate_stride, int32_t heads, const void* residual,
                            const float* res_scale, float res_scale_value, float eps, int32_t fn,
                            void* out, int64_t rows, int32_t dim, int32_t dtype,
                            cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_norm(rows, dim, dtype, dtype, eps, res_scale, res_scale_value);
  if (st != KDA_OK) return st;
  if (fn != KDA_FN_SILU && fn != KDA_FN_SIGMOID) return KDA_ERR_INVALID_ARG;
  if (gate && (heads < 1 || rows % heads != 0 || gate_stride < (int64_t)heads * dim ||
               gate_stride >= (int64_t(1) << 31)))
    return KDA_ERR_INVALID_SHAPE;
  if (!weight || (rows > 0 && (!x || !out))) return KDA_ERR_NULL_POINTER;
  const size_t e = dtype == KDA_ROW_FP32 ? 4 : 2;
  if (!al_to(x, e) || !al_to(out, e) || !al_to(gate, e) || !al_to(residual, e) ||
      !al_to(weight, 4) || !al_to(res_scale, 4))
    return KDA_ERR_MISALIGNED;
  st = check_device();
  if (st != KDA_OK || rows == 0) return st;
  int num_sms = 0;
  if (sm_count(&num_sms) != KDA_OK) return KDA_ERR_CUDA;
  const NormPlan n = norm_plan(dim, dim % 8 == 0 && al16(x) && al16(out) && al16(residual) &&
                                        al16(gate) && (!gate || gate_stride * e % 16 == 0) && al16(weight) &&
                                        al16(res_scale));
  NormParams p = {};
  p.a = x, p.b = gate, p.c = residual, p.o0 = out, p.fn = fn;
  p.gate_stride = gate ? gate_stride : dim, p.heads = gate ? heads : 1;
  p.weight = weight, p.scale = res_scale, p.scale_value = res_scale_value, p.eps = eps;
  p.n_rows = rows, p.dim = dim;
  // bf16 rows of some lanes: as many blocks as run at once (2^27 gated values in rows of 128:
  // 137 us, with eight times as many 140), while fp32 rows, twice the bytes for the same work,
  // gain from more (7.0 TB/s against 6.4)
  const int per_sm = n.G && dtype == KDA_ROW_BF16 ? 4 : 32;
  return run_norm(pick_postnorm_fwd(n, dtype, dtype), n, p, norm_grid(n, rows, num_sms, per_sm), 0,
                  stream);
}

kda_status kda_postnorm_bwd(const void* dout, const void* x, const float* weight, const void* gate,
                            int64_t gate_stride, int32_t heads, const float* res_scale,
                            float res_scale_value, float eps, int32_t fn, void* dx, void* dgate,
                            float* dweight, float* dres_scale, int64_t rows, int32_t dim,
                            int32_t dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_norm(rows, dim, dtype, dtype, eps, res_scale, res_scale_value);
  if (st != KDA_OK) return st;
  if (fn != KDA_FN_SILU && fn != KDA_FN_SIGMOID) return KDA_ERR_INVALID_ARG;
  if (gate && (heads < 1 || rows % heads != 0 || gate_stride < (int64_t)heads * dim ||
               gate_stride >= (int64_t(1) << 31)))
    return KDA_ERR_INVALID_SHAPE;
  if (!weight || !dweight || !workspace || (rows > 0 && (!dout || !x || !dx)) || (dgate && !gate))
    return KDA_ERR_NULL_POINTER;
  const size_t e = dtype == KDA_ROW_FP32 ? 4 : 2;
  if (!al_to(x, e) || !al_to(dout, e) || !al_to(gate, e) || !al_to(dx, e) || !al_to(dgate, e) ||
      !al_to(weight, 4) || !al_to(res_scale, 4) || !al_to(dweight, 4) || !al_to(dres_scale, 4) ||
      !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  size_t need = 0;
  kda_norm_bwd_get_workspace_size(rows, dim, &need);
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  int num_sms = 0;
  if (sm_count(&num_sms) != KDA_OK) return KDA_ERR_CUDA;
  const NormPlan n = norm_plan(dim, dim % 8 == 0 && al16(dout) && al16(x) && al16(dx) &&
                                        al16(dgate) && al16(gate) &&
                                        (!gate || gate_stride * e % 16 == 0) && al16(weight) &&
                                        al16(res_scale));
  NormParams p = {};
  p.a = dout, p.b = gate, p.c = x, p.o0 = dx, p.o1 = dgate, p.fn = fn;
  p.gate_stride = gate ? gate_stride : dim, p.heads = gate ? heads : 1;
  p.weight = weight, p.scale = res_scale, p.scale_value = res_scale_value, p.eps = eps;
  p.n_rows = rows, p.dim = dim;
  p.want_scale = dres_scale != nullptr;
  return run_norm_bwd(pick_postnorm_bwd(n, dtype, dtype), n, p, num_sms, 24 * (int)e, workspace,
                      dweight, dres_scale, stream);
}

}  // extern "C"
