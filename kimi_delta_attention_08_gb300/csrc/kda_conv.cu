// kda_conv.cu -- the short causal depthwise convolution with its activation, forward and
// backward, over batched or packed sequences.
//
//   p[t] = bias + sum_{j < W} w[j] xx[t - W + 1 + j],   out = fn(p)
// with xx the sequence's rows after the W - 1 rows of its initial state.  Backward, with
// dp = dout fn'(p):
//   dxx[t] = sum_j w[j] dp[t + W - 1 - j]  (the rows before the sequence: dinitial_state)
//   dw[j] = sum_t dp[t] xx[t - W + 1 + j],   dbias = sum_t dp[t]
//
// Each value takes W multiplications, so the operator is bound by HBM: x is read once and
// out written once.  A thread holds 16 bytes of channels and walks a run of consecutive
// tokens with the last W - 1 rows in registers, so a row is loaded once per run, plus the
// W - 1 rows before the run (its neighbour's, from L2); rows are fetched kBatch at a
// time to keep that many loads in flight.
#include "kda_internal.h"
#include "kda_rows.cuh"
#include "../../include/kda_layer.h"

namespace kda {
namespace {

using namespace rows;

constexpr int kBatch = 8;     // rows in flight per thread
constexpr int kWarps = 4;

struct ConvParams {
  const void* x;
  int64_t x_stride;
  const float *weight, *bias;
  void* outs[KDA_CONV_MAX_OUTS];      // forward: out; backward: dout (read)
  int32_t out_lo[KDA_CONV_MAX_OUTS + 1];
  int32_t num_outs, dout_f32;
  const void* init;
  void* fin;
  const void* dfin;
  void* dx;
  float* dinit;
  float* part;                        // [token blocks][W + 1][C]
  const int64_t* cu;
  unsigned* status;
  int64_t T, total;
  int32_t N, C, fn;
  int32_t run;                        // tokens per run
  int32_t whole;                      // 1: run r is the whole of sequence r (batched)
  int32_t runs_per_warp;
  int64_t runs;
  int32_t tiles;                      // channel tiles; block = row block * tiles + tile
  int64_t run_blocks;                 // row blocks of runs; those after them hold states
};

// The channels of a thread: V consecutive ones (vector path), or V of them 32 apart.
template <int V, bool VEC>
struct Chan {
  int c0, step;
  __device__ Chan(int tile, int lane) {
    c0 = tile * 32 * V + (VEC ? lane * V : lane);
    step = VEC ? 1 : 32;
  }
  __device__ int at(int i) const { return c0 + i * step; }
};

// The buffer and offset that channel c of the concatenated outputs lies in.
__device__ __forceinline__ int out_of(const ConvParams& p, int c) {
  int i = 0;
#pragma unroll
  for (int k = 1; k < KDA_CONV_MAX_OUTS; ++k) i += (k < p.num_outs && c >= p.out_lo[k]) ? 1 : 0;
  return i;
}

template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_out(const ConvParams& p, const Chan<V, VEC>& ch, int64_t t,
                                          const float (&f)[V]) {
  if constexpr (VEC) {  // output boundaries are multiples of V
    const int o = out_of(p, ch.c0);
    const int w = p.out_lo[o + 1] - p.out_lo[o];
    store_row<T, V, true>(static_cast<T*>(p.outs[o]) + t * w + (ch.c0 - p.out_lo[o]), f, 1, 0);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = ch.at(i);
      if (c >= p.C) break;
      const int o = out_of(p, c);
      const int w = p.out_lo[o + 1] - p.out_lo[o];
      static_cast<T*>(p.outs[o])[t * w + (c - p.out_lo[o])] = from_f<T>(f[i]);
    }
  }
}

template <int W, int V, bool VEC>
__device__ __forceinline__ void load_weights(const ConvParams& p, const Chan<V, VEC>& ch,
                                             float (&w)[W][V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = ch.at(i);
    const bool ok = VEC || c < p.C;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = ok ? __ldg(p.weight + (int64_t)c * W + j) : 0.f;
    b[i] = ok && p.bias ? __ldg(p.bias + c) : 0.f;
  }
}

// Row `pos` (counted from the sequence's first token, negative: its initial state).
template <typename T, int W, int V, bool VEC>
__device__ __forceinline__ void load_xx(const ConvParams& p, const Chan<V, VEC>& ch, int n,
                                        int64_t bos, int64_t pos, float (&f)[V]) {
  Raw<T, V> r = {};
  if (pos >= 0)
    load_row<T, V, VEC>(r, static_cast<const T*>(p.x) + (bos + pos) * p.x_stride + ch.c0, ch.step,
                        p.C - ch.c0);
  else if (p.init && pos >= 1 - W)
    load_row<T, V, VEC>(r,
                        static_cast<const T*>(p.init) + ((int64_t)n * (W - 1) + pos + W - 1) * p.C + ch.c0,
                        ch.step, p.C - ch.c0);
  unpack(r, f);
}

__device__ __forceinline__ void bounds_of(const ConvParams& p, int n, int64_t& bos, int64_t& eos) {
  if (p.cu) {
    bos = __ldg(p.cu + n);
    eos = __ldg(p.cu + n + 1);
    bos = bos < 0 ? 0 : bos;
    eos = eos > p.total ? p.total : eos;
  } else {
    bos = (int64_t)n * p.T;
    eos = bos + p.T;
  }
}

template <typename T, int W, int V, bool VEC>
__device__ __forceinline__ void final_rows(const ConvParams& p, const Chan<V, VEC>& ch, int n) {
  int64_t bos, eos;
  bounds_of(p, n, bos, eos);
  float f[W - 1][V];
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {  // all read before any is written: fin may be init
    const int64_t pos = (eos > bos ? eos - bos : 0) - (W - 1) + r;
    load_xx<T, W, V, VEC>(p, ch, n, bos, pos, f[r]);
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r)
    store_row<T, V, VEC>(static_cast<T*>(p.fin) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0, f[r],
                         ch.step, p.C - ch.c0);
}

template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) conv_fwd_kernel(const ConvParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x % p.tiles;
  const int64_t rblk = blockIdx.x / p.tiles;
  const Chan<V, VEC> ch(tile, lane);
  if (p.status && blockIdx.x == 0 && warp == 0) {
    if (p.cu) check_seqlens(p.cu, p.N, p.total, p.status, kDevStatusBadSeqlens);
    else if (lane == 0) *p.status = 0u;
  }
  const bool mine = ch.c0 < p.C;
  if (rblk >= p.run_blocks) {  // final states of whole sequences
    const int n = (int)(rblk - p.run_blocks) * kWarps + warp;
    if (n < p.N && mine) final_rows<T, W, V, VEC>(p, ch, n);
    return;
  }
  float w[W][V], b[V];
  load_weights<W, V, VEC>(p, ch, w, b);
  int64_t run = (rblk * kWarps + warp) * p.runs_per_warp;
  const int64_t run_end = min(run + p.runs_per_warp, p.runs);
  for (; run < run_end; ++run) {
    int n;
    int64_t t, end, bos, eos;
    if (p.cu) {
      t = run * p.run;
      end = min(t + p.run, p.total);
      n = find_sequence(p.cu, p.N, t);
      bounds_of(p, n, bos, eos);
      if (t < bos) continue;  // inconsistent cu_seqlens
    } else {
      n = (int)(p.whole ? run : run * p.run / p.T);
      t = p.whole ? run * p.T : run * p.run;
      end = p.whole ? t + p.T : min(t + p.run, p.total);
      bounds_of(p, n, bos, eos);
    }
    float h[W - 1][V];  // rows t - W + 1 .. t - 1
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
#pragma unroll
      for (int i = 0; i < V; ++i) h[r][i] = 0.f;
      if (mine) load_xx<T, W, V, VEC>(p, ch, n, bos, t - bos - (W - 1) + r, h[r]);
    }
    for (; t < end; t += kBatch) {
      Raw<T, V> raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (mine && t + u < end)
          load_row<T, V, VEC>(raw[u], static_cast<const T*>(p.x) + (t + u) * p.x_stride + ch.c0,
                              ch.step, p.C - ch.c0);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (t + u >= end) break;
        if (t + u >= eos) {  // the next sequence that has tokens
          while (t + u >= eos && n + 1 < p.N) bounds_of(p, ++n, bos, eos);
          if (t + u >= eos) break;  // rows of no sequence
#pragma unroll
          for (int r = 0; r < W - 1; ++r)
            if (mine) load_xx<T, W, V, VEC>(p, ch, n, bos, t + u - bos - (W - 1) + r, h[r]);
        }
        float xv[V], y[V];
        unpack(raw[u], xv);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float s = fmaf(w[W - 1][i], xv[i], b[i]);
#pragma unroll
          for (int r = 0; r < W - 1; ++r) s = fmaf(w[r][i], h[r][i], s);
          y[i] = p.fn == KDA_FN_SILU ? s * sigmoid(s) : s;
        }
        if (mine && t + u >= bos) store_out<T, V, VEC>(p, ch, t + u, y);
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
          for (int r = 0; r + 1 < W - 1; ++r) h[r][i] = h[r + 1][i];
          h[W - 2][i] = xv[i];
        }
      }
    }
    if (p.whole && p.fin && mine) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r)
        store_row<T, V, VEC>(static_cast<T*>(p.fin) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0,
                             h[r], ch.step, p.C - ch.c0);
    }
  }
}

template <typename T, int W, int V, bool VEC>
__device__ __forceinline__ void load_dout(const ConvParams& p, const Chan<V, VEC>& ch, int64_t t,
                                          float (&f)[V]) {
  if constexpr (VEC) {
    const int o = out_of(p, ch.c0);
    const int64_t at = t * (p.out_lo[o + 1] - p.out_lo[o]) + (ch.c0 - p.out_lo[o]);
    if (p.dout_f32) {
      Raw<float, V> r;
      load_words(r.w, static_cast<const float*>(p.outs[o]) + at);
      unpack(r, f);
    } else {
      Raw<T, V> r;
      load_words(r.w, static_cast<const T*>(p.outs[o]) + at);
      unpack(r, f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = ch.at(i);
      f[i] = 0.f;
      if (c >= p.C) continue;
      const int o = out_of(p, c);
      const int64_t at = t * (p.out_lo[o + 1] - p.out_lo[o]) + (c - p.out_lo[o]);
      f[i] = p.dout_f32 ? __ldg(static_cast<const float*>(p.outs[o]) + at)
                        : to_f(static_cast<const T*>(p.outs[o])[at]);
    }
  }
}

// Backward: a run emits the dx rows of its tokens.  dx[t] needs dp[t .. t + W - 1], so the
// run computes dp for W - 1 tokens more than it emits (never past the sequence's end) and
// emits row t - W + 1 at step t; before a sequence's first token the emitted rows are
// those of dinitial_state.
template <typename T, int W, int V, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) conv_bwd_kernel(const ConvParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile = blockIdx.x % p.tiles;
  const int64_t rblk = blockIdx.x / p.tiles;
  const Chan<V, VEC> ch(tile, lane);
  if (p.status && blockIdx.x == 0 && warp == 0) {
    if (p.cu) check_seqlens(p.cu, p.N, p.total, p.status, kDevStatusBadSeqlens);
    else if (lane == 0) *p.status = 0u;
  }
  const bool mine = ch.c0 < p.C;
  if (rblk >= p.run_blocks) {  // empty sequences: dinitial = dfinal
    const int n = (int)(rblk - p.run_blocks) * kWarps + warp;
    if (n >= p.N || !mine) return;
    int64_t bos, eos;
    bounds_of(p, n, bos, eos);
    if (eos > bos) return;
    for (int r = 0; r < W - 1; ++r) {
      const int64_t at = ((int64_t)n * (W - 1) + r) * p.C + ch.c0;
      Raw<T, V> raw = {};
      float f[V];
      if (p.dfin) load_row<T, V, VEC>(raw, static_cast<const T*>(p.dfin) + at, ch.step, p.C - ch.c0);
      unpack(raw, f);
      store_row<float, V, VEC>(p.dinit + at, f, ch.step, p.C - ch.c0);
    }
    return;
  }
  float w[W][V], b[V], dw[W][V] = {}, db[V] = {};
  load_weights<W, V, VEC>(p, ch, w, b);
  int64_t run = (rblk * kWarps + warp) * p.runs_per_warp;
  const int64_t run_end = min(run + p.runs_per_warp, p.runs);
  for (; run < run_end; ++run) {
    const int64_t t0 = run * p.run, t1 = min(t0 + p.run, p.total);
    int n = p.cu ? find_sequence(p.cu, p.N, t0) : (int)(t0 / p.T);
    int64_t a = t0;
    while (a < t1) {  // pieces of one sequence each
      int64_t bos, eos;
      bounds_of(p, n, bos, eos);
      if (a >= eos) {
        if (++n >= p.N) break;
        continue;
      }
      if (a < bos) break;  // inconsistent cu_seqlens
      const int64_t end = min(eos, t1);
      float h[W - 1][V], q[W - 1][V];  // xx and dp of the last W - 1 tokens
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[r][i] = q[r][i] = 0.f;
        if (mine) load_xx<T, W, V, VEC>(p, ch, n, bos, a - bos - (W - 1) + r, h[r]);
      }
      for (int64_t t = a; t < end + W - 1; ++t) {
        float d[V] = {};
        if (t < eos && mine) {
          float xv[V], dy[V];
          Raw<T, V> raw;
          load_row<T, V, VEC>(raw, static_cast<const T*>(p.x) + t * p.x_stride + ch.c0, ch.step,
                              p.C - ch.c0);
          load_dout<T, W, V, VEC>(p, ch, t, dy);
          unpack(raw, xv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float s = fmaf(w[W - 1][i], xv[i], b[i]);
#pragma unroll
            for (int r = 0; r < W - 1; ++r) s = fmaf(w[r][i], h[r][i], s);
            d[i] = dy[i];
            if (p.fn == KDA_FN_SILU) {
              const float g = sigmoid(s);
              d[i] *= g * fmaf(s, 1.f - g, 1.f);
            }
            if (t < end) {
#pragma unroll
              for (int r = 0; r < W - 1; ++r) dw[r][i] = fmaf(d[i], h[r][i], dw[r][i]);
              dw[W - 1][i] = fmaf(d[i], xv[i], dw[W - 1][i]);
              db[i] += d[i];
            }
#pragma unroll
            for (int r = 0; r + 1 < W - 1; ++r) h[r][i] = h[r + 1][i];
            h[W - 2][i] = xv[i];
          }
        }
        // emit row te: dxx[te] = sum_s w[W - 1 - s] dp[te + s], s = 0 .. W - 1
        const int64_t te = t - (W - 1);
        if (mine && (te >= a || (a == bos && p.dinit))) {
          float dx[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float s = w[0][i] * d[i];
#pragma unroll
            for (int r = 0; r < W - 1; ++r) s = fmaf(w[W - 1 - r][i], q[r][i], s);
            dx[i] = s;
          }
          if (p.dfin && te >= eos - (W - 1)) {
            Raw<T, V> raw;
            float f[V];
            load_row<T, V, VEC>(raw,
                                static_cast<const T*>(p.dfin) +
                                    ((int64_t)n * (W - 1) + te - eos + W - 1) * p.C + ch.c0,
                                ch.step, p.C - ch.c0);
            unpack(raw, f);
#pragma unroll
            for (int i = 0; i < V; ++i) dx[i] += f[i];
          }
          if (te >= a)
            store_row<T, V, VEC>(static_cast<T*>(p.dx) + te * p.C + ch.c0, dx, ch.step, p.C - ch.c0);
          else
            store_row<float, V, VEC>(p.dinit + ((int64_t)n * (W - 1) + te - bos + W - 1) * p.C + ch.c0,
                                     dx, ch.step, p.C - ch.c0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
          for (int r = 0; r + 1 < W - 1; ++r) q[r][i] = q[r + 1][i];
          q[W - 2][i] = d[i];
        }
      }
      a = end;
    }
    const float zero[V] = {};
    for (; a < t1 && mine; ++a)  // rows of no sequence
      store_row<T, V, VEC>(static_cast<T*>(p.dx) + a * p.C + ch.c0, zero, ch.step, p.C - ch.c0);
  }
  // the block's warps added in their order, then one partial row per block
  __shared__ float acc[W + 1][32 * V + 1];
  for (int k = 0; k < kWarps; ++k) {
    if (warp == k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * 32 + lane;
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j][c] = k ? acc[j][c] + dw[j][i] : dw[j][i];
        acc[W][c] = k ? acc[W][c] + db[i] : db[i];
      }
    }
    __syncthreads();
  }
  float* out = p.part + rblk * (W + 1) * p.C;
  for (int e = threadIdx.x; e < 32 * V; e += blockDim.x) {
    // channel lane * V + i lies at i * 32 + lane on the vector path
    const int s = VEC ? (e % V) * 32 + e / V : e;
    const int c = tile * 32 * V + e;
    if (c >= p.C) continue;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
      // columns of the sums: the weights' [C][W] first, then the biases
      const int64_t col = j < W ? (int64_t)c * W + j : (int64_t)p.C * W + c;
      out[col] = acc[j][s];
    }
  }
}

bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <bool BWD, typename T, int V, bool VEC>
void (*conv_kernel_w(int width))(ConvParams) {
  if constexpr (BWD)
    return width == 2   ? conv_bwd_kernel<T, 2, V, VEC>
           : width == 3 ? conv_bwd_kernel<T, 3, V, VEC>
                        : conv_bwd_kernel<T, 4, V, VEC>;
  else
    return width == 2   ? conv_fwd_kernel<T, 2, V, VEC>
           : width == 3 ? conv_fwd_kernel<T, 3, V, VEC>
                        : conv_fwd_kernel<T, 4, V, VEC>;
}

constexpr int kFwdV16 = 8, kFwdV32 = 4, kBwdV = 4;

template <bool BWD>
void (*conv_kernel(bool f32, bool vec, int width))(ConvParams) {
  constexpr int V16 = BWD ? kBwdV : kFwdV16, V32 = BWD ? kBwdV : kFwdV32;
  if (f32) return vec ? conv_kernel_w<BWD, float, V32, true>(width)
                      : conv_kernel_w<BWD, float, V32, false>(width);
  return vec ? conv_kernel_w<BWD, bf16, V16, true>(width)
             : conv_kernel_w<BWD, bf16, V16, false>(width);
}

int vec_of(bool bwd, bool f32) { return bwd ? kBwdV : f32 ? kFwdV32 : kFwdV16; }

// Tokens per run and runs per warp of the backward: a run of 64 tokens costs 5 % more
// rows than it emits; a block's runs are consecutive.
constexpr int kBwdRun = 64;
int64_t bwd_blocks(int64_t total) { return (total + kBwdRun * kWarps - 1) / (kBwdRun * kWarps); }

kda_status check_conv(const void* x, int64_t x_stride, const float* weight, const float* bias,
                      const void* const* outs, const int32_t* out_channels, int32_t num_outs,
                      const void* init, const void* fin, const int64_t* cu, int64_t B, int64_t T,
                      int32_t C, int32_t* N, int32_t width, int32_t fn, int32_t dtype,
                      int32_t out_dtype) {
  if (!weight || !outs || !out_channels) return KDA_ERR_NULL_POINTER;
  if (B < 1 || T < 0 || C < 1 || width < 2 || width > KDA_CONV_MAX_WIDTH || x_stride < C ||
      x_stride >= (int64_t(1) << 31) || B >= (int64_t(1) << 31) || T >= (int64_t(1) << 31) ||
      B * T >= (int64_t(1) << 31) || num_outs < 1 || num_outs > KDA_CONV_MAX_OUTS)
    return KDA_ERR_INVALID_SHAPE;
  int64_t sum = 0;
  for (int i = 0; i < num_outs; ++i) {
    if (out_channels[i] < 1) return KDA_ERR_INVALID_SHAPE;
    sum += out_channels[i];
  }
  if (sum != C) return KDA_ERR_INVALID_SHAPE;
  if (cu) {
    if (B != 1 || *N < 1) return KDA_ERR_INVALID_SHAPE;
  } else {
    *N = (int32_t)B;
  }
  if ((fn != KDA_FN_NONE && fn != KDA_FN_SILU) || (dtype != KDA_ROW_BF16 && dtype != KDA_ROW_FP32) ||
      (out_dtype != KDA_ROW_FP32 && out_dtype != dtype))
    return KDA_ERR_INVALID_ARG;
  const size_t e = dtype == KDA_ROW_FP32 ? 4 : 2, oe = out_dtype == KDA_ROW_FP32 ? 4 : 2;
  if (B * T > 0 && !x) return KDA_ERR_NULL_POINTER;
  for (int i = 0; i < num_outs; ++i) {
    if (B * T > 0 && !outs[i]) return KDA_ERR_NULL_POINTER;
    if (!al_to(outs[i], oe)) return KDA_ERR_MISALIGNED;
  }
  if (!al_to(x, e) || !al_to(init, e) || !al_to(fin, e) || !al_to(weight, 4) || !al_to(bias, 4) ||
      !al_to(cu, 8))
    return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

// Whether every row starts on 16 bytes, for V elements a thread.
bool conv_vec(const void* x, int64_t x_stride, const void* const* outs,
              const int32_t* out_channels, int32_t num_outs, const void* init, const void* fin,
              int32_t C, int V, size_t e, size_t oe) {
  bool ok = C % V == 0 && x_stride * e % 16 == 0 && al_to(x, 16) && al_to(init, 16) &&
            al_to(fin, 16);
  for (int i = 0; i < num_outs; ++i)
    ok = ok && out_channels[i] % V == 0 && al_to(outs[i], 16) && out_channels[i] * oe % 16 == 0;
  return ok && C * e % 16 == 0;
}

void fill(ConvParams& p, const void* x, int64_t x_stride, const float* weight, const float* bias,
          const void* const* outs, const int32_t* out_channels, int32_t num_outs, const void* init,
          const int64_t* cu, int64_t B, int64_t T, int32_t C, int32_t N, int32_t fn) {
  p.x = x, p.x_stride = x_stride, p.weight = weight, p.bias = bias, p.init = init, p.cu = cu;
  p.num_outs = num_outs;
  p.out_lo[0] = 0;
  for (int i = 0; i < KDA_CONV_MAX_OUTS; ++i) {
    p.outs[i] = i < num_outs ? const_cast<void*>(outs[i]) : nullptr;
    p.out_lo[i + 1] = p.out_lo[i] + (i < num_outs ? out_channels[i] : 0);
  }
  p.T = T, p.total = B * T, p.N = N, p.C = C, p.fn = fn;
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_conv_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        void* const* outs, const int32_t* out_channels, int32_t num_outs,
                        const void* initial_state, void* final_state, const int64_t* cu_seqlens,
                        int64_t B, int64_t T, int32_t C, int32_t N, int32_t width, int32_t fn,
                        int32_t dtype, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_conv(x, x_stride, weight, bias, outs, out_channels, num_outs,
                             initial_state, final_state, cu_seqlens, B, T, C, &N, width, fn, dtype,
                             dtype);
  if (st != KDA_OK) return st;
  if (workspace && workspace_bytes < KDA_STATUS_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  if (!al_to(workspace, 128)) return KDA_ERR_MISALIGNED;
  st = check_device();
  if (st != KDA_OK) return st;
  int num_sms = 0;
  if (sm_count(&num_sms) != KDA_OK) return KDA_ERR_CUDA;
  const bool f32 = dtype == KDA_ROW_FP32;
  const int V = vec_of(false, f32);
  const bool vec = conv_vec(x, x_stride, outs, out_channels, num_outs, initial_state, final_state,
                            C, V, f32 ? 4 : 2, f32 ? 4 : 2);
  ConvParams p = {};
  fill(p, x, x_stride, weight, bias, outs, out_channels, num_outs, initial_state, cu_seqlens, B, T,
       C, N, fn);
  p.fin = final_state;
  p.status = static_cast<unsigned*>(workspace);
  const int64_t tiles = (C + 32 * V - 1) / (32 * V);
  // A short batched sequence is one run of its own, which also writes its final state.
  p.whole = !cu_seqlens && T <= 32 && T > 0;
  if (p.whole) {
    p.run = (int32_t)T;
    p.runs = N;
  } else {
    p.run = 32;
    // runs of batched input do not straddle sequences: they are cut like packed ones
    p.runs = (p.total + p.run - 1) / p.run;
  }
  p.runs_per_warp = 1;
  const int64_t run_blocks = (p.runs + kWarps * p.runs_per_warp - 1) / (kWarps * p.runs_per_warp);
  const bool split_state = final_state && !p.whole;
  const bool same = final_state && final_state == initial_state;
  const int64_t state_blocks = split_state ? ((int64_t)N + kWarps - 1) / kWarps : 0;
  if ((run_blocks + state_blocks) * tiles >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
  auto kernel = conv_kernel<false>(f32, vec, width);
  p.tiles = (int32_t)tiles;
  p.run_blocks = run_blocks;
  // An in-place state is written by a second launch, after every run has read it.
  const int64_t blocks = (run_blocks + (same ? 0 : state_blocks)) * tiles;
  if (blocks > 0) {
    kernel<<<(unsigned)blocks, 32 * kWarps, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  } else if (p.status) {
    if (cudaMemsetAsync(p.status, 0, 4, stream) != cudaSuccess) return KDA_ERR_CUDA;
  }
  if (same && state_blocks > 0) {
    p.status = nullptr;
    p.run_blocks = 0;
    kernel<<<(unsigned)(state_blocks * tiles), 32 * kWarps, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  }
  return KDA_OK;
}

kda_status kda_conv_bwd_get_workspace_size(int64_t total_tokens, int32_t C, int32_t width,
                                           size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  if (total_tokens < 0 || total_tokens >= (int64_t(1) << 31) || C < 1 || width < 2 ||
      width > KDA_CONV_MAX_WIDTH)
    return KDA_ERR_INVALID_SHAPE;
  *bytes = KDA_STATUS_BYTES +
           (size_t)kda::bwd_blocks(total_tokens) * (width + 1) * (size_t)C * sizeof(float);
  return KDA_OK;
}

kda_status kda_conv_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const void* const* douts, const int32_t* out_channels, int32_t num_outs,
                        int32_t dout_dtype, const void* initial_state, const void* dfinal_state,
                        const int64_t* cu_seqlens, void* dx, float* dweight, float* dbias,
                        float* dinitial_state, int64_t B, int64_t T, int32_t C, int32_t N,
                        int32_t width, int32_t fn, int32_t dtype, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_conv(x, x_stride, weight, bias, douts, out_channels, num_outs,
                             initial_state, dfinal_state, cu_seqlens, B, T, C, &N, width, fn, dtype,
                             dout_dtype);
  if (st != KDA_OK) return st;
  if (!dweight || !workspace || (B * T > 0 && !dx)) return KDA_ERR_NULL_POINTER;
  const bool f32 = dtype == KDA_ROW_FP32;
  if (!al_to(dx, f32 ? 4 : 2) || !al_to(dweight, 4) || !al_to(dbias, 4) ||
      !al_to(dinitial_state, 4) || !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  size_t need = 0;
  st = kda_conv_bwd_get_workspace_size(B * T, C, width, &need);
  if (st != KDA_OK) return st;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  const int V = vec_of(true, f32);
  const bool vec = conv_vec(x, x_stride, douts, out_channels, num_outs, initial_state,
                            dfinal_state, C, V, f32 ? 4 : 2, dout_dtype == KDA_ROW_FP32 ? 4 : 2) &&
                   al_to(dx, 16) && al_to(dinitial_state, 16);
  ConvParams p = {};
  fill(p, x, x_stride, weight, bias, douts, out_channels, num_outs, initial_state, cu_seqlens, B,
       T, C, N, fn);
  p.dout_f32 = dout_dtype == KDA_ROW_FP32;
  p.dfin = dfinal_state, p.dx = dx, p.dinit = dinitial_state;
  p.status = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
  p.run = kBwdRun;
  p.runs_per_warp = 1;
  p.runs = (p.total + p.run - 1) / p.run;
  const int64_t tiles = (C + 32 * V - 1) / (32 * V);
  const int64_t blocks = bwd_blocks(p.total);
  // empty sequences can only come with cu_seqlens or T = 0
  const int64_t state_blocks =
      dinitial_state && (cu_seqlens || T == 0) ? ((int64_t)N + kWarps - 1) / kWarps : 0;
  if ((blocks + state_blocks) * tiles >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
  p.tiles = (int32_t)tiles;
  p.run_blocks = blocks;
  if (blocks + state_blocks > 0) {
    conv_kernel<true>(f32, vec, width)<<<(unsigned)((blocks + state_blocks) * tiles), 32 * kWarps,
                                         0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  } else if (cudaMemsetAsync(p.status, 0, 4, stream) != cudaSuccess) {
    return KDA_ERR_CUDA;
  }
  if (launch_column_sums(p.part, blocks, (int64_t)(width + 1) * C, (int64_t)width * C, C,
                         dweight, dbias, nullptr, stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"
