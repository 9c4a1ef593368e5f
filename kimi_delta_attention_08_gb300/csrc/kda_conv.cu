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
// out written once.  A thread holds 16 bytes of channels and walks a run of 8 to 256
// tokens with the last W - 1 rows in registers, so a row is loaded once per run, plus the
// W - 1 rows before the run (its neighbour's, from L2).  The next rows are on their way
// into shared memory meanwhile, asked for by the thread that reads them, so without a barrier.
//
// Device time, and bytes of the rows over it (SiLU, width 4, bf16): 74,080 packed tokens of
// 6,144 channels with states 284 us (6.4 TB/s; 413 with the next rows in registers; fp32 538,
// 6.8 TB/s); single tokens of 256 sequences of 12,288 channels 9.8 us (fp32 17.6); backward of
// 32,768 tokens of 12,288 channels 441 us (5.5 TB/s; 636 with the rows in registers; fp32 723,
// 6.7 TB/s; bf16 with fp32 gradients of the outputs 497, 6.5 TB/s), which the FMA pipe's latency
// with 12 warps of 164 registers per SM keeps from the 356 us that its bytes take.  The weights'
// gradients are summed in fp32 and within 2.3e-7 of their 64-bit values over 32,768 tokens.
#include "kda_internal.h"
#include "kda_rows.cuh"
#include "../../include/kda_layer.h"

#include <type_traits>

namespace kda {
namespace {

using namespace rows;

constexpr int kRing = 8;      // rows of a thread in shared memory or on their way (vector path)
constexpr int kBatch = 4;     // rows that it loads together (scalar path)
constexpr int kWarps = 4;
constexpr int kStepSeqs = 4;  // sequences per thread of the single-token kernel

struct ConvParams {
  const void* x;
  int64_t x_stride;
  const float *weight, *bias;
  void* outs[KDA_CONV_MAX_OUTS];      // forward: out; backward: dout (read)
  int32_t out_lo[KDA_CONV_MAX_OUTS + 1];
  int32_t num_outs;
  const void* init;
  void* fin;
  const void* dfin;
  void* dx;
  float* dinit;
  float* part;                        // [token blocks][W + 1][C]
  const int64_t* cu;
  unsigned* status;
  int64_t T, total;
  int32_t N, C;
  int32_t run;                        // tokens per run
  int32_t whole;                      // 1: run r is the whole of sequence r (batched)
  int32_t weight_vec;                 // weight is 16-byte aligned
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

// The rows of the concatenated tensors outs (out or dout) that a thread's channels lie in: on
// the vector path in one of them (boundaries are multiples of V), so its place is found
// once; on the scalar path likewise where there is only one.
template <typename TQ, int V, bool VEC>
struct OutRows {
  using TD = std::remove_const_t<TQ>;
  TQ* base;
  int width;
  __device__ OutRows(const ConvParams& p, const Chan<V, VEC>& ch) {
    const int o = VEC ? out_of(p, ch.c0) : 0;
    width = p.out_lo[o + 1] - p.out_lo[o];
    base = static_cast<TQ*>(p.outs[o]) + (ch.c0 - p.out_lo[o]);
  }
  __device__ TQ* at(const ConvParams& p, const Chan<V, VEC>& ch, int64_t t, int i) const {
    const int c = ch.at(i), o = out_of(p, c);
    return static_cast<TQ*>(p.outs[o]) + t * (p.out_lo[o + 1] - p.out_lo[o]) + (c - p.out_lo[o]);
  }
  __device__ void store(const ConvParams& p, const Chan<V, VEC>& ch, int64_t t,
                        const float (&f)[V]) const {
    if (VEC || p.num_outs == 1) {
      store_row<TD, V, VEC>(base + t * width, f, ch.step, p.C - ch.c0);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ch.at(i) < p.C) *at(p, ch, t, i) = from_f<TD>(f[i]);
    }
  }
  __device__ void load(const ConvParams& p, const Chan<V, VEC>& ch, int64_t t,
                       Raw<TD, V>& r) const {
    if (VEC || p.num_outs == 1) {
      load_row<TD, V, VEC>(r, base + t * width, ch.step, p.C - ch.c0);
    } else {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = ch.at(i) < p.C ? to_f(*at(p, ch, t, i)) : 0.f;
      pack(r, f);
    }
  }
};

// Weights and biases of a thread's channels, in pairs of channels.
template <int W, int V, bool VEC>
__device__ __forceinline__ void load_weights(const ConvParams& p, const Chan<V, VEC>& ch,
                                             pair (&w)[W][V / 2], pair (&b)[V / 2]) {
  float f[V][W], bf[V];
  if (VEC && p.weight_vec) {  // W * V floats in a row, 16-byte aligned
    uint32_t raw[V * W] = {};
    if (ch.c0 < p.C) load_words(raw, p.weight + (int64_t)ch.c0 * W);
#pragma unroll
    for (int i = 0; i < V * W; ++i) f[i / W][i % W] = __uint_as_float(raw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j)
        f[i][j] = ch.at(i) < p.C ? __ldg(p.weight + (int64_t)ch.at(i) * W + j) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) bf[i] = p.bias && ch.at(i) < p.C ? __ldg(p.bias + ch.at(i)) : 0.f;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    b[i / 2] = pr(bf[i], bf[i + 1]);
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i / 2] = pr(f[i][j], f[i + 1][j]);
  }
}

template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Raw<T, V>& r, pair (&v)[V / 2]) {
  float f[V];
  unpack(r, f);
#pragma unroll
  for (int i = 0; i < V; i += 2) v[i / 2] = pr(f[i], f[i + 1]);
}
template <int V>
__device__ __forceinline__ void from_pairs(const pair (&v)[V / 2], float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) f[i] = un(v[i / 2]).x, f[i + 1] = un(v[i / 2]).y;
}

// The pre-activation from the last W - 1 rows and the current one.
template <int W, int V>
__device__ __forceinline__ void pre_activation(const pair (&w)[W][V / 2], const pair (&b)[V / 2],
                                               const pair (&h)[W - 1][V / 2],
                                               const pair (&x)[V / 2], pair (&s)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    s[i] = pfma(w[W - 1][i], x[i], b[i]);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) s[i] = pfma(w[r][i], h[r][i], s[i]);
  }
}
template <int W, int V>
__device__ __forceinline__ void shift(pair (&h)[W - 1][V / 2], const pair (&x)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
#pragma unroll
    for (int r = 0; r + 1 < W - 1; ++r) h[r][i] = h[r + 1][i];
    h[W - 2][i] = x[i];
  }
}

// Row `pos` (counted from the sequence's first token, negative: its initial state).
template <typename T, int W, int V, bool VEC>
__device__ __forceinline__ void load_xx(const ConvParams& p, const Chan<V, VEC>& ch, int n,
                                        int64_t bos, int64_t pos, Raw<T, V>& r) {
  r = Raw<T, V>{};
  if (pos >= 0)
    load_row<T, V, VEC>(r, static_cast<const T*>(p.x) + (bos + pos) * p.x_stride + ch.c0, ch.step,
                        p.C - ch.c0);
  else if (p.init && pos >= 1 - W)  // the final state may be this buffer
    load_row<T, V, VEC, true>(r,
                              static_cast<const T*>(p.init) + ((int64_t)n * (W - 1) + pos + W - 1) * p.C + ch.c0,
                              ch.step, p.C - ch.c0);
}

// A thread's rows on their way through shared memory: kRing slots, a group of copies for
// each token (an empty one past the end), read back by the thread that asked for them.
template <typename T, int V>
struct alignas(V * sizeof(T)) RingSlot {
  T v[V];
};
template <typename T, int V>
struct Ring {
  RingSlot<T, V>* base;  // [kRing][32] of a warp, at this lane
  __device__ explicit Ring(RingSlot<T, V>* b) : base(b) {}
  __device__ void copy(int slot, const T* from, bool ok) {
    RingSlot<T, V>* const to = base + (slot % kRing) * 32;
    if (!ok) return;
    if constexpr (sizeof(RingSlot<T, V>) == 16) ptx::cp_async16(to, from, 16);
    else ptx::cp_async8(to, from);
  }
  __device__ void issue(int slot, const T* from, bool ok) {
    copy(slot, from, ok);
    ptx::cp_async_commit();
  }
  __device__ void read(int slot, Raw<T, V>& r) { load_words<true>(r.w, base + (slot % kRing) * 32); }
};

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
  Raw<T, V> f[W - 1];
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {  // all read before any is written: fin may be init
    const int64_t pos = (eos > bos ? eos - bos : 0) - (W - 1) + r;
    load_xx<T, W, V, VEC>(p, ch, n, bos, pos, f[r]);
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {
    float v[V];
    unpack(f[r], v);
    store_row<T, V, VEC>(static_cast<T*>(p.fin) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0, v,
                         ch.step, p.C - ch.c0);
  }
}

template <typename T, int W, int V, bool VEC, bool SILU>
__global__ void __launch_bounds__(32 * kWarps) conv_fwd_kernel(const ConvParams p) {
  __shared__ RingSlot<T, V> s_ring[VEC ? kWarps : 1][VEC ? kRing : 1][32];
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
  const int64_t run = rblk * kWarps + warp;
  if (run >= p.runs) return;
  const int64_t t0 = p.whole ? run * p.T : run * p.run;
  const int64_t t1 = p.whole ? t0 + p.T : min(t0 + p.run, p.total);
  const T* const px = static_cast<const T*>(p.x) + ch.c0;
  Ring<T, V> ring(&s_ring[VEC ? warp : 0][0][lane]);
  const T* next = px + t0 * p.x_stride;  // the row to ask for next
  auto start = [&](int rows) {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i, next += p.x_stride) ring.issue(i, next, mine && i < rows);
  };
  // the first rows are on their way while the sequence is looked up
  if constexpr (VEC) start((int)(t1 - t0));
  const OutRows<T, V, VEC> out(p, ch);
  pair w[W][V / 2], b[V / 2];
  load_weights<W, V, VEC>(p, ch, w, b);
  int n = p.cu ? find_sequence(p.cu, p.N, t0) : (int)(t0 / p.T);
  pair h[W - 1][V / 2];  // rows t - W + 1 .. t - 1
  auto emit = [&](int64_t at, const Raw<T, V>& r) {
    pair x[V / 2], s[V / 2];
    to_pairs(r, x);
    pre_activation<W, V>(w, b, h, x, s);
    if constexpr (SILU) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) s[i] = silu<T>(s[i]);
    }
    float y[V];
    from_pairs<V>(s, y);
    if (mine) out.store(p, ch, at, y);
    shift<W, V>(h, x);
  };
  for (int64_t a = t0; a < t1;) {  // pieces of one sequence each
    int64_t bos, eos;
    bounds_of(p, n, bos, eos);
    if (a >= eos) {
      if (++n >= p.N) break;  // rows of no sequence
      continue;
    }
    if (a < bos) break;  // inconsistent cu_seqlens
    const int64_t end = min(eos, t1);
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      Raw<T, V> x = {};
      if (mine) load_xx<T, W, V, VEC>(p, ch, n, bos, a - bos - (W - 1) + r, x);
      to_pairs(x, h[r]);
    }
    if constexpr (VEC) {
      const int rows = (int)(end - a);
      if (a > t0) {  // another piece: the ring starts anew
        ptx::cp_async_wait_all();
        next = px + a * p.x_stride;
        start(rows);
      }
      auto turn = [&](int i, int slot) {  // row i of the piece
        ring.issue(slot + kRing - 1, next, mine && i + kRing - 1 < rows);
        next += p.x_stride;
        ptx::cp_async_wait<kRing - 1>();
        Raw<T, V> x;
        ring.read(slot, x);
        emit(a + i, x);
      };
      int i = 0;
      for (; i + kRing <= rows; i += kRing) {
#pragma unroll
        for (int u = 0; u < kRing; ++u) turn(i + u, u);
      }
      for (; i < rows; ++i) turn(i, i);
    } else {
      for (int64_t t = a; t < end; t += kBatch) {
        Raw<T, V> x[kBatch] = {};
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (mine && t + u < end)
            load_row<T, V, VEC>(x[u], px + (t + u) * p.x_stride, ch.step, p.C - ch.c0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (t + u < end) emit(t + u, x[u]);
      }
    }
    a = end;
  }
  if constexpr (VEC) ptx::cp_async_wait_all();
  if (p.whole && p.fin && mine) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      float f[V];
      from_pairs<V>(h[r], f);
      store_row<T, V, VEC>(static_cast<T*>(p.fin) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0, f,
                           ch.step, p.C - ch.c0);
    }
  }
}

// One token for each sequence: a thread takes kStepSeqs sequences' channels, all their rows
// in flight at once, so that its weights are loaded once for them.
template <typename T, int W, int V, bool VEC, bool SILU>
__global__ void __launch_bounds__(32 * kWarps) conv_step_kernel(const ConvParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Chan<V, VEC> ch(blockIdx.x % p.tiles, lane);
  if (p.status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
  if (ch.c0 >= p.C) return;
  const OutRows<T, V, VEC> out(p, ch);
  const int n0 = (int)(blockIdx.x / p.tiles * kWarps + warp) * kStepSeqs;
  Raw<T, V> rows[kStepSeqs][W];  // the state's rows, then x
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int n = n0 + q;
#pragma unroll
    for (int r = 0; r < W; ++r) rows[q][r] = Raw<T, V>{};
    if (n >= p.N) continue;
#pragma unroll
    for (int r = 0; r < W - 1; ++r)
      if (p.init)  // the final state may be this buffer
        load_row<T, V, VEC, true>(rows[q][r],
                                  static_cast<const T*>(p.init) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0,
                                  ch.step, p.C - ch.c0);
    load_row<T, V, VEC>(rows[q][W - 1], static_cast<const T*>(p.x) + (int64_t)n * p.x_stride + ch.c0,
                        ch.step, p.C - ch.c0);
  }
  pair w[W][V / 2], b[V / 2];
  load_weights<W, V, VEC>(p, ch, w, b);
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) {
    const int n = n0 + q;
    if (n >= p.N) break;
    pair h[W - 1][V / 2], x[V / 2], s[V / 2];
#pragma unroll
    for (int r = 0; r < W - 1; ++r) to_pairs(rows[q][r], h[r]);
    to_pairs(rows[q][W - 1], x);
    pre_activation<W, V>(w, b, h, x, s);
    if constexpr (SILU) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) s[i] = silu<T>(s[i]);
    }
    float y[V];
    from_pairs<V>(s, y);
    out.store(p, ch, n, y);
    if (p.fin) {
#pragma unroll
      for (int r = 0; r < W - 1; ++r) {
        float f[V];
        unpack(rows[q][r + 1], f);
        store_row<T, V, VEC>(static_cast<T*>(p.fin) + ((int64_t)n * (W - 1) + r) * p.C + ch.c0, f,
                             ch.step, p.C - ch.c0);
      }
    }
  }
}

// Backward: a run emits the dx rows of its tokens.  dx[t] needs dp[t .. t + W - 1], so the
// run computes dp for W - 1 tokens more than it emits (never past the sequence's end) and
// emits row t - W + 1 at step t; before a sequence's first token the emitted rows are
// those of dinitial_state.
template <typename T, typename TD, int W, int V, bool VEC, bool SILU>
__global__ void __launch_bounds__(32 * kWarps) conv_bwd_kernel(const ConvParams p) {
  __shared__ RingSlot<T, V> s_x[VEC ? kWarps : 1][VEC ? kRing : 1][32];
  __shared__ RingSlot<TD, V> s_d[VEC ? kWarps : 1][VEC ? kRing : 1][32];
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
  pair w[W][V / 2], b[V / 2], dw[W][V / 2], db[V / 2];
  load_weights<W, V, VEC>(p, ch, w, b);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    db[i] = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0;
  }
  const OutRows<const TD, V, VEC> dout(p, ch);
  const T* const px = static_cast<const T*>(p.x) + ch.c0;
  Ring<T, V> rx(&s_x[VEC ? warp : 0][0][lane]);
  Ring<TD, V> rd(&s_d[VEC ? warp : 0][0][lane]);
  const int64_t run = rblk * kWarps + warp;
  const int64_t t0 = min(run * p.run, p.total), t1 = min(t0 + p.run, p.total);
  int n = 0;
  if (t0 < t1) n = p.cu ? find_sequence(p.cu, p.N, t0) : (int)(t0 / p.T);
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
    pair h[W - 1][V / 2], q[W - 1][V / 2];  // xx and dp of the last W - 1 tokens
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      Raw<T, V> x = {};
      if (mine) load_xx<T, W, V, VEC>(p, ch, n, bos, a - bos - (W - 1) + r, x);
      to_pairs(x, h[r]);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) q[r][i] = 0;
    }
    // dp of token t; `sum`: it belongs to this run, so it counts for the weights
    auto token = [&](const Raw<T, V>& rx, const Raw<TD, V>& rd, bool sum, pair (&d)[V / 2]) {
      pair x[V / 2], s[V / 2];
      to_pairs(rx, x);
      to_pairs(rd, d);
      if constexpr (SILU) {
        pre_activation<W, V>(w, b, h, x, s);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          d[i] = pmul(d[i], silu_slope(s[i], sigmoid<T>(s[i])));
        }
      }
      if (sum) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
#pragma unroll
          for (int r = 0; r < W - 1; ++r) dw[r][i] = pfma(d[i], h[r][i], dw[r][i]);
          dw[W - 1][i] = pfma(d[i], x[i], dw[W - 1][i]);
          db[i] = padd(db[i], d[i]);
        }
      }
      shift<W, V>(h, x);
    };
    // row te = t - W + 1: dxx[te] = sum_s w[W - 1 - s] dp[te + s], s = 0 .. W - 1
    auto row_sum = [&](const pair (&d)[V / 2], pair (&s)[V / 2]) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        s[i] = pmul(w[0][i], d[i]);
#pragma unroll
        for (int r = 0; r < W - 1; ++r) s[i] = pfma(w[W - 1 - r][i], q[r][i], s[i]);
      }
      shift<W, V>(q, d);
    };
    auto emit = [&](int64_t t, const pair (&d)[V / 2]) {  // at the ends of the piece
      const int64_t te = t - (W - 1);
      pair s[V / 2];
      row_sum(d, s);
      if (!mine || !(te >= a || (a == bos && p.dinit))) return;
      if (p.dfin && te >= eos - (W - 1)) {
        Raw<T, V> raw;
        pair f[V / 2];
        load_row<T, V, VEC>(raw,
                            static_cast<const T*>(p.dfin) +
                                ((int64_t)n * (W - 1) + te - eos + W - 1) * p.C + ch.c0,
                            ch.step, p.C - ch.c0);
        to_pairs(raw, f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) s[i] = padd(s[i], f[i]);
      }
      float dx[V];
      from_pairs<V>(s, dx);
      if (te >= a)
        store_row<T, V, VEC>(static_cast<T*>(p.dx) + te * p.C + ch.c0, dx, ch.step, p.C - ch.c0);
      else
        store_row<float, V, VEC>(p.dinit + ((int64_t)n * (W - 1) + te - bos + W - 1) * p.C + ch.c0,
                                 dx, ch.step, p.C - ch.c0);
    };
    const int64_t last = min(end + W - 1, eos);  // tokens that are loaded
    pair d[V / 2];
    auto plain = [&](const Raw<T, V>& x, const Raw<TD, V>& g, T* row) {
      pair s[V / 2];
      float dx[V];
      token(x, g, true, d);
      row_sum(d, s);
      from_pairs<V>(s, dx);
      if (mine) store_row<T, V, VEC>(row, dx, ch.step, p.C - ch.c0);
    };
    T* const pdx = static_cast<T*>(p.dx) + ch.c0 - (int64_t)(W - 1) * p.C;
    if constexpr (VEC) {
      const int rows = (int)(last - a), own = (int)(end - a);
      const T* xnext = px + a * p.x_stride;  // the rows to ask for next
      const TD* dnext = dout.base + a * dout.width;
      auto issue = [&](int i, int slot) {
        rx.copy(slot, xnext, mine && i < rows);
        rd.issue(slot, dnext, mine && i < rows);
        xnext += p.x_stride, dnext += dout.width;
      };
#pragma unroll
      for (int i = 0; i < kRing - 1; ++i) issue(i, i);
      Raw<T, V> x;
      Raw<TD, V> g;
      auto arrive = [&](int i, int slot) {
        issue(i + kRing - 1, slot + kRing - 1);
        ptx::cp_async_wait<kRing - 1>();
        rx.read(slot, x);
        rd.read(slot, g);
      };
      int i = 0;
#pragma unroll
      for (int u = 0; u < W - 1; ++u) {  // rows before the piece
        if (u >= rows) break;
        arrive(u, u);
        token(x, g, u < own, d);
        emit(a + u, d);
        ++i;
      }
      T* row = pdx + (a + i) * p.C;
      for (; i + kRing <= own; i += kRing) {
#pragma unroll
        for (int u = 0; u < kRing; ++u) {
          arrive(i + u, W - 1 + u);
          plain(x, g, row);
          row += p.C;
        }
      }
      for (; i < own; ++i) {
        arrive(i, i);
        plain(x, g, row);
        row += p.C;
      }
      for (; i < rows; ++i) {  // tokens of the next run
        arrive(i, i);
        token(x, g, false, d);
        emit(a + i, d);
      }
      ptx::cp_async_wait_all();
    } else {
      for (int64_t t = a; t < last; t += kBatch) {
        Raw<T, V> x[kBatch] = {};
        Raw<TD, V> g[kBatch] = {};
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (!mine || t + u >= last) continue;
          load_row<T, V, VEC>(x[u], px + (t + u) * p.x_stride, ch.step, p.C - ch.c0);
          dout.load(p, ch, t + u, g[u]);
        }
        if (t >= a + W - 1 && t + kBatch <= end) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) plain(x[u], g[u], pdx + (t + u) * p.C);
        } else {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            if (t + u >= last) break;
            token(x[u], g[u], t + u < end, d);
            emit(t + u, d);
          }
        }
      }
    }
    const pair none[V / 2] = {};
    for (int64_t t = last; t < end + W - 1; ++t) emit(t, none);  // past the sequence
    a = end;
  }
  const float zero[V] = {};
  for (; a < t1 && mine; ++a)  // rows of no sequence
    store_row<T, V, VEC>(static_cast<T*>(p.dx) + a * p.C + ch.c0, zero, ch.step, p.C - ch.c0);
  // the block's warps added in their order, then one partial row per block
  __shared__ float acc[W + 1][32 * V + 1];
  for (int k = 0; k < kWarps; ++k) {
    if (warp == k) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * 32 + lane;
        auto half = [&](pair v) { return i & 1 ? un(v).y : un(v).x; };
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j][c] = (k ? acc[j][c] : 0.f) + half(dw[j][i / 2]);
        acc[W][c] = (k ? acc[W][c] : 0.f) + half(db[i / 2]);
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

enum ConvPass { kFwd, kStep, kBwd };

template <int PASS, typename T, typename TD, int W, int V, bool VEC, bool SILU>
void (*conv_kernel_w())(ConvParams) {
  if constexpr (PASS == kFwd) return conv_fwd_kernel<T, W, V, VEC, SILU>;
  else if constexpr (PASS == kStep) return conv_step_kernel<T, W, V, VEC, SILU>;
  else return conv_bwd_kernel<T, TD, W, V, VEC, SILU>;
}
template <int PASS, typename T, typename TD, int V, bool VEC, bool SILU>
void (*conv_kernel_s(int width))(ConvParams) {
  return width == 2   ? conv_kernel_w<PASS, T, TD, 2, V, VEC, SILU>()
         : width == 3 ? conv_kernel_w<PASS, T, TD, 3, V, VEC, SILU>()
                      : conv_kernel_w<PASS, T, TD, 4, V, VEC, SILU>();
}
template <int PASS, typename T, typename TD, int V, bool VEC>
void (*conv_kernel_v(int width, int fn))(ConvParams) {
  return fn == KDA_FN_SILU ? conv_kernel_s<PASS, T, TD, V, VEC, true>(width)
                           : conv_kernel_s<PASS, T, TD, V, VEC, false>(width);
}

// Channels per thread.  Forward: 16 bytes (one token: 8, for twice the threads: 10.3 us
// against 13.3 for 256 sequences of 12,288 channels); backward: 4, whose weights, their gradients
// and two histories take 164 registers, 12 warps per SM.
constexpr int kFwdV16 = 8, kFwdV32 = 4, kStepV = 4, kBwdV = 4;

template <int PASS>
void (*conv_kernel(bool f32, bool dout_f32, bool vec, int width, int fn))(ConvParams) {
  constexpr int V16 = PASS == kBwd ? kBwdV : PASS == kStep ? kStepV : kFwdV16;
  constexpr int V32 = PASS == kBwd ? kBwdV : kFwdV32;
  if (f32) return vec ? conv_kernel_v<PASS, float, float, V32, true>(width, fn)
                      : conv_kernel_v<PASS, float, float, V32, false>(width, fn);
  if constexpr (PASS == kBwd) {
    if (dout_f32) return vec ? conv_kernel_v<PASS, bf16, float, V16, true>(width, fn)
                             : conv_kernel_v<PASS, bf16, float, V16, false>(width, fn);
  }
  return vec ? conv_kernel_v<PASS, bf16, bf16, V16, true>(width, fn)
             : conv_kernel_v<PASS, bf16, bf16, V16, false>(width, fn);
}

// Tokens per run.  A run loads W - 1 rows more than its own (the backward 2 (W - 1)) and
// looks its sequence up, so long runs are cheaper where there are values enough to fill the
// GPU with them; short ones take less from their first token to their last.  Measured with
// 8 to 256 tokens over 1,024, 4,096 and 12,288 bf16 channels, the best one follows the
// number of values: forward, 0.5 million 4.7 us with 8 (32: 8.1), 8 million 10.4 with 32
// (8: 13.4), 402 million 250 with 64 (32: 267); backward, 2 million 11.0 with 16 (8: 14.4),
// 8 million 20.6 with 64 (32: 23.4), 402 million 446 with 256 (128: 464, 32: 643).
int64_t run_of(int64_t total, int32_t C, bool bwd) {
  const int64_t values = total * C, million = 1000000;
  if (!bwd) return values < 3 * million ? 8 : values < 8 * million ? 16 : values < 20 * million ? 32 : 64;
  return values < 3 * million / 2 ? 8 : values < 4 * million ? 16 : values < 7 * million ? 32
         : values < 12 * million ? 64 : values < 300 * million ? 128 : 256;
}
int64_t row_blocks(int64_t total, int32_t C, bool bwd) {
  const int64_t per = run_of(total, C, bwd) * kWarps;
  return (total + per - 1) / per;
}

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
          const int64_t* cu, int64_t B, int64_t T, int32_t C, int32_t N) {
  p.x = x, p.x_stride = x_stride, p.weight = weight, p.bias = bias, p.init = init, p.cu = cu;
  p.num_outs = num_outs;
  p.out_lo[0] = 0;
  for (int i = 0; i < KDA_CONV_MAX_OUTS; ++i) {
    p.outs[i] = i < num_outs ? const_cast<void*>(outs[i]) : nullptr;
    p.out_lo[i + 1] = p.out_lo[i] + (i < num_outs ? out_channels[i] : 0);
  }
  p.T = T, p.total = B * T, p.N = N, p.C = C;
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
  const bool f32 = dtype == KDA_ROW_FP32;
  const bool step = !cu_seqlens && T == 1;
  const int V = f32 ? kFwdV32 : step ? kStepV : kFwdV16;
  const bool vec = conv_vec(x, x_stride, outs, out_channels, num_outs, initial_state, final_state,
                            C, V, f32 ? 4 : 2, f32 ? 4 : 2);
  ConvParams p = {};
  fill(p, x, x_stride, weight, bias, outs, out_channels, num_outs, initial_state, cu_seqlens, B, T,
       C, N);
  p.fin = final_state;
  p.status = static_cast<unsigned*>(workspace);
  const int64_t tiles = (C + 32 * V - 1) / (32 * V);
  // A short batched sequence is one run of its own, which also writes its final state.
  p.whole = !cu_seqlens && T <= 32 && T > 0;
  if (p.whole) {
    p.run = (int32_t)T;
    p.runs = N;
  } else {
    p.run = (int32_t)run_of(p.total, C, false);
    p.runs = (p.total + p.run - 1) / p.run;
  }
  const int64_t per_block = kWarps * (step ? kStepSeqs : 1);
  const int64_t run_blocks = (p.runs + per_block - 1) / per_block;
  const bool split_state = final_state && !p.whole;
  const bool same = final_state && final_state == initial_state;
  const int64_t state_blocks = split_state ? ((int64_t)N + kWarps - 1) / kWarps : 0;
  if ((run_blocks + state_blocks) * tiles >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
  auto kernel = step ? conv_kernel<kStep>(f32, f32, vec, width, fn)
                     : conv_kernel<kFwd>(f32, f32, vec, width, fn);
  p.weight_vec = al_to(weight, 16);
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
           (size_t)kda::row_blocks(total_tokens, C, true) * (width + 1) * (size_t)C * sizeof(float);
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
  const int V = kBwdV;
  const bool vec = conv_vec(x, x_stride, douts, out_channels, num_outs, initial_state,
                            dfinal_state, C, V, f32 ? 4 : 2, dout_dtype == KDA_ROW_FP32 ? 4 : 2) &&
                   al_to(dx, 16) && al_to(dinitial_state, 16);
  ConvParams p = {};
  fill(p, x, x_stride, weight, bias, douts, out_channels, num_outs, initial_state, cu_seqlens, B,
       T, C, N);
  p.dfin = dfinal_state, p.dx = dx, p.dinit = dinitial_state;
  p.status = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
  p.run = (int32_t)run_of(p.total, C, true);
  p.weight_vec = al_to(weight, 16);
  const int64_t tiles = (C + 32 * V - 1) / (32 * V);
  const int64_t blocks = row_blocks(p.total, C, true);
  // empty sequences can only come with cu_seqlens or T = 0
  const int64_t state_blocks =
      dinitial_state && (cu_seqlens || T == 0) ? ((int64_t)N + kWarps - 1) / kWarps : 0;
  if ((blocks + state_blocks) * tiles >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
  p.tiles = (int32_t)tiles;
  p.run_blocks = blocks;
  if (blocks + state_blocks > 0) {
    conv_kernel<kBwd>(f32, dout_dtype == KDA_ROW_FP32, vec, width, fn)<<<(unsigned)((blocks + state_blocks) * tiles), 32 * kWarps,
                                         0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  } else if (cudaMemsetAsync(p.status, 0, 4, stream) != cudaSuccess) {
    return KDA_ERR_CUDA;
  }
  if (launch_column_sums(p.part, blocks, (int64_t)(width + 1) * C, (int64_t)(width + 1) * C,
                         (int64_t)width * C, C,
                         dweight, dbias, nullptr, stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"
