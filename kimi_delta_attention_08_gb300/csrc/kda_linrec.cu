// kda_linrec.cu -- the gated linear recurrence, forward and backward.
//
// Per channel, with R = sigmoid(r + r_bias), I = sigmoid(i + i_bias), L = exp(A_log) R:
//   a = exp(-L),  m = sqrt(1 - a^2),  h_t = a h_{t-1} + m I x,  out = h silu(z)
// and backwards, with g_t the gradient of h_t and c_t = a_t g_t what it hands to t - 1:
//   g_t = dout silu(z) + c_{t+1},    dz = dout h silu'(z),
//   dx = g m I,   di = g m x I (1 - I),
//   e = g L (a^2 / m I x - a h_{t-1}),  dr = e (1 - R),  dA_log = sum of e.
// L / m, not 1 / m, is what e needs: it goes to zero with L where 1 / m has no bound.
//
// Bound by HBM: each row is read once and written once.  A block takes a tile of rows by
// channels; its warps take consecutive runs of rows, a lane one or two channels.  A run is
// scanned in registers from zero (h) along with the product of its decays (P), runs are
// joined in shared memory, tiles through the workspace: h_t = h + P_t X with X the state
// before the tile.  So a prompt of any length fills the GPU in one pass over its rows.
//
// X.  Each tile publishes what it does to a state, (product, end), as soon as it has it.
// Every kGroup tiles one also publishes its end state itself.  A tile composes what the
// tiles since then published, in their order, and that state: the same sums in every run.
// A tile that holds the sequence's first row ends the look back.  Tiles are handed out by
// an atomic counter in the order of their rows, so a tile only waits for tiles that
// already run, and what is published is its own flag: words that were filled with ones
// before (no arithmetic result has these bits).  Waits give up after half a second.
#include <cstring>

#include "kda_internal.h"
#include "kda_rows.cuh"
#include "kda_scan.cuh"
#include "../../include/kda_layer.h"

namespace kda {
namespace {

using namespace rows;

constexpr int kWarps = 8;
constexpr int kRowsF = 16, kRowsB = 8;            // rows per warp: forward, backward
constexpr int kTileF = kWarps * kRowsF, kTileB = kWarps * kRowsB;
constexpr int kGroup = 16;                        // tiles between two published end states
constexpr int kStepTokens = 8;                    // prompts up to this length: the step kernel
constexpr uint64_t kWaitNs = 500000000ull;
constexpr uint64_t kUnset = ~0ull;
static_assert(kTileF % KDA_LINREC_CHUNK == 0 && kTileB == KDA_LINREC_CHUNK, "saved states");
static_assert(kGroup == 2 * kWarps, "each warp looks at two tiles");

struct LinrecParams {
  const void *x, *r, *i, *z, *dout;
  int64_t x_s, r_s, i_s, z_s;
  const float *A_log, *r_bias, *i_bias;
  const void *init, *dfin;
  int32_t state_bf16, stall;
  const int64_t* cu;
  int64_t T, total;
  int32_t N, dim, blocks;    // blocks: of channels
  int64_t tiles;             // of rows
  void *out, *fin;
  float* states;             // [total / KDA_LINREC_CHUNK + 1][dim]
  unsigned *status, *ticket;
  uint64_t* agg;             // [tiles][dim]: (product, end) of each tile
  unsigned* ends;            // [tiles / kGroup][dim]: end states
  void *dx, *dr, *di, *dz;
  float *part, *dinit;       // part: [tiles][3][dim]
};

__device__ __forceinline__ uint64_t ld_word(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ unsigned ld_word(const unsigned* p) {
  unsigned v;
  asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_word(uint64_t* p, uint64_t v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void st_word(unsigned* p, unsigned v) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// The word at p once it is set; after the limit (or another wait's) zero, with the status.
template <typename W>
__device__ __forceinline__ W await_word(const W* p, unsigned* status) {
  W v = ld_word(p);
  if (v != static_cast<W>(kUnset)) return v;
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      v = ld_word(p);
      if (v != static_cast<W>(kUnset)) return v;
    }
    if (ptx::global_timer_ns() - t0 > kWaitNs || (ld_word(status) & kDevStatusTimeout)) {
      atomicOr(status, kDevStatusTimeout);
      return 0;
    }
  }
}

// Bits that are published: those of all ones mean "not set", so that NaN becomes another.
__device__ __forceinline__ unsigned published(float v) {
  const unsigned b = __float_as_uint(v);
  return b == ~0u ? 0x7FFFFFFFu : b;
}

// The sequence of row t and its bounds; false where t belongs to none.
__device__ __forceinline__ bool row_sequence(const LinrecParams& p, int64_t t, int& n, int64_t& bos,
                                             int64_t& eos) {
  if (t >= p.total) return false;
  if (!p.cu) {
    n = (int)((uint32_t)t / (uint32_t)p.T);
    bos = (int64_t)n * p.T, eos = bos + p.T;
    return true;
  }
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  n = lo, bos = __ldg(p.cu + lo), eos = __ldg(p.cu + lo + 1);
  return bos >= 0 && bos <= t && t < eos && eos <= p.total;
}

template <int V>
__device__ __forceinline__ void load_state(float (&h)[V], const void* p, int64_t at, bool b16) {
#pragma unroll
  for (int k = 0; k < V; ++k)
    h[k] = b16 ? __bfloat162float(static_cast<const bf16*>(p)[at + k]) : static_cast<const float*>(p)[at + k];
}
template <int V>
__device__ __forceinline__ void store_state(void* p, int64_t at, const float (&h)[V], bool b16) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (b16) static_cast<bf16*>(p)[at + k] = __float2bfloat16_rn(h[k]);
    else static_cast<float*>(p)[at + k] = h[k];
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_vals(Raw<T, V>& r, const void* p, int64_t at) {
  if constexpr (V == 1) r.w[0] = __float_as_uint(to_f(__ldg(static_cast<const T*>(p) + at)));
  else load_words(r.w, static_cast<const T*>(p) + at);
}
template <typename T, int V>
__device__ __forceinline__ void vals_of(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (V == 1) f[0] = __uint_as_float(r.w[0]);
  else unpack(r, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vals(void* p, int64_t at, const float (&f)[V]) {
  store_row<T, V, (V > 1)>(static_cast<T*>(p) + at, f, 1, 1);
}

// The channel's rate (base 2, negative) and biases.
template <int V>
struct Channel {
  float A2[V], rb[V], ib[V];
};
template <int V>
__device__ __forceinline__ void load_channel(Channel<V>& c, const LinrecParams& p, int ch, bool ok) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    c.A2[k] = ok ? scan::rate_of(__ldg(p.A_log + ch + k)) : 0.f;
    c.rb[k] = ok && p.r_bias ? __ldg(p.r_bias + ch + k) : 0.f;
    c.ib[k] = ok && p.i_bias ? __ldg(p.i_bias + ch + k) : 0.f;
  }
}

// a = 2^L2 and m^2 = 1 - a^2 from L2 = -L log2 e <= 0.  The exponent is raised by the
// hardware exponential's mean error (see the scan's decay).  Small steps, u = 2 L up to 1/2,
// take 1 - exp(-u) = u P(u), P of degree 5 with P(0) = 1 fitted by reweighted least squares
// to an even relative error (1.5e-9; 1e-7 as evaluated in fp32); 1 - a^2 would have none
// of its digits right for them.  From there on 1 - a^2 is good to 4e-7.
__device__ __forceinline__ float decay_of(float L2, float& m2) {
  const float a = ptx::ex2_approx(L2 + 2.5e-8f);
  const float u = L2 * (-2.f * kLn2);
  float s = fmaf(-0.00112592906f, u, 0.00819330197f);
  s = fmaf(s, u, -0.0416320525f);
  s = fmaf(s, u, 0.166662887f);
  s = fmaf(s, u, -0.499999851f);
  s = fmaf(s, u, 1.0f);
  m2 = u > 0.5f ? fmaf(-a, a, 1.0f) : u * s;
  return a;
}
// Finite at zero; scaled, since the hardware takes what is below 2^-126 for zero.
__device__ __forceinline__ float rsqrt_of(float m2) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(m2 * 0x1p64f, 1e-37f)));
  return r * 0x1p32f;
}

// a and b = m I x of one value.
template <typename T>
__device__ __forceinline__ void step_of(float x, float r, float i, float A2, float& a, float& b) {
  float m2;
  a = decay_of(A2 * sigmoid<T>(r), m2);
  b = m2 * rsqrt_of(m2) * sigmoid<T>(i) * x;
}

// What a warp knows about its rows: bit j for row j.
struct RowBits {
  unsigned start, last, live;
};

// Rows of the tile: every row's sequence (shared), and for the look back the first row's
// sequence start and the last row's end.
struct TileRows {
  int n[kTileF];
  unsigned char flags[kTileF];   // 1: first row of its sequence, 2: last, 4: of a sequence
  int64_t bos, eos;
};
template <int TILE>
__device__ __forceinline__ void find_rows(TileRows& s, const LinrecParams& p, int64_t row0) {
  if (threadIdx.x < TILE) {
    const int64_t t = row0 + threadIdx.x;
    int n = 0;
    int64_t bos = 0, eos = 0;
    const bool live = row_sequence(p, t, n, bos, eos);
    s.n[threadIdx.x] = n;
    s.flags[threadIdx.x] = live ? 4 | (t == bos ? 1 : 0) | (t + 1 == eos ? 2 : 0) : 0;
    if (threadIdx.x == 0) s.bos = bos;
    if (threadIdx.x == TILE - 1) s.eos = eos;
  }
}
template <int R>
__device__ __forceinline__ RowBits warp_rows(const TileRows& s, int warp, int lane) {
  const unsigned f = lane < R ? s.flags[warp * R + lane] : 0u;
  RowBits b;
  b.start = __ballot_sync(0xffffffffu, f & 1);
  b.last = __ballot_sync(0xffffffffu, f & 2);
  b.live = __ballot_sync(0xffffffffu, f & 4);
  return b;
}

// An affine step (product, end) of a lane's channels, joined along the rows.
template <int V>
struct Affine {
  float P[V], H[V];
};
template <int V>
__device__ __forceinline__ void unit_of(Affine<V>& e) {
#pragma unroll
  for (int k = 0; k < V; ++k) e.P[k] = 1.f, e.H[k] = 0.f;
}
// e <- e, then f; `cut`: f does not depend on what was before it.
template <int V>
__device__ __forceinline__ void then(Affine<V>& e, const Affine<V>& f, bool cut) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    e.H[k] = cut ? f.H[k] : fmaf(f.P[k], e.H[k], f.H[k]);
    e.P[k] = cut ? f.P[k] : e.P[k] * f.P[k];
  }
}

template <int V>
struct JoinShared {
  Affine<V> run[kWarps][32];   // of the warps' runs
  Affine<V> back[kWarps][32];  // of the tiles looked back at
  int cut[kWarps];
  unsigned next;
};

// What the tile does to a state, published by the warp that holds its last run.
template <int V>
__device__ __forceinline__ void publish(const LinrecParams& p, int64_t slot, int ch, const Affine<V>& e) {
#pragma unroll
  for (int k = 0; k < V; ++k)
    st_word(p.agg + slot * p.dim + ch + k,
            (uint64_t)published(e.P[k]) | ((uint64_t)published(e.H[k]) << 32));
}

// The warp's part of the look back from slot `s`: tiles first + 2 warp and the next one, of
// first .. s - 1; `edge`: the slot whose tile starts the sequence (its step is cut off from
// what was before), or below `first`.
template <int V>
__device__ __forceinline__ void look_back(const LinrecParams& p, int64_t s, int64_t first, int64_t edge,
                                          int warp, int ch, bool ok, Affine<V>& e) {
  unit_of(e);
  const int64_t at = first + 2 * warp;
  uint64_t w[2][V];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int k = 0; k < V; ++k)
      w[q][k] = ok && at + q < s ? ld_word(p.agg + (at + q) * p.dim + ch + k) : 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (at + q >= s) break;
    Affine<V> f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (w[q][k] == kUnset) w[q][k] = await_word(p.agg + (at + q) * p.dim + ch + k, p.status);
      f.P[k] = __uint_as_float((unsigned)w[q][k]);
      f.H[k] = __uint_as_float((unsigned)(w[q][k] >> 32));
    }
    then(e, f, at + q == edge);
  }
}

// The state before the tile in slot s of the walking order (X), once the warps' parts are
// in shared memory.
template <int V>
__device__ __forceinline__ void carried(float (&X)[V], const LinrecParams& p, const JoinShared<V>& sh,
                                        int64_t s, int64_t first, int64_t edge, int lane, int ch, bool ok) {
  const bool from_end = edge < first;
#pragma unroll
  for (int k = 0; k < V; ++k)
    X[k] = from_end && ok
               ? __uint_as_float(await_word(p.ends + (first / kGroup - 1) * p.dim + ch + k, p.status))
               : 0.f;
  const int parts = (int)((s - first + 1) / 2);
  for (int w = 0; w < parts; ++w) {
    const Affine<V> f = sh.back[w][lane];
    const bool cut = edge >= first + 2 * w && edge < first + 2 * w + 2;
#pragma unroll
    for (int k = 0; k < V; ++k) X[k] = cut ? f.H[k] : fmaf(f.P[k], X[k], f.H[k]);
  }
}

// ---------------------------------------------------------------- forward --
template <typename T, int V, bool OUT>
__global__ void __launch_bounds__(32 * kWarps, 2) linrec_fwd_kernel(LinrecParams p) {
  constexpr int R = kRowsF;
  __shared__ TileRows rows_s;
  __shared__ JoinShared<V> sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t units = p.tiles * p.blocks;
  if (threadIdx.x == 0) sh.next = atomicAdd(p.ticket, 1u);
  __syncthreads();
  int64_t unit = sh.next;
  while (unit < units) {
    const int64_t s = unit / p.blocks;
    const int ch = (int)(unit % p.blocks) * 32 * V + lane * V;
    const bool ok = ch < p.dim;
    const int64_t row0 = s * kTileF + warp * R;
    unsigned next = 0;
    if (threadIdx.x == 0) next = atomicAdd(p.ticket, 1u);
    Raw<T, V> rx[R], rr[R], ri[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool in = ok && row0 + j < p.total;
      rx[j] = {}, rr[j] = {}, ri[j] = {};
      if (in) {
        load_vals<T, V>(rx[j], p.x, (row0 + j) * p.x_s + ch);
        load_vals<T, V>(rr[j], p.r, (row0 + j) * p.r_s + ch);
        load_vals<T, V>(ri[j], p.i, (row0 + j) * p.i_s + ch);
      }
    }
    Channel<V> c;
    load_channel(c, p, ch, ok);
    find_rows<kTileF>(rows_s, p, s * kTileF);
    __syncthreads();
    const RowBits bits = warp_rows<R>(rows_s, warp, lane);
    float a[R][V], b[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float x[V], r[V], i[V];
      vals_of(rx[j], x), vals_of(rr[j], r), vals_of(ri[j], i);
#pragma unroll
      for (int k = 0; k < V; ++k) step_of<T>(x[k], r[k] + c.rb[k], i[k] + c.ib[k], c.A2[k], a[j][k], b[j][k]);
    }
    if (bits.start && p.init) {
      float h0[R][V];
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (ok && (bits.start >> j & 1))
          load_state<V>(h0[j], p.init, (int64_t)rows_s.n[warp * R + j] * p.dim + ch, p.state_bf16);
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (ok && (bits.start >> j & 1)) {
#pragma unroll
          for (int k = 0; k < V; ++k) b[j][k] = fmaf(a[j][k], h0[j][k], b[j][k]);
        }
    }
    // the run from zero: a <- the product of decays, b <- h
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool cut = bits.start >> j & 1;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (j == 0) {
          a[0][k] = cut ? 0.f : a[0][k];
        } else {
          b[j][k] = cut ? b[j][k] : fmaf(a[j][k], b[j - 1][k], b[j][k]);
          a[j][k] = cut ? 0.f : a[j][k] * a[j - 1][k];
        }
      }
    }
    Affine<V> own;
#pragma unroll
    for (int k = 0; k < V; ++k) own.P[k] = a[R - 1][k], own.H[k] = b[R - 1][k];
    sh.run[warp][lane] = own;
    if (lane == 0) sh.cut[warp] = bits.start != 0;
    __syncthreads();
    Affine<V> ex;
    unit_of(ex);
    bool cut_before = false;
    for (int w = 0; w < warp; ++w) {
      then(ex, sh.run[w][lane], sh.cut[w]);
      cut_before |= sh.cut[w] != 0;
    }
    if (warp == kWarps - 1 && ok && !(p.stall && s == 0)) {
      Affine<V> all = ex;
      then(all, own, bits.start != 0);
      publish(p, s, ch, all);
    }
    // the state before the tile
    float X[V] = {};
    const unsigned char f0 = rows_s.flags[0];
    if ((f0 & 4) && !(f0 & 1) && s > 0) {
      const int64_t group = s / kGroup * kGroup, edge = rows_s.bos / kTileF;
      const int64_t first = edge > group ? edge : group;
      look_back(p, s, first, edge, warp, ch, ok, sh.back[warp][lane]);
      __syncthreads();
      carried(X, p, sh, s, first, edge, lane, ch, ok);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) X[k] = cut_before ? ex.H[k] : fmaf(ex.P[k], X[k], ex.H[k]);
    if (p.states && ok && row0 % KDA_LINREC_CHUNK == 0 && row0 < p.total) {
#pragma unroll
      for (int k = 0; k < V; ++k) p.states[row0 / KDA_LINREC_CHUNK * p.dim + ch + k] = X[k];
    }
    const int open = bits.start ? __ffs(bits.start) - 1 : R;  // rows that X reaches
    if (warp == kWarps - 1 && ok && s % kGroup == kGroup - 1) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        st_word(p.ends + s / kGroup * p.dim + ch + k,
                published(open < R ? own.H[k] : fmaf(own.P[k], X[k], own.H[k])));
    }
    if constexpr (OUT) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!ok || !(bits.live >> j & 1)) continue;
        float h[V], y[V];
#pragma unroll
        for (int k = 0; k < V; ++k) y[k] = h[k] = j < open ? fmaf(a[j][k], X[k], b[j][k]) : b[j][k];
        if (p.z) {
          Raw<T, V> rz;
          float z[V];
          load_vals<T, V>(rz, p.z, (row0 + j) * p.z_s + ch);
          vals_of(rz, z);
#pragma unroll
          for (int k = 0; k < V; ++k) y[k] = h[k] * z[k] * sigmoid<T>(z[k]);
        }
        store_vals<T, V>(p.out, (row0 + j) * p.dim + ch, y);
        if (p.fin && (bits.last >> j & 1))
          store_state<V>(p.fin, (int64_t)rows_s.n[warp * R + j] * p.dim + ch, h, p.state_bf16);
      }
    }
    if (threadIdx.x == 0) sh.next = next;
    __syncthreads();
    unit = sh.next;
  }
}

// Single tokens and prompts of a few: a thread takes the channels of one sequence.
template <typename T, int V>
__global__ void __launch_bounds__(256) linrec_step_kernel(LinrecParams p) {
  const int per = (p.dim + V - 1) / V;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = at / per;
  const int ch = (int)(at % per) * V;
  if (n >= p.N) return;
  float h[V] = {};
  if (p.init) load_state<V>(h, p.init, n * p.dim + ch, p.state_bf16);
  Channel<V> c;
  load_channel(c, p, ch, true);
  for (int64_t t = n * p.T; t < (n + 1) * p.T; ++t) {
    Raw<T, V> rx, rr, ri, rz = {};
    load_vals<T, V>(rx, p.x, t * p.x_s + ch);
    load_vals<T, V>(rr, p.r, t * p.r_s + ch);
    load_vals<T, V>(ri, p.i, t * p.i_s + ch);
    if (p.z) load_vals<T, V>(rz, p.z, t * p.z_s + ch);
    float x[V], r[V], i[V], z[V], y[V];
    vals_of(rx, x), vals_of(rr, r), vals_of(ri, i), vals_of(rz, z);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float a, b;
      step_of<T>(x[k], r[k] + c.rb[k], i[k] + c.ib[k], c.A2[k], a, b);
      h[k] = fmaf(a, h[k], b);
      y[k] = p.z ? h[k] * z[k] * sigmoid<T>(z[k]) : h[k];
    }
    store_vals<T, V>(p.out, t * p.dim + ch, y);
  }
  if (p.fin) store_state<V>(p.fin, n * p.dim + ch, h, p.state_bf16);
}

// --------------------------------------------------------------- backward --
template <typename T, int V>
__global__ void __launch_bounds__(32 * kWarps, 2) linrec_bwd_kernel(LinrecParams p) {
  constexpr int R = kRowsB;
  __shared__ TileRows rows_s;
  __shared__ JoinShared<V> sh;           // of the gradients, last run first
  __shared__ Affine<V> fwd[kWarps][32];  // of the states
  __shared__ int fwd_cut[kWarps];
  __shared__ float sums[3][kWarps][32 * V];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t units = p.tiles * p.blocks;
  if (threadIdx.x == 0) sh.next = atomicAdd(p.ticket, 1u);
  __syncthreads();
  int64_t unit = sh.next;
  while (unit < units) {
    const int64_t s = unit / p.blocks;            // counted from the last tile back
    const int64_t tile = p.tiles - 1 - s;
    const int cb = (int)(unit % p.blocks) * 32 * V;
    const int ch = cb + lane * V;
    const bool ok = ch < p.dim;
    const int64_t row0 = tile * kTileB + warp * R;
    unsigned next = 0;
    if (threadIdx.x == 0) next = atomicAdd(p.ticket, 1u);
    Raw<T, V> rx[R], rr[R], ri[R], rd[R], rz[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool in = ok && row0 + j < p.total;
      rx[j] = {}, rr[j] = {}, ri[j] = {}, rd[j] = {}, rz[j] = {};
      if (in) {
        load_vals<T, V>(rx[j], p.x, (row0 + j) * p.x_s + ch);
        load_vals<T, V>(rr[j], p.r, (row0 + j) * p.r_s + ch);
        load_vals<T, V>(ri[j], p.i, (row0 + j) * p.i_s + ch);
        load_vals<T, V>(rd[j], p.dout, (row0 + j) * p.dim + ch);
        if (p.z) load_vals<T, V>(rz[j], p.z, (row0 + j) * p.z_s + ch);
      }
    }
    Channel<V> c;
    load_channel(c, p, ch, ok);
    float X[V] = {};
    if (ok) {
#pragma unroll
      for (int k = 0; k < V; ++k) X[k] = __ldg(p.states + tile * p.dim + ch + k);
    }
    find_rows<kTileB>(rows_s, p, tile * kTileB);
    __syncthreads();
    const RowBits bits = warp_rows<R>(rows_s, warp, lane);
    if (bits.live != (1u << R) - 1) {  // rows of no sequence count for nothing
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (!(bits.live >> j & 1)) rx[j] = {}, rr[j] = {}, ri[j] = {}, rd[j] = {}, rz[j] = {};
    }
    // what the run does to a state, and backwards to a gradient
    float a[R][V], b[R][V], dy[R][V];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      float x[V], r[V], i[V], z[V];
      vals_of(rx[j], x), vals_of(rr[j], r), vals_of(ri[j], i), vals_of(rd[j], dy[j]), vals_of(rz[j], z);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        step_of<T>(x[k], r[k] + c.rb[k], i[k] + c.ib[k], c.A2[k], a[j][k], b[j][k]);
        if (p.z) dy[j][k] *= z[k] * sigmoid<T>(z[k]);
      }
    }
    auto initial = [&](int j, float (&h0)[V]) {
#pragma unroll
      for (int k = 0; k < V; ++k) h0[k] = 0.f;
      if (p.init && ok) load_state<V>(h0, p.init, (int64_t)rows_s.n[warp * R + j] * p.dim + ch, p.state_bf16);
    };
    Affine<V> own;
    unit_of(own);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (bits.start >> j & 1) {
        initial(j, own.H);
#pragma unroll
        for (int k = 0; k < V; ++k) own.P[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) own.H[k] = fmaf(a[j][k], own.H[k], b[j][k]), own.P[k] *= a[j][k];
    }
    fwd[warp][lane] = own;
    if (bits.last && p.dfin && ok) {  // the final state's gradient joins the last row's
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (bits.last >> j & 1) {
          float d[V];
          load_state<V>(d, p.dfin, (int64_t)rows_s.n[warp * R + j] * p.dim + ch, p.state_bf16);
#pragma unroll
          for (int k = 0; k < V; ++k) dy[j][k] += d[k];
        }
    }
    unit_of(own);
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const bool cut = bits.last >> j & 1;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        own.H[k] = a[j][k] * (cut ? dy[j][k] : dy[j][k] + own.H[k]);
        own.P[k] = cut ? 0.f : a[j][k] * own.P[k];
      }
    }
    sh.run[warp][lane] = own;
    if (lane == 0) sh.cut[warp] = bits.last != 0, fwd_cut[warp] = bits.start != 0;
    __syncthreads();
    Affine<V> ex;
    unit_of(ex);
    bool cut_before = false;
    for (int w = kWarps - 1; w > warp; --w) {
      then(ex, sh.run[w][lane], sh.cut[w]);
      cut_before |= sh.cut[w] != 0;
    }
    if (warp == 0 && ok && !(p.stall && s == 0)) {
      Affine<V> all = ex;
      then(all, own, bits.last != 0);
      publish(p, s, ch, all);
    }
    for (int w = 0; w < warp; ++w) {
      const Affine<V> f = fwd[w][lane];
#pragma unroll
      for (int k = 0; k < V; ++k) X[k] = fwd_cut[w] ? f.H[k] : fmaf(f.P[k], X[k], f.H[k]);
    }
    // the gradient that the rows after the tile hand on
    float C[V] = {};
    const unsigned char fl = rows_s.flags[kTileB - 1];
    if ((fl & 4) && !(fl & 2) && s > 0) {
      const int64_t group = s / kGroup * kGroup, edge = p.tiles - 1 - (rows_s.eos - 1) / kTileB;
      const int64_t first = edge > group ? edge : group;
      look_back(p, s, first, edge, warp, ch, ok, sh.back[warp][lane]);
      __syncthreads();
      carried(C, p, sh, s, first, edge, lane, ch, ok);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) C[k] = cut_before ? ex.H[k] : fmaf(ex.P[k], C[k], ex.H[k]);
    if (warp == 0 && ok && s % kGroup == kGroup - 1) {
#pragma unroll
      for (int k = 0; k < V; ++k)
        st_word(p.ends + s / kGroup * p.dim + ch + k,
                published(bits.last ? own.H[k] : fmaf(own.P[k], C[k], own.H[k])));
    }
    // states again, b <- the one before each row; dz
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (bits.start >> j & 1) initial(j, X);
      float h[V];
#pragma unroll
      for (int k = 0; k < V; ++k) h[k] = fmaf(a[j][k], X[k], b[j][k]), b[j][k] = X[k], X[k] = h[k];
      if (p.z && ok && row0 + j < p.total) {
        float z[V], d[V];
        vals_of(rz[j], z), vals_of(rd[j], d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float q = sigmoid<T>(z[k]);
          d[k] *= h[k] * fmaf(z[k] * q, 1.f - q, q);
        }
        if (!(bits.live >> j & 1)) {
#pragma unroll
          for (int k = 0; k < V; ++k) d[k] = 0.f;
        }
        store_vals<T, V>(p.dz, (row0 + j) * p.dim + ch, d);
      }
    }
    float se[V] = {}, sr[V] = {}, si[V] = {};
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const bool live = bits.live >> j & 1;
      float x[V], r[V], i[V], dx[V], dr[V], di[V];
      vals_of(rx[j], x), vals_of(rr[j], r), vals_of(ri[j], i);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float er = exp_minus<T>(r[k] + c.rb[k]), Rg = ptx::rcp_approx(1.f + er);
        float di_slope;
        const float I = sigmoid<T>(i[k] + c.ib[k], di_slope);
        const float g = bits.last >> j & 1 ? dy[j][k] : dy[j][k] + C[k];
        float m2;
        const float L2 = c.A2[k] * Rg;
        decay_of(L2, m2);
        const float rs = rsqrt_of(m2), m = m2 * rs, L = -kLn2 * L2;
        const float gm = g * m, av = a[j][k];
        const float e = live ? g * (av * av * (L * rs) * (I * x[k]) - av * b[j][k] * L) : 0.f;
        C[k] = av * g;
        dx[k] = live ? gm * I : 0.f;
        di[k] = live ? gm * x[k] * di_slope : 0.f;
        dr[k] = e * (er < 1.f ? er * Rg : 1.f - Rg);
        se[k] += e, sr[k] += dr[k], si[k] += di[k];
      }
      if (ok && row0 + j < p.total) {
        const int64_t at = (row0 + j) * p.dim + ch;
        store_vals<T, V>(p.dx, at, dx);
        store_vals<T, V>(p.dr, at, dr);
        store_vals<T, V>(p.di, at, di);
        if (p.dinit && (bits.start >> j & 1)) {
#pragma unroll
          for (int k = 0; k < V; ++k) p.dinit[(int64_t)rows_s.n[warp * R + j] * p.dim + ch + k] = C[k];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      sums[0][warp][lane * V + k] = se[k];
      sums[1][warp][lane * V + k] = sr[k];
      sums[2][warp][lane * V + k] = si[k];
    }
    if (threadIdx.x == 0) sh.next = next;
    __syncthreads();
    for (int q = threadIdx.x; q < 3 * 32 * V; q += 32 * kWarps) {
      const int w = q / (32 * V), l = q % (32 * V);
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += sums[w][k][l];
      if (cb + l < p.dim) p.part[(tile * 3 + w) * p.dim + cb + l] = v;
    }
    unit = sh.next;
    __syncthreads();
  }
}

// Before a pass: what is published is unset, the counters are zero, cu_seqlens is checked
// and what an empty sequence hands on is copied.
struct SetupParams {
  unsigned* status;
  uint64_t* words;           // from here on `count` words of ones
  int64_t count;
  const int64_t* cu;
  int64_t T, total;
  int32_t N, dim;
  const void* src;           // NULL: zeros
  void* dst;                 // NULL: nothing
  int32_t src_bf16, dst_bf16;
};
__global__ void __launch_bounds__(256) linrec_setup_kernel(SetupParams p) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t k = at; k < p.count; k += step) p.words[k] = kUnset;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    if (p.cu) check_seqlens(p.cu, p.N, p.total, p.status, kDevStatusBadSeqlens);
    else if (threadIdx.x == 0) p.status[0] = 0u;
    if (threadIdx.x >= 1) p.status[threadIdx.x] = 0u;
  }
  if (!p.dst || (!p.cu && p.T > 0)) return;
  for (int64_t n = blockIdx.x; n < p.N; n += gridDim.x) {
    if (p.cu && p.cu[n + 1] > p.cu[n]) continue;
    for (int d = threadIdx.x; d < p.dim; d += 256) {
      float h[1] = {};
      if (p.src) load_state<1>(h, p.src, n * p.dim + d, p.src_bf16);
      store_state<1>(p.dst, n * p.dim + d, h, p.dst_bf16);
    }
  }
}

// ------------------------------------------------------------------- host --
bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t tiles_of(int64_t total, int rows) { return (total + rows - 1) / rows; }
size_t join_bytes(int64_t tiles, int32_t dim) {  // what tiles publish
  return up256((size_t)tiles * dim * 8) + up256((size_t)(tiles / kGroup) * dim * 4);
}

kda_status check_sizes(const kda_linrec_problem* q, LinrecParams& p) {
  if (!q) return KDA_ERR_NULL_POINTER;
  const int64_t lim = int64_t(1) << 31;
  if (q->batch < 1 || q->T < 0 || q->dim < 1 || q->batch >= lim || q->T >= lim || q->batch * q->T >= lim)
    return KDA_ERR_INVALID_SHAPE;
  if (q->cu_seqlens && (q->batch != 1 || q->N < 1)) return KDA_ERR_INVALID_SHAPE;
  p.cu = q->cu_seqlens, p.T = q->T, p.total = q->batch * q->T;
  p.N = q->cu_seqlens ? q->N : (int32_t)q->batch, p.dim = q->dim;
  return KDA_OK;
}

// `pairs`: every row can be read two channels at a time.
kda_status check_linrec(const kda_linrec_problem* q, LinrecParams& p, bool& pairs) {
  const kda_status sizes = check_sizes(q, p);
  if (sizes != KDA_OK) return sizes;
  if (!q->A_log) return KDA_ERR_NULL_POINTER;
  const void* row[4] = {q->x, q->r, q->i, q->z};
  const int64_t stride[4] = {q->x_stride, q->r_stride, q->i_stride, q->z ? q->z_stride : q->dim};
  for (int64_t st : stride)
    if (st < q->dim || st >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
  if ((q->dtype != KDA_ROW_BF16 && q->dtype != KDA_ROW_FP32) ||
      (q->state_dtype != KDA_STATE_FP32 && q->state_dtype != KDA_STATE_BF16))
    return KDA_ERR_INVALID_ARG;
  if (p.total > 0 && (!q->x || !q->r || !q->i)) return KDA_ERR_NULL_POINTER;
  const size_t e = q->dtype == KDA_ROW_FP32 ? 4 : 2, se = q->state_dtype == KDA_STATE_FP32 ? 4 : 2;
  pairs = q->dtype == KDA_ROW_BF16 && q->dim % 2 == 0;
  for (int k = 0; k < 4; ++k) {
    if (!al_to(row[k], e)) return KDA_ERR_MISALIGNED;
    pairs = pairs && al_to(row[k], 4) && stride[k] % 2 == 0;
  }
  if (!al_to(q->A_log, 4) || !al_to(q->r_bias, 4) || !al_to(q->i_bias, 4) ||
      !al_to(q->initial_state, se) || !al_to(q->cu_seqlens, 8))
    return KDA_ERR_MISALIGNED;
  p.x = q->x, p.r = q->r, p.i = q->i, p.z = q->z;
  p.x_s = q->x_stride, p.r_s = q->r_stride, p.i_s = q->i_stride, p.z_s = stride[3];
  p.A_log = q->A_log, p.r_bias = q->r_bias, p.i_bias = q->i_bias;
  p.init = q->initial_state, p.state_bf16 = q->state_dtype == KDA_STATE_BF16;
  p.stall = q->debug_stall;
  return KDA_OK;
}

// Tiles and channel blocks of a pass, and its part of the workspace.
bool plan_pass(LinrecParams& p, int rows, int channels, uint8_t*& ws) {
  p.tiles = tiles_of(p.total, rows);
  p.blocks = (p.dim + channels - 1) / channels;
  p.agg = reinterpret_cast<uint64_t*>(ws);
  p.ends = reinterpret_cast<unsigned*>(ws + up256((size_t)p.tiles * p.dim * 8));
  ws += join_bytes(p.tiles, p.dim);
  return p.tiles * p.blocks < (int64_t(1) << 31);
}

cudaError_t launch_setup(const LinrecParams& p, void* words, size_t bytes, const void* src, bool src_bf16,
                         void* dst, bool dst_bf16, cudaStream_t stream) {
  SetupParams s = {};
  s.status = p.status, s.words = static_cast<uint64_t*>(words), s.count = (int64_t)(bytes / 8);
  s.cu = p.cu, s.T = p.T, s.total = p.total, s.N = p.N, s.dim = p.dim;
  s.src = src, s.dst = dst, s.src_bf16 = src_bf16, s.dst_bf16 = dst_bf16;
  const int64_t want = (s.count + 1023) / 1024 + (dst && p.cu ? p.N : 1);
  linrec_setup_kernel<<<(unsigned)(want < 608 ? want : 608), 256, 0, stream>>>(s);
  return cudaGetLastError();
}

template <typename K>
cudaError_t launch_tiles(K kernel, const LinrecParams& p, cudaStream_t stream) {
  int sms = 0;
  if (sm_count(&sms) != KDA_OK) return cudaErrorUnknown;
  const int64_t units = p.tiles * p.blocks, most = 2 * (int64_t)sms;
  kernel<<<(unsigned)(units < most ? units : most), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}
template <bool OUT>
cudaError_t launch_fwd(const LinrecParams& p, bool f32, bool pairs, cudaStream_t stream) {
  return f32     ? launch_tiles(linrec_fwd_kernel<float, 1, OUT>, p, stream)
         : pairs ? launch_tiles(linrec_fwd_kernel<bf16, 2, OUT>, p, stream)
                 : launch_tiles(linrec_fwd_kernel<bf16, 1, OUT>, p, stream);
}

size_t states_bytes(int64_t total, int32_t dim) {
  return (size_t)(total / KDA_LINREC_CHUNK + 1) * dim * sizeof(float);
}
size_t fwd_bytes(const LinrecParams& p) {
  return KDA_STATUS_BYTES + join_bytes(tiles_of(p.total, kTileF), p.dim);
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_linrec_get_states_size(int64_t total_tokens, int32_t dim, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  if (total_tokens < 0 || total_tokens >= (int64_t(1) << 31) || dim < 1) return KDA_ERR_INVALID_SHAPE;
  *bytes = kda::states_bytes(total_tokens, dim);
  return KDA_OK;
}

kda_status kda_linrec_get_workspace_size(const kda_linrec_problem* problem, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  kda::LinrecParams p = {};
  const kda_status st = kda::check_sizes(problem, p);
  if (st != KDA_OK) return st;
  *bytes = kda::fwd_bytes(p);
  return KDA_OK;
}

kda_status kda_linrec_bwd_get_workspace_size(const kda_linrec_problem* problem, int32_t have_states,
                                             size_t* bytes) {
  using namespace kda;
  if (!bytes) return KDA_ERR_NULL_POINTER;
  LinrecParams p = {};
  const kda_status st = check_sizes(problem, p);
  if (st != KDA_OK) return st;
  const int64_t tiles = tiles_of(p.total, kTileB);
  *bytes = KDA_STATUS_BYTES + join_bytes(tiles, p.dim) + up256((size_t)tiles * 3 * p.dim * sizeof(float));
  if (!have_states)
    *bytes += join_bytes(tiles_of(p.total, kTileF), p.dim) + up256(states_bytes(p.total, p.dim));
  return KDA_OK;
}

kda_status kda_linrec_fwd(const kda_linrec_problem* problem, void* out, void* final_state,
                          void* chunk_states, size_t chunk_states_bytes, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  LinrecParams p = {};
  bool pairs = false;
  kda_status st = check_linrec(problem, p, pairs);
  if (st != KDA_OK) return st;
  const bool f32 = problem->dtype == KDA_ROW_FP32;
  if (p.total > 0 && !out) return KDA_ERR_NULL_POINTER;
  if (!al_to(out, f32 ? 4 : 2) || !al_to(final_state, p.state_bf16 ? 2 : 4) || !al_to(chunk_states, 16) ||
      !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  if (chunk_states && chunk_states_bytes < states_bytes(p.total, p.dim)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  const bool step = !p.cu && p.T > 0 && p.T <= kStepTokens && !chunk_states;
  if (!step && !workspace) return KDA_ERR_NULL_POINTER;
  if (workspace && workspace_bytes < (step ? KDA_STATUS_BYTES : fwd_bytes(p)))
    return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  pairs = pairs && al_to(out, 4);
  p.out = out, p.fin = final_state, p.states = static_cast<float*>(chunk_states);
  p.status = static_cast<unsigned*>(workspace);
  if (step) {
    if (workspace && cudaMemsetAsync(workspace, 0, 4, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const int V = pairs ? 2 : 1;
    const int64_t blocks = ((int64_t)p.N * ((p.dim + V - 1) / V) + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
    auto kernel = f32 ? linrec_step_kernel<float, 1> : pairs ? linrec_step_kernel<bf16, 2> : linrec_step_kernel<bf16, 1>;
    kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES;
  if (!plan_pass(p, kTileF, pairs ? 64 : 32, ws)) return KDA_ERR_INVALID_SHAPE;
  p.ticket = p.status + 1;
  cudaError_t e = launch_setup(p, p.agg, fwd_bytes(p) - KDA_STATUS_BYTES, p.init, p.state_bf16,
                               p.fin == p.init ? nullptr : p.fin, p.state_bf16, stream);
  if (e == cudaSuccess && p.total > 0) e = launch_fwd<true>(p, f32, pairs, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_linrec_bwd(const kda_linrec_problem* problem, const void* dout, const void* dfinal_state,
                          const void* chunk_states, size_t chunk_states_bytes, void* dx, void* dr,
                          void* di, void* dz, float* dA_log, float* dr_bias, float* di_bias,
                          float* dinitial_state, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  using namespace kda;
  LinrecParams p = {};
  bool pairs = false;
  kda_status st = check_linrec(problem, p, pairs);
  if (st != KDA_OK) return st;
  const bool f32 = problem->dtype == KDA_ROW_FP32;
  const size_t e = f32 ? 4 : 2;
  if (!dA_log || !workspace || (p.total > 0 && (!dout || !dx || !dr || !di || (p.z && !dz))))
    return KDA_ERR_NULL_POINTER;
  for (const void* q : {dout, (const void*)dx, (const void*)dr, (const void*)di, (const void*)dz}) {
    if (!al_to(q, e)) return KDA_ERR_MISALIGNED;
    pairs = pairs && al_to(q, 4);
  }
  if (!al_to(dA_log, 4) || !al_to(dr_bias, 4) || !al_to(di_bias, 4) || !al_to(dinitial_state, 4) ||
      !al_to(dfinal_state, p.state_bf16 ? 2 : 4) || !al_to(chunk_states, 16) || !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  if (chunk_states && chunk_states_bytes < states_bytes(p.total, p.dim)) return KDA_ERR_WORKSPACE_TOO_SMALL;
  size_t need = 0;
  st = kda_linrec_bwd_get_workspace_size(problem, chunk_states != nullptr, &need);
  if (st != KDA_OK) return st;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  p.status = static_cast<unsigned*>(workspace);
  uint8_t* ws = static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES;
  uint8_t* const published_at = ws;
  LinrecParams f = p;
  f.stall = 0;
  const int channels = pairs ? 64 : 32;
  bool fits = plan_pass(p, kTileB, channels, ws);
  if (!chunk_states) fits = fits && plan_pass(f, kTileF, channels, ws);
  if (!fits) return KDA_ERR_INVALID_SHAPE;
  const size_t published_bytes = (size_t)(ws - published_at);
  p.part = reinterpret_cast<float*>(ws);
  ws += up256((size_t)p.tiles * 3 * p.dim * sizeof(float));
  p.states = const_cast<float*>(static_cast<const float*>(chunk_states));
  if (!chunk_states) p.states = f.states = reinterpret_cast<float*>(ws);
  p.ticket = p.status + 1, f.ticket = p.status + 2;
  p.dout = dout, p.dfin = dfinal_state;
  p.dx = dx, p.dr = dr, p.di = di, p.dz = dz, p.dinit = dinitial_state;
  cudaError_t err = launch_setup(p, published_at, published_bytes, dfinal_state, p.state_bf16,
                                 dinitial_state, false, stream);
  if (err == cudaSuccess && p.total > 0) {
    if (!chunk_states) err = launch_fwd<false>(f, f32, pairs, stream);
    if (err == cudaSuccess)
      err = f32     ? launch_tiles(linrec_bwd_kernel<float, 1>, p, stream)
            : pairs ? launch_tiles(linrec_bwd_kernel<bf16, 2>, p, stream)
                    : launch_tiles(linrec_bwd_kernel<bf16, 1>, p, stream);
  }
  if (err == cudaSuccess)
    err = launch_column_sums(p.part, p.tiles, 3 * (int64_t)p.dim, 3 * (int64_t)p.dim, p.dim, p.dim, dA_log,
                             dr_bias, di_bias, stream);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
