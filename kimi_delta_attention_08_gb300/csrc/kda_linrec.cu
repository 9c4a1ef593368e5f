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
// Each row is read once and written once.  A block takes a tile of 128 rows (backward: 64) by
// 64 channels; its warps take consecutive runs of 16 (8) rows, a lane two channels (fp32 rows, and
// bf16 ones off 4 bytes: 32 channels, a lane one).  A run is
// scanned in registers from zero along with the product of its decays; runs, tiles and
// groups of tiles are joined as affine steps, in shared memory and through the workspace;
// then each run is walked again from the state before it.  So a prompt of any length fills
// the GPU in one pass over its rows, with the same sums in every run of the program.
//
// Tiles.  Each publishes what it does to a state, (product, end from zero), as soon as it has
// it.  Tiles are handed out by an atomic counter in the order of their rows, so a tile only
// waits for tiles that already run, and what is published is its own flag: words that were
// filled with ones before (no arithmetic result has these bits).  Waits give up after half a
// second; what they waited for is then taken as no number, so that no result looks right.
//
// Device time: forward, 8 x 4,096 tokens of 4,096 channels, bf16, 257 us (4.2 TB/s of rows; fp32
// 342, 6.3 TB/s); 74,080 packed tokens of 2,048 channels with a gate 431; 65,536 + 5 x 1,024
// tokens of 1,024 channels 201; forward and backward of 4 x 4,096 tokens of 4,096 channels with a
// gate 556.  Bound by latency: no unit is near its peak (of 2 x 4,096 tokens, forward and
// backward: 0.52 and 0.50 instructions a clock and scheduler, which could issue one, FMA pipe 21 %,
// special-function unit 25 and 24 %, DRAM 42 and 28 %).  Decays and inputs in registers leave 16 warps
// per SM, too few to cover the three barriers at which a tile's runs meet: more warps wait
// there (1.8 and 1.6 for each instruction that issues) than for anything else.  Where few channels
// leave many tiles of one at work they also wait for each other: 154 us for the long prompt
// without that.  41 instructions a value forward, 124 backward.  Runs of 8 rows by four channels
// take 262, 502 and 261 us for the three forwards, decays and inputs in shared memory with three
// blocks per SM 287, 450 and 266.
#include <algorithm>
#include <type_traits>

#include "kda_internal.h"
#include "kda_rows.cuh"
#include "kda_scan.cuh"
#include "../../include/kda_layer.h"

namespace kda {
namespace {

using namespace rows;

constexpr int kWarps = 8;
constexpr int kRowsF = 16, kRowsB = 8;            // rows of a run: forward, backward
constexpr int kTileF = kWarps * kRowsF, kTileB = kWarps * kRowsB;
constexpr int kGroup = 16;                        // tiles of a group
constexpr int kStepTokens = 8;                    // prompts up to this length: the step kernel
constexpr uint64_t kWaitNs = 500000000ull;
constexpr uint64_t kUnset = ~0ull;
static_assert(kTileB == KDA_LINREC_CHUNK && kTileF == 2 * kTileB, "one and two saved states per tile");

struct LinrecParams {
  const void *x, *r, *i, *z, *dout;
  uint32_t x_s, r_s, i_s, z_s;
  float* gates;              // [3][dim]: what load_gates computes
  const float *A_log, *r_bias, *i_bias;
  const void *init, *dfin;
  int32_t state_bf16, stall;
  const int64_t* cu;
  int64_t T, total;
  int32_t N, dim, blocks;    // blocks: of channels
  int64_t tiles;             // of rows
  unsigned units, strips, strip_tiles;  // see unit_of
  void *out, *fin;
  float* states;             // [total / KDA_LINREC_CHUNK + 1][dim]
  unsigned *status, *ticket;
  uint64_t* agg;             // [tiles][dim]: (product, end from zero) of each tile
  uint64_t* group_agg;       // [tiles / kGroup][dim]: the same of each whole group
  unsigned* ends;            // [tiles / kGroup][dim]: the state after each whole group
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

// Bits that are published: those of all ones mean "not set", so that NaN becomes another.
__device__ __forceinline__ unsigned published(float v) {
  const unsigned b = __float_as_uint(v);
  return b == ~0u ? 0x7FFFFFFFu : b;
}

// The last sequence that starts at row t or before, searched for by a warp, 32 places at a time.
__device__ __noinline__ int sequence_at(const int64_t* cu, int N, int64_t t, int lane) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const unsigned each = ((unsigned)(hi - lo) + 31) / 32, at = lo + lane * each;
    const unsigned below = __ballot_sync(0xffffffffu, at < (unsigned)hi && (lane == 0 || __ldg(cu + at) <= t));
    lo += (31 - __clz(below)) * each;
    hi = (int)min((unsigned)hi, lo + each);
  }
  return lo;
}
// The sequence of row t, a lane's of 32 that follow one another, and its bounds; false where t belongs
// to none.  Of many sequences the first row's is found by all lanes together; the others' are among the
// next 32 but for empty ones (2,000 single tokens of 4,096 channels 81 us without, 58 with it; not
// `TOGETHER` in the kernels for rows off 16 bytes, whose registers would not take it).
template <bool TOGETHER>
__device__ __forceinline__ bool row_sequence(const LinrecParams& p, int64_t t, int lane, int& n, int64_t& bos,
                                             int64_t& eos) {
  if (!p.cu) {
    if (t >= p.total) return false;
    n = (int)((uint32_t)t / (uint32_t)p.T);
    bos = (int64_t)n * p.T, eos = bos + p.T;
    return true;
  }
  int lo = 0, hi = p.N;
  if (TOGETHER && hi > 64) {
    lo = sequence_at(p.cu, hi, t - lane, lane);
    if (hi - lo > 33 && __ldg(p.cu + lo + 33) > t) hi = lo + 33;
  }
  if (t >= p.total) return false;
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
// What a value's gates and step need of its channel (load_gates).
template <int V>
struct Gates {
  Vals<V> A2, cr, ci;
};
// Copies of a thread's own: its values of the tile to come wait in shared memory, in slots
// that no other thread touches, so that nothing but its own copies is waited for.
template <int BYTES>
__device__ __forceinline__ void copy_own(uint32_t slot, const void* p, bool there) {
  static_assert(BYTES == 2 || BYTES == 4 || BYTES == 8, "one or two channels");
  if constexpr (BYTES == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(slot), "l"(p), "r"(there ? 8 : 0) : "memory");
  else if constexpr (BYTES == 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(slot), "l"(p), "r"(there ? 4 : 0) : "memory");
  else {  // rows at odd addresses
    const unsigned short v = there ? __ldg(static_cast<const unsigned short*>(p)) : (unsigned short)0;
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(slot), "h"(v) : "memory");
  }
}
template <typename T, int V, int kRows>
struct Slots {
  static constexpr int kBytes = V * (int)sizeof(T), kRow = 32 * kBytes;  // of a lane, of a warp's row
  static constexpr int kRun = kRows * kRow, kArray = kWarps * kRun;      // of a run, of a tile, of one array
  // the lane's values of a run's rows, `stride` elements apart, of which the first n exist
  static __device__ __forceinline__ void copy(uint32_t at, const void* p, int64_t row0, uint32_t stride, int ch,
                                              int n) {
    const char* const from = reinterpret_cast<const char*>(static_cast<const T*>(p) + row0 * stride + ch);
    if (n == kRows) {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        copy_own<kBytes>(at + j * kRow, from + (uint64_t)stride * (uint32_t)(j * sizeof(T)), true);
    } else {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        copy_own<kBytes>(at + j * kRow,
                         j < n ? from + (uint64_t)stride * (uint32_t)(j * sizeof(T)) : static_cast<const char*>(p),
                         j < n);
    }
  }
  static __device__ __forceinline__ Vals<V> get(const uint8_t* at, int j) {
    Raw<T, V> r;
    const uint8_t* const q = at + j * kRow;
    static_assert(kBytes == 2 || kBytes == 4, "one channel, or two of bf16");
    if constexpr (kBytes == 2) r.w[0] = (uint32_t)*reinterpret_cast<const unsigned short*>(q);
    else r.w[0] = *reinterpret_cast<const uint32_t*>(q);
    float f[V];
    if constexpr (V == 1 && sizeof(T) == 4) f[0] = __uint_as_float(r.w[0]);
    else unpack(r, f);
    return vals_from(f);
  }
  // the channel's gates, one lane's after the other's
  static constexpr int kGates = 3 * 32 * kWarps * V * 4;
  static __device__ __forceinline__ void copy_gates(uint32_t at, const float* g, int dim, int ch, bool ok) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      copy_own<4 * V>(at + k * 32 * kWarps * V * 4, ok ? g + k * (int64_t)dim + ch : g, ok);
  }
  static __device__ __forceinline__ void gates(Gates<V>& c, const uint8_t* at) {
    Vals<V>* const to[3] = {&c.A2, &c.cr, &c.ci};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      Raw<float, V> r;
      load_words<true>(r.w, at + k * 32 * kWarps * V * 4);
      float f[V];
      unpack(r, f);
      *to[k] = vals_from(f);
    }
  }
};
template <typename T, int V>
__device__ __forceinline__ void vals_of(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (V == 1) f[0] = __uint_as_float(r.w[0]);
  else unpack(r, f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vals(void* p, int64_t at, const float (&f)[V]) {
  store_row<T, V, (V > 1)>(static_cast<T*>(p) + at, f, 1, 1);
}

// Rows of a tile: every row's sequence, and a bit per row.
template <int TILE>
struct TileRows {
  int n[TILE];
  uint32_t start[TILE / 32], last[TILE / 32], live[TILE / 32];  // first row of its sequence, last one, of any
  int64_t bos, eos;              // of the first row's sequence, of the last row's
};
template <bool TOGETHER, int TILE>
__device__ __forceinline__ void find_rows(TileRows<TILE>& s, const LinrecParams& p, int64_t row0, int lane,
                                          int first = 0, int step = 1) {  // of a tile's 32 rows each
#pragma unroll
  for (int h = first; h < TILE / 32; h += step) {
    const int64_t t = row0 + 32 * h + lane;
    int n = 0;
    int64_t bos = 0, eos = 0;
    const bool live = row_sequence<TOGETHER>(p, t, lane, n, bos, eos);
    s.n[32 * h + lane] = n;
    const unsigned start = __ballot_sync(0xffffffffu, live && t == bos);
    const unsigned last = __ballot_sync(0xffffffffu, live && t + 1 == eos);
    const unsigned alive = __ballot_sync(0xffffffffu, live);
    if (lane == 0) s.start[h] = start, s.last[h] = last, s.live[h] = alive;
    if (h == 0 && lane == 0) s.bos = bos;
    if (h == TILE / 32 - 1 && lane == 31) s.eos = eos;
  }
}
// A run's rows: bit j for row j.
struct RowBits {
  unsigned start, last, live;
};
template <int TILE>
__device__ __forceinline__ RowBits run_rows(const TileRows<TILE>& s, int warp) {
  constexpr int R = TILE / kWarps;
  constexpr unsigned mask = (1u << R) - 1;
  const int at = warp * R / 32, by = warp * R % 32;
  return {s.start[at] >> by & mask, s.last[at] >> by & mask, s.live[at] >> by & mask};
}

constexpr float kBiasScale16 = -kLog2e, kBiasScale32 = 1.f;
template <typename T, int V>
__device__ __forceinline__ void load_gates(Gates<V>& c, const LinrecParams& p, int ch, bool ok) {
  // bf16 rows: exp(-(v + bias)) = 2^(-v log2 e - bias log2 e)
  constexpr float k = sizeof(T) < 4 ? kBiasScale16 : kBiasScale32;
  float A2[V], cr[V], ci[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    A2[e] = ok ? scan::rate_of(__ldg(p.A_log + ch + e)) : 0.f;
    cr[e] = ok && p.r_bias ? k * __ldg(p.r_bias + ch + e) : 0.f;
    ci[e] = ok && p.i_bias ? k * __ldg(p.i_bias + ch + e) : 0.f;
  }
  c.A2 = vals_from(A2), c.cr = vals_from(cr), c.ci = vals_from(ci);
}

// a and b = m I x of a pair of values.  m^2 and m come scaled by 2^24 and 2^12, so that what
// the hardware takes for zero (below 2^-126) is zero in fp32 too, and I (fp32 rows) by 2^-12.  From
// L2 = -L log2 e: small steps, u = 2 L up to 1/4, take 1 - exp(-u) = u P(u), P of degree 3 with
// P(0) = 1 fitted by reweighted least squares to an even relative error (2.9e-7, half of
// that in m); 1 - a^2 would have none of its digits right for them.  From there on 1 - a^2
// is good to 8e-7.  The exponent is raised by the hardware exponential's mean error (see the
// scan's decay).
template <typename T>
__device__ __forceinline__ pair gate_exp(pair v, pair c) {  // exp(-(v + bias))
  if constexpr (sizeof(T) < 4) return pex2(pfma(v, pr(-kLog2e), c));
  else return exp_minus<T>(padd(v, c));
}
// exp(v + bias) of bf16 rows, at most 2^30: E / (1 + E) is 1 from 2^24 on.  NaN stays.
__device__ __forceinline__ pair plus_exp(pair v, pair c) {
  const float2 n = un(pfma(v, pr(-kLog2e), c));
  float2 e = make_float2(ptx::ex2_approx(-n.x), ptx::ex2_approx(-n.y));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.x) : "f"(0x1p30f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(e.y) : "f"(0x1p30f));
  return pr(e.x, e.y);
}
__device__ __forceinline__ pair rcp_of(pair v) {
  return pr(ptx::rcp_approx(un(v).x), ptx::rcp_approx(un(v).y));
}
__device__ __forceinline__ pair rsqrt_of(pair v) {  // finite at zero; else v is 2^-125 at least
  float2 r = un(padd(v, pr(FLT_MIN)));
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(r.x));
  asm("rsqrt.approx.ftz.f32 %0, %0;" : "+f"(r.y));
  return pr(r.x, r.y);
}
constexpr float kSmallStep = -0.18033688f;  // L2 at u = 1/4
__device__ __forceinline__ pair scaled_m2(pair L2, pair a) {
  pair q = pfma(pr(-2346124.25f), L2, pr(-7425258.5f));
  q = pfma(q, L2, pr(-16120601.f));
  q = pfma(q, L2, pr(-23258160.f));
  const float2 small = un(pmul(q, L2)), big = un(pfma(pmul(a, pr(-0x1p24f)), a, pr(0x1p24f))), l = un(L2);
  return pr(l.x < kSmallStep ? big.x : small.x, l.y < kSmallStep ? big.y : small.y);
}
template <typename T>
__device__ __forceinline__ void step_of(pair x, pair r, pair i, pair A2, pair cr, pair ci, pair& a, pair& b) {
  const pair L2 = pmul(A2, rcp_of(padd(gate_exp<T>(r, cr), pr(1.f))));
  a = pex2(padd(L2, pr(2.5e-8f)));
  const pair m2 = scaled_m2(L2, a);
  if constexpr (sizeof(T) < 4) {
    // m I = m^2 E / sqrt(m^2 (1 + E)^2), E = exp(i): one operation of the special-function unit for
    // the root and the reciprocal (8 x 4,096 tokens of 4,096 channels 265 to 259 us; fp32 rows, whose
    // exponential costs more on this side, 342 to 347)
    const pair E = plus_exp(i, ci), d = pfma(E, pr(4096.f), pr(4096.f));
    b = pmul(pmul(pmul(m2, rsqrt_of(pmul(pmul(m2, d), d))), E), x);
  } else {
    const pair I = rcp_of(pfma(gate_exp<T>(i, ci), pr(4096.f), pr(4096.f)));
    b = pmul(pmul(pmul(m2, rsqrt_of(m2)), I), x);
  }
}
// Two rows' steps: single channels pair up across them.
__device__ __forceinline__ pair two(const Vals<1>& u, const Vals<1>& v) { return pr(u.v[0], v.v[0]); }
__device__ __forceinline__ void apart(pair p, Vals<1>& u, Vals<1>& v) { u.v[0] = un(p).x, v.v[0] = un(p).y; }
template <typename T, int V>
__device__ __forceinline__ void step_of(const Vals<V> (&x)[2], const Vals<V> (&r)[2], const Vals<V> (&i)[2],
                                        const Gates<V>& c, Vals<V>& a0, Vals<V>& b0, Vals<V>& a1, Vals<V>& b1) {
  if constexpr (V == 1) {
    pair a, b;
    step_of<T>(two(x[0], x[1]), two(r[0], r[1]), two(i[0], i[1]), pr(c.A2.v[0]), pr(c.cr.v[0]), pr(c.ci.v[0]), a, b);
    apart(a, a0, a1), apart(b, b0, b1);
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      step_of<T>(x[0].v[k], r[0].v[k], i[0].v[k], c.A2.v[k], c.cr.v[k], c.ci.v[k], a0.v[k], b0.v[k]);
      step_of<T>(x[1].v[k], r[1].v[k], i[1].v[k], c.A2.v[k], c.cr.v[k], c.ci.v[k], a1.v[k], b1.v[k]);
    }
  }
}
// `row(array, j)`: the values of x, r and i.
template <typename T, int V, int kRows, typename ROW>
__device__ __forceinline__ void steps_of(ROW row, const Gates<V>& c, Vals<V> (&a)[kRows], Vals<V> (&b)[kRows]) {
#pragma unroll
  for (int j = 0; j < kRows; j += 2) {
    const Vals<V> x[2] = {row(0, j), row(0, j + 1)}, r[2] = {row(1, j), row(1, j + 1)}, i[2] = {row(2, j), row(2, j + 1)};
    step_of<T>(x, r, i, c, a[j], b[j], a[j + 1], b[j + 1]);
  }
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> vals_of(const Raw<T, V>& r) {
  float f[V];
  vals_of(r, f);
  return vals_from(f);
}
template <typename T, int V>
__device__ __forceinline__ Vals<V> silu_of(const Vals<V>& z) {
  return mul_of(z, sigmoid<T>(z));
}

// The runs of a tile.
template <int V>
struct Runs {
  float P[kWarps][32 * V], H[kWarps][32 * V];  // what each run does to a state; H then holds
                                               // the state before it
  float parts[kWarps / V][2][32 * V], tile[2][32 * V];  // the join's
  unsigned char cut[kWarps];                   // whether a run holds a sequence's start
};
// The unit of work that a ticket stands for: rows' tile first, all channel blocks of one before
// the next.  A batch of sequences that are whole tiles is walked a tile of each in turn: a tile
// then rarely waits for the one before it (8 x 4,096 tokens of 4,096 channels 379 us without,
// 311 with it).
struct Unit {
  int tile, block;                             // the tile in the order of the walk; -1: none
};
__device__ __forceinline__ Unit unit_of(const LinrecParams& p, unsigned ticket) {
  const unsigned blocks = p.blocks, w = ticket / blocks, q = w / p.strips;
  return {ticket < p.units ? (int)((w - q * p.strips) * p.strip_tiles + q) : -1, (int)(ticket - w * blocks)};
}
// What a block's warps share.  This turn's unit and rows and the next one's alternate, so that
// three barriers a turn are enough: the runs are there, the parts of the look back are, and
// the states before the runs are.
template <int V, int TILE>
struct BlockShared {
  Runs<V> runs;
  TileRows<TILE> rows[2];
  Unit unit[2];
};
// The first turn's unit and rows.
template <bool FORWARD, bool TOGETHER, int V, int TILE>
__device__ __forceinline__ void start_block(const LinrecParams& p, BlockShared<V, TILE>& sh, int warp, int lane) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the launch before, see launch_behind
  if (threadIdx.x == 0) sh.unit[0] = unit_of(p, atomicAdd(p.ticket, 1u));
  __syncthreads();
  const int64_t s = sh.unit[0].tile;
  if (s >= 0) find_rows<TOGETHER>(sh.rows[0], p, (FORWARD ? s : p.tiles - 1 - s) * TILE, lane, warp, kWarps);
  __syncthreads();
}
template <int V>
__device__ __forceinline__ void put(float (&at)[32 * V], int lane, const Vals<V>& v) {
  float f[V];
  vals_to(v, f);
#pragma unroll
  for (int k = 0; k < V; ++k) at[lane * V + k] = f[k];
}
template <int V>
__device__ __forceinline__ Vals<V> read_vals(const float* at) {
  Raw<float, V> r;
  load_words(r.w, at);
  float f[V];
  unpack(r, f);
  return vals_from(f);
}
template <int V>
__device__ __forceinline__ void read_gates(Gates<V>& c, const LinrecParams& p, int ch) {
  c.A2 = read_vals<V>(p.gates + ch);
  c.cr = read_vals<V>(p.gates + p.dim + ch);
  c.ci = read_vals<V>(p.gates + 2 * (int64_t)p.dim + ch);
}
template <int V>
__device__ __forceinline__ Vals<V> get(const float (&at)[32 * V], int lane) {
  float f[V];
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = at[lane * V + k];
  return vals_from(f);
}

// The word at `p` once it is set; after the limit (or another wait's) NaN, with the status.
template <typename W>
__device__ __noinline__ W await_word(const W* p, unsigned* status) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const W v = ld_word(p);
      if (v != static_cast<W>(kUnset)) return v;
    }
    if (ptx::global_timer_ns() - t0 > kWaitNs || (ld_word(status) & kDevStatusTimeout)) {
      atomicOr(status, kDevStatusTimeout);
      return static_cast<W>(0x7FFFFFFF7FFFFFFFull);
    }
  }
}

// Tiles form groups of kGroup.  The state before a tile is that before its group, taken through
// what the tiles of the group before it do together; this is composed from zero in parts of
// the group, by the threads that share a channel, and the parts in their order: the same sums
// in every run.  A group's last tile also publishes what the whole group does, and the state
// at its end, so those follow one from the other without the tiles between.
__device__ __forceinline__ float stepped(uint64_t w, float X) {
  return fmaf(__uint_as_float((unsigned)w), X, __uint_as_float((unsigned)(w >> 32)));
}
__device__ __forceinline__ uint64_t step_word(float P, float H) {
  return (uint64_t)published(P) | ((uint64_t)published(H) << 32);
}

// The state at the end of group g, in a sequence that starts in group `edge` or before the
// window: that of the nearest group which has published one (the window's last is waited
// for), taken through the groups since then.  found: the word of group g, as it was.
constexpr int kWindow = 4;
__device__ __forceinline__ float state_after_group(const LinrecParams& p, int64_t g, int64_t edge, int ch,
                                                   unsigned found) {
  if (found != ~0u) return __uint_as_float(found);
  const int64_t dim = p.dim;
  const unsigned* const ends = p.ends + g * dim + ch;
  const uint64_t* const agg = p.group_agg + g * dim + ch;
  const int last = (int)min((int64_t)kWindow - 1, g - edge);
  unsigned e[kWindow];
  uint64_t w[kWindow - 1];
#pragma unroll
  for (int q = 0; q < kWindow; ++q) {
    e[q] = q <= last ? ld_word(ends - q * dim) : ~0u;
    if (q < kWindow - 1) w[q] = q < last ? ld_word(agg - q * dim) : 0;
  }
  int at = last;
#pragma unroll
  for (int q = kWindow - 1; q >= 0; --q)
    if (e[q] != ~0u) at = q, found = e[q];
  if (found == ~0u) found = await_word(ends - last * dim, p.status);
  float X = __uint_as_float(found);
#pragma unroll
  for (int q = kWindow - 2; q >= 0; --q)
    if (q < at) {
      if (w[q] == kUnset) w[q] = await_word(agg - q * dim, p.status);
      X = stepped(w[q], X);
    }
  return X;
}

// The join of a tile, by all threads: kParts of them share a channel.
template <int V, bool FORWARD>
struct Join {
  static constexpr int kParts = kWarps / V, kPer = kGroup / kParts;
  const LinrecParams& p;
  int64_t s, first, from;    // the tile, its group's first, the first that is looked back at
  int c, part, ch;
  bool carry, whole, ok;     // the tile goes on; so does its group
  uint64_t w[kPer];
  unsigned before;           // the state before the group

  // Before the runs are there: what the tiles before this one have published so far.
  __device__ __forceinline__ Join(const LinrecParams& p, int64_t s, int64_t edge, bool carry, int c0)
      : p(p), s(s), first(s / kGroup * kGroup), c(threadIdx.x % (32 * V)), part(threadIdx.x / (32 * V)),
        ch(c0 + c), carry(carry), ok(ch < p.dim) {
    from = edge > first ? edge : first;
    whole = carry && edge < first;
    before = ~0u;
    if (!carry || !ok) return;
    if (part == 0 && whole) before = ld_word(p.ends + (s / kGroup - 1) * p.dim + ch);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int64_t at = first + part * kPer + q;
      w[q] = at >= from && at < s ? ld_word(p.agg + at * p.dim + ch) : 0;
    }
  }
  // The runs are there: together they are published; the part's tiles are composed.
  __device__ __forceinline__ void parts(Runs<V>& sh, float& Pt, float& Ht) {
    Pt = 1.f, Ht = 0.f;      // of the tiles
    if (part == kParts - 1 && ok) {
      const uint64_t cuts = *reinterpret_cast<const uint64_t*>(sh.cut);
      float P = 1.f, H = 0.f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        const int r = FORWARD ? q : kWarps - 1 - q;
        const float Pr = sh.P[r][c], Hr = sh.H[r][c];
        H = cuts >> (8 * r) & 1 ? Hr : fmaf(Pr, H, Hr);
        P *= Pr;
      }
      if (cuts) P = 0.f;
      // (a tile that does not hand on what it is given is only asked for its step where
      // cu_seqlens is inconsistent; no wait is left without an answer then either)
      if (!(p.stall && s == 0)) st_word(p.agg + s * p.dim + ch, step_word(P, H));
      sh.tile[0][c] = P, sh.tile[1][c] = H;
    }
    if (carry && ok) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int64_t at = first + part * kPer + q;
        if (at < from || at >= s) continue;
        if (w[q] == kUnset) w[q] = await_word(p.agg + at * p.dim + ch, p.status);
        Ht = stepped(w[q], Ht);
        Pt *= __uint_as_float((unsigned)w[q]);
      }
    }
    if (part > 0) sh.parts[part - 1][0][c] = Pt, sh.parts[part - 1][1][c] = Ht;
  }
  // The parts are there (part 0 only): the state before the tile, and before each run.
  __device__ __forceinline__ float finish(Runs<V>& sh, int64_t edge, float Pt, float Ht) {
    float X = 0.f;
    const uint64_t cuts = *reinterpret_cast<const uint64_t*>(sh.cut);
    const float P = sh.tile[0][c], H = sh.tile[1][c];
    const int64_t g = s / kGroup;
    const bool last = s == first + kGroup - 1 && !(p.stall && s == 0);
    if (carry) {
#pragma unroll
      for (int q = 0; q < kParts - 1; ++q) {
        const float Pq = sh.parts[q][0][c];
        Ht = fmaf(Pq, Ht, sh.parts[q][1][c]), Pt *= Pq;
      }
      const float Hg = fmaf(P, Ht, H), Pg = P * Pt;
      X = Ht;
      if (whole) {
        if (last) st_word(p.group_agg + g * p.dim + ch, step_word(Pg, Hg));
        const float G = state_after_group(p, g - 1, edge / kGroup, ch, before);
        X = fmaf(Pt, G, Ht);
        if (last) st_word(p.ends + g * p.dim + ch, published(cuts ? H : fmaf(Pg, G, Hg)));
      } else if (last) {
        st_word(p.group_agg + g * p.dim + ch, step_word(0.f, cuts ? H : Hg));
        st_word(p.ends + g * p.dim + ch, published(cuts ? H : Hg));
      }
    } else if (last) {
      st_word(p.group_agg + g * p.dim + ch, step_word(0.f, H));
      st_word(p.ends + g * p.dim + ch, published(H));
    }
    before_runs<FORWARD>(sh.P, sh.H, cuts, X);
    return X;
  }
  // H of each run becomes the state before it.
  template <bool ORDER>
  __device__ __forceinline__ void before_runs(const float (&P)[kWarps][32 * V], float (&H)[kWarps][32 * V],
                                              uint64_t cuts, float S) const {
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      const int r = ORDER ? q : kWarps - 1 - q;
      const float Hr = H[r][c];
      H[r][c] = S;
      S = cuts >> (8 * r) & 1 ? Hr : fmaf(P[r][c], S, Hr);
    }
  }
};

// ---------------------------------------------------------------- forward --
// TMA: rows come by tensor maps, one copy per run and array (16-byte aligned rows); else each
// lane copies its own.  A warp asks for the next tile's rows as soon as it has read this one's.
struct LinrecMaps {
  CUtensorMap x, r, i, z;
};
template <int V>
constexpr int kFwdBlocks = V == 1 ? 3 : 2;  // per SM, by the registers of a lane's channels
template <typename T, int V, bool OUT, bool TMA>
__global__ void __launch_bounds__(32 * kWarps, kFwdBlocks<V>)
    linrec_fwd_kernel(const __grid_constant__ LinrecParams p, const __grid_constant__ LinrecMaps maps) {
  constexpr int R = kRowsF, CH = 32 * V;
  using S = Slots<T, V, R>;
  extern __shared__ __align__(128) uint8_t slots[];  // x, r, i, z
  __shared__ __align__(16) BlockShared<V, kTileF> sh;
  __shared__ uint64_t full[2][kWarps];               // x, r, i are there; z is
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (TMA && threadIdx.x < 2 * kWarps) {
    ptx::mbar_init(&full[0][threadIdx.x], 1);
    ptx::fence_mbar_init();
  }
  start_block<true, TMA || V == 2>(p, sh, warp, lane);
  uint8_t* const run = slots + warp * S::kRun;
  const uint8_t* const mine = run + lane * S::kBytes;
  auto place = [&](const Unit& u, int64_t& row0, int& ch) {  // the rows that exist
    row0 = (int64_t)u.tile * kTileF + warp * R;
    ch = u.block * CH + lane * V;
    return ch < p.dim && u.tile >= 0 ? (int)max((int64_t)0, min((int64_t)R, p.total - row0)) : 0;
  };
  auto copy = [&](const Unit& u) {
    if constexpr (TMA) {
      if (u.tile >= 0 && lane == 0) {
        const int row0 = u.tile * kTileF + warp * R, c0 = u.block * CH;
        ptx::mbar_arrive_expect_tx(&full[0][warp], 3 * S::kRun);
        ptx::tma_load_2d(run, &maps.x, &full[0][warp], c0, row0);
        ptx::tma_load_2d(run + S::kArray, &maps.r, &full[0][warp], c0, row0);
        ptx::tma_load_2d(run + 2 * S::kArray, &maps.i, &full[0][warp], c0, row0);
      }
    } else {
      if (u.tile >= 0) {
        int64_t row0;
        int ch;
        const int n = place(u, row0, ch);
        const uint32_t at = ptx::smem_u32(mine);
        S::copy(at, p.x, row0, p.x_s, ch, n);
        S::copy(at + S::kArray, p.r, row0, p.r_s, ch, n);
        S::copy(at + 2 * S::kArray, p.i, row0, p.i_s, ch, n);
      }
      ptx::cp_async_commit();
    }
  };
  auto copy_z = [&](const Unit& u) {
    const bool want = OUT && p.z && u.tile >= 0;
    if constexpr (TMA) {
      if (want && lane == 0) {
        ptx::mbar_arrive_expect_tx(&full[1][warp], S::kRun);
        ptx::tma_load_2d(run + 3 * S::kArray, &maps.z, &full[1][warp], u.block * CH, u.tile * kTileF + warp * R);
      }
    } else {
      if (want) {
        int64_t row0;
        int ch;
        const int n = place(u, row0, ch);
        S::copy(ptx::smem_u32(mine) + 3 * S::kArray, p.z, row0, p.z_s, ch, n);
      }
      ptx::cp_async_commit();
    }
  };
  auto arrived = [&](int which, unsigned turn) {
    if constexpr (TMA) {
      if (!ptx::mbar_wait(&full[which][warp], turn & 1, kWaitNs)) atomicOr(p.status, kDevStatusTimeout);
    } else {
      ptx::cp_async_wait<1>();
    }
  };
  copy(sh.unit[0]);
  copy_z(sh.unit[0]);
  for (unsigned turn = 0;; ++turn) {
    const Unit unit = sh.unit[turn & 1];
    if (unit.tile < 0) break;
    const int64_t s = unit.tile;
    const int c0 = unit.block * CH;
    int64_t row0;
    int ch;
    const bool ok = place(unit, row0, ch) > 0;
    unsigned ticket = 0;
    if (threadIdx.x == 32 * kWarps - 32) ticket = atomicAdd(p.ticket, 1u);
    const auto& rows = sh.rows[turn & 1];
    const RowBits bits = run_rows(rows, warp);
    Gates<V> c = {};
    if (ch < p.dim) read_gates(c, p, ch);
    arrived(0, turn);
    Vals<V> a[R], b[R];
    steps_of<T>([&](int k, int j) { return S::get(mine + k * S::kArray, j); }, c, a, b);
    if (bits.start && p.init) {  // a sequence's first step starts from its initial state
      constexpr int kAhead = 4;  // loads on their way at once (256 single tokens 18.7 to 16.9 us)
#pragma unroll
      for (int j = 0; j < R; j += kAhead) {
        float h0[kAhead][V] = {};
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (ok && (bits.start >> (j + k) & 1))
            load_state<V>(h0[k], p.init, (int64_t)rows.n[warp * R + j + k] * p.dim + ch, p.state_bf16);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (bits.start >> (j + k) & 1) b[j + k] = fma_of(a[j + k], vals_from(h0[k]), b[j + k]);
      }
    }
    // what the run does to a state
    Vals<V> P = a[0], h = b[0];
    if (!bits.start) {
#pragma unroll
      for (int j = 1; j < R; ++j) h = fma_of(a[j], h, b[j]), P = mul_of(P, a[j]);
    } else {
#pragma unroll
      for (int j = 1; j < R; ++j) h = bits.start >> j & 1 ? b[j] : fma_of(a[j], h, b[j]);
    }
    put<V>(sh.runs.P[warp], lane, P);
    put<V>(sh.runs.H[warp], lane, h);
    if (lane == 0) sh.runs.cut[warp] = bits.start != 0;
    if (threadIdx.x == 32 * kWarps - 32) sh.unit[(turn + 1) & 1] = unit_of(p, ticket);
    const int64_t edge = rows.bos / kTileF;
    Join<V, true> join(p, s, edge, (rows.live[0] & 1) && !(rows.start[0] & 1) && s > 0, c0);
    __syncthreads();
    const Unit next = sh.unit[(turn + 1) & 1];
    copy(next);
    float Pt, Ht;
    join.parts(sh.runs, Pt, Ht);
    __syncthreads();
    if (join.part == 0 && join.ok) {
      const float X = join.finish(sh.runs, edge, Pt, Ht);
      if (p.states) {  // before the tile's first row, and before its second half
        p.states[2 * s * p.dim + join.ch] = X;
        if ((2 * s + 1) * KDA_LINREC_CHUNK < p.total)
          p.states[(2 * s + 1) * p.dim + join.ch] = sh.runs.H[kWarps / 2][join.c];
      }
    }
    if (warp == kWarps - 1 && next.tile >= 0)  // meanwhile: the next turn's rows
      find_rows<TMA || V == 2>(sh.rows[(turn + 1) & 1], p, (int64_t)next.tile * kTileF, lane);
    __syncthreads();
    if constexpr (OUT) {
      if (p.z) arrived(1, turn);
      h = get<V>(sh.runs.H[warp], lane);
      char* const to = reinterpret_cast<char*>(static_cast<T*>(p.out) + row0 * p.dim + ch);
      auto put_row = [&](int j) {
        float y[V];
        if (p.z) vals_to(mul_of(h, silu_of<T>(S::get(mine + 3 * S::kArray, j))), y);
        else vals_to(h, y);
        store_vals<T, V>(to + (uint64_t)(uint32_t)p.dim * (uint32_t)(j * sizeof(T)), 0, y);
      };
      if (!ok) {
      } else if (!bits.start && !bits.last && bits.live == (1u << R) - 1) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
          h = fma_of(a[j], h, b[j]);
          put_row(j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < R; ++j) {
          h = bits.start >> j & 1 ? b[j] : fma_of(a[j], h, b[j]);
          if (!(bits.live >> j & 1)) continue;
          put_row(j);
          if (p.fin && (bits.last >> j & 1)) {
            float f[V];
            vals_to(h, f);
            store_state<V>(p.fin, (int64_t)rows.n[warp * R + j] * p.dim + ch, f, p.state_bf16);
          }
        }
      }
      __syncwarp();
    }
    copy_z(next);
  }
  if constexpr (!TMA) ptx::cp_async_wait_all();
}

// V states at once, which lie on V times their size.
template <int V>
__device__ __forceinline__ void load_states(float (&h)[V], const void* p, int64_t at, bool b16) {
  if constexpr (V == 1) {
    load_state<1>(h, p, at, b16);
  } else if (b16) {
    Raw<bf16, V> r;
    load_words<true>(r.w, static_cast<const bf16*>(p) + at);
    unpack(r, h);
  } else {
    Raw<float, V> r;
    load_words<true>(r.w, static_cast<const float*>(p) + at);
    unpack(r, h);
  }
}
template <int V>
__device__ __forceinline__ void store_states(void* p, int64_t at, const float (&h)[V], bool b16) {
  if (b16) store_row<bf16, V, (V > 1)>(static_cast<bf16*>(p) + at, h, 1, 1);
  else store_row<float, V, (V > 1)>(static_cast<float*>(p) + at, h, 1, 1);
}

// Single tokens and prompts of a few: a thread takes four channels of one sequence, or as
// many as their alignment allows.
template <typename T, int V>
__global__ void __launch_bounds__(256) linrec_step_kernel(LinrecParams p) {
  const unsigned per = (unsigned)p.dim / V;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = p.units ? (unsigned)at / per : at / per;  // (units: 32 bits are enough)
  const int ch = (int)(at - n * per) * V;
  if (n >= p.N) return;
  float h0[V] = {};
  if (p.init) load_states<V>(h0, p.init, n * p.dim + ch, p.state_bf16);
  Gates<V> c;
  load_gates<T>(c, p, ch, true);
  Vals<V> h = vals_from(h0);
  for (int64_t t = n * p.T; t < (n + 1) * p.T; ++t) {
    Raw<T, V> rx, rr, ri, rz = {};
    load_vals<T, V>(rx, p.x, t * p.x_s + ch);
    load_vals<T, V>(rr, p.r, t * p.r_s + ch);
    load_vals<T, V>(ri, p.i, t * p.i_s + ch);
    if (p.z) load_vals<T, V>(rz, p.z, t * p.z_s + ch);
    const Vals<V> x2[2] = {vals_of(rx), {}}, r2[2] = {vals_of(rr), {}}, i2[2] = {vals_of(ri), {}};
    Vals<V> a, b, none, none2;
    step_of<T>(x2, r2, i2, c, a, b, none, none2);
    h = fma_of(a, h, b);
    vals_to(p.z ? mul_of(h, silu_of<T>(vals_of(rz))) : h, h0);
    store_vals<T, V>(p.out, t * p.dim + ch, h0);
  }
  vals_to(h, h0);
  if (p.fin) store_states<V>(p.fin, n * p.dim + ch, h0, p.state_bf16);
}

// --------------------------------------------------------------- backward --
// The gradients of a pair of values: g of the state, a its decay, h the state before.  On
// return g holds a g, what goes on to the row before.  1 - sigmoid(v) = exp(-v) sigmoid(v) keeps its
// digits on both sides; in that product an infinite exponential, whose sigmoid is 0, becomes a finite
// one (2^115: times 4096 still is).  The sigmoids take the exponentials as they are, so that a
// gate that is no number makes gradients that are none, and one far out the forward's decay.
__device__ __forceinline__ pair at_most(pair v, float top) {
  return pr(fminf(un(v).x, top), fminf(un(v).y, top));
}
template <typename T>
__device__ __forceinline__ void grads_of(pair x, pair r, pair i, pair A2, pair cr, pair ci, pair a, pair h,
                                         pair& g, pair& e, pair& dx, pair& dr, pair& di) {
  const pair er = gate_exp<T>(r, cr), ei = gate_exp<T>(i, ci);
  const pair R = rcp_of(padd(er, pr(1.f)));
  const pair I = rcp_of(pfma(ei, pr(4096.f), pr(4096.f)));  // by 2^-12, as m is by 2^12
  const pair L2 = pmul(A2, R);
  const pair m2 = scaled_m2(L2, a), rsm = rsqrt_of(m2);     // 2^-12 / m
  dx = pmul(pmul(g, pmul(m2, rsm)), I);
  di = pmul(pmul(dx, x), pmul(pmul(at_most(ei, 0x1p115f), pr(4096.f)), I));
  g = pmul(g, a);
  // g L2 and L2 / m before what could leave the range for an infinite rate
  const pair in = pmul(pmul(a, pmul(pmul(L2, rsm), I)), x);  // by 2^-24
  e = pfma(pmul(g, in), pr(-kLn2 * 0x1p24f), pmul(pmul(pmul(g, L2), h), pr(kLn2)));
  dr = pmul(e, pmul(at_most(er, FLT_MAX), R));
}
// Of two rows; g: of each one's state.
template <typename T, int V>
__device__ __forceinline__ void grads_of(const Vals<V> (&x)[2], const Vals<V> (&r)[2], const Vals<V> (&i)[2],
                                         const Gates<V>& c, const Vals<V> (&a)[2], const Vals<V> (&h)[2],
                                         const Vals<V> (&g)[2], Vals<V> (&e)[2], Vals<V> (&dx)[2], Vals<V> (&dr)[2],
                                         Vals<V> (&di)[2]) {
  if constexpr (V == 1) {
    pair pg = two(g[0], g[1]), pe, px, pq, pi;
    grads_of<T>(two(x[0], x[1]), two(r[0], r[1]), two(i[0], i[1]), pr(c.A2.v[0]), pr(c.cr.v[0]), pr(c.ci.v[0]),
                two(a[0], a[1]), two(h[0], h[1]), pg, pe, px, pq, pi);
    apart(pe, e[0], e[1]), apart(px, dx[0], dx[1]), apart(pq, dr[0], dr[1]), apart(pi, di[0], di[1]);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        pair pg = g[q].v[k];
        grads_of<T>(x[q].v[k], r[q].v[k], i[q].v[k], c.A2.v[k], c.cr.v[k], c.ci.v[k], a[q].v[k], h[q].v[k], pg,
                    e[q].v[k], dx[q].v[k], dr[q].v[k], di[q].v[k]);
      }
  }
}
template <int V>
__device__ __forceinline__ Vals<V> add_of(const Vals<V>& a, const Vals<V>& b) {
  Vals<V> r;
  if constexpr (V == 1) {
    r.v[0] = a.v[0] + b.v[0];
  } else {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) r.v[k] = padd(a.v[k], b.v[k]);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_of(void* p, int64_t at, const Vals<V>& v) {
  float f[V];
  vals_to(v, f);
  store_vals<T, V>(p, at, f);
}

template <typename T, int V, bool Z>
__global__ void __launch_bounds__(32 * kWarps, 2) linrec_bwd_kernel(const __grid_constant__ LinrecParams p) {
  constexpr int R = kRowsB, CH = 32 * V;
  using S = Slots<T, V, R>;
  constexpr int kBuffer = 5 * S::kArray + S::kGates;  // x, r, i, dout, z, gates; two by turns
  extern __shared__ __align__(128) uint8_t slots[];
  __shared__ __align__(16) BlockShared<V, kTileB> sh;         // runs of the gradients, last run first
  __shared__ __align__(16) float fw_H[kWarps][CH];    // of the states; the products are the same
  __shared__ __align__(8) unsigned char fw_cut[kWarps];
  __shared__ __align__(16) float sums[3][kWarps][CH];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  start_block<false, true>(p, sh, warp, lane);
  const uint8_t* const mine0 = slots + warp * S::kRun + lane * S::kBytes;
  const uint32_t at0 = ptx::smem_u32(mine0), at_gates0 = ptx::smem_u32(slots + 5 * S::kArray + threadIdx.x * V * 4);
  auto place = [&](const Unit& u, int64_t& row0, int& ch) {  // the rows that exist
    row0 = (p.tiles - 1 - u.tile) * kTileB + warp * R;
    ch = u.block * CH + lane * V;
    return ch < p.dim ? (int)max((int64_t)0, min((int64_t)R, p.total - row0)) : 0;
  };
  auto copy = [&](const Unit& u, unsigned turn) {
    if (u.tile >= 0) {
      int64_t row0;
      int ch;
      const int n = place(u, row0, ch);
      const uint32_t at = at0 + (turn & 1) * kBuffer;
      S::copy(at, p.x, row0, p.x_s, ch, n);
      S::copy(at + S::kArray, p.r, row0, p.r_s, ch, n);
      S::copy(at + 2 * S::kArray, p.i, row0, p.i_s, ch, n);
      S::copy(at + 3 * S::kArray, p.dout, row0, p.dim, ch, n);
      if constexpr (Z) S::copy(at + 4 * S::kArray, p.z, row0, p.z_s, ch, n);
      S::copy_gates(at_gates0 + (turn & 1) * kBuffer, p.gates, p.dim, ch, ch < p.dim);
    }
    ptx::cp_async_commit();
  };
  // the sums over a tile's rows, by a warp that has nothing else to do in the turn after
  int64_t last_tile = -1;
  int last_c0 = 0;
  auto add_runs = [&](int64_t tile, int c0) {
    for (int q = lane; q < 3 * CH; q += 32) {
      const int w = q / CH, k = q % CH;
      float v = 0.f;
#pragma unroll
      for (int e = 0; e < kWarps; ++e) v += sums[w][e][k];
      if (c0 + k < p.dim) p.part[(tile * 3 + w) * p.dim + c0 + k] = v;
    }
  };
  copy(sh.unit[0], 0);
  for (unsigned turn = 0;; ++turn) {
    const Unit unit = sh.unit[turn & 1];
    if (unit.tile < 0) break;
    const int64_t s = unit.tile, tile = p.tiles - 1 - s;  // s: counted from the last tile back
    const int c0 = unit.block * CH;
    unsigned ticket = 0;
    if (threadIdx.x == 32 * kWarps - 32) ticket = atomicAdd(p.ticket, 1u);
    int64_t row0;
    int ch;
    const int n = place(unit, row0, ch);
    const bool ok = n > 0;
    const auto& rows = sh.rows[turn & 1];
    const RowBits bits = run_rows(rows, warp);
    const uint8_t* const mine = mine0 + (turn & 1) * kBuffer;
    ptx::cp_async_wait_all();
    Gates<V> c;
    S::gates(c, slots + 5 * S::kArray + threadIdx.x * V * 4 + (turn & 1) * kBuffer);
    Vals<V> a[R], b[R], dy[R], dq[R];  // dq: dout silu'(z), what dz takes times h
    Vals<V> h, P;
    auto initial = [&](int j) {
      float h0[V] = {};
      if (p.init && ok) load_state<V>(h0, p.init, (int64_t)rows.n[warp * R + j] * p.dim + ch, p.state_bf16);
      return vals_from(h0);
    };
    // A run within one sequence asks nothing row by row (`inner`).
    const bool within = __all_sync(0xffffffffu, n == R) && !bits.start && !bits.last && bits.live == (1u << R) - 1;
    auto row = [&](auto inner, int k, int j) {  // rows of no sequence count for nothing
      constexpr bool IN = decltype(inner)::value;
      return IN || (bits.live >> j & 1) ? S::get(mine + k * S::kArray, j) : splat<V>(0.f);
    };
    // what the run does to a state, and to a gradient
    auto compose = [&](auto inner) {
      constexpr bool IN = decltype(inner)::value;
      steps_of<T>([&](int k, int j) { return row(inner, k, j); }, c, a, b);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        dy[j] = row(inner, 3, j);
        if constexpr (Z) {
          const Vals<V> z = row(inner, 4, j), q = sigmoid<T>(z), zq = mul_of(z, q);
          // silu' = q + z q (1 - q)
          dq[j] = mul_of(dy[j], fma_of(zq, fma_of(q, splat<V>(-1.f), splat<V>(1.f)), q));
          dy[j] = mul_of(dy[j], zq);
        }
      }
      if constexpr (IN) {
        h = b[0], P = a[0];
#pragma unroll
        for (int j = 1; j < R; ++j) h = fma_of(a[j], h, b[j]), P = mul_of(P, a[j]);
        put<V>(fw_H[warp], lane, h);
        h = mul_of(a[R - 1], dy[R - 1]);
#pragma unroll
        for (int j = R - 2; j >= 0; --j) h = mul_of(a[j], add_of(h, dy[j]));
      } else {
        h = splat<V>(0.f), P = splat<V>(1.f);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          if (bits.start >> j & 1) h = initial(j);
          h = fma_of(a[j], h, b[j]);
          P = mul_of(P, a[j]);
        }
        put<V>(fw_H[warp], lane, h);
#pragma unroll
        for (int j = 0; j < R; ++j)
          if (p.dfin && ok && (bits.last >> j & 1)) {  // the final state's gradient joins the last row's
            float d[V];
            load_state<V>(d, p.dfin, (int64_t)rows.n[warp * R + j] * p.dim + ch, p.state_bf16);
            dy[j] = add_of(dy[j], vals_from(d));
          }
        h = splat<V>(0.f);
#pragma unroll
        for (int j = R - 1; j >= 0; --j) h = mul_of(a[j], bits.last >> j & 1 ? dy[j] : add_of(h, dy[j]));
      }
    };
    if (within) compose(std::true_type{});
    else compose(std::false_type{});
    put<V>(sh.runs.P[warp], lane, P);
    put<V>(sh.runs.H[warp], lane, h);
    if (lane == 0) sh.runs.cut[warp] = bits.last != 0, fw_cut[warp] = bits.start != 0;
    if (threadIdx.x == 32 * kWarps - 32) sh.unit[(turn + 1) & 1] = unit_of(p, ticket);
    const int64_t edge = p.tiles - 1 - (rows.eos - 1) / kTileB;
    Join<V, false> join(p, s, edge, (rows.live[1] >> 31) && !(rows.last[1] >> 31) && s > 0, c0);
    __syncthreads();
    float Pt, Ht;
    join.parts(sh.runs, Pt, Ht);
    __syncthreads();
    if (join.part == 0) {
      if (join.ok) join.finish(sh.runs, edge, Pt, Ht);
    } else if (join.part == 1) {
      if (join.ok)
        join.template before_runs<true>(sh.runs.P, fw_H, *reinterpret_cast<const uint64_t*>(fw_cut),
                                        p.states[tile * p.dim + join.ch]);
    } else if (warp == kWarps - 1) {  // meanwhile: the next turn's rows
      const Unit next = sh.unit[(turn + 1) & 1];
      if (next.tile >= 0) find_rows<true>(sh.rows[(turn + 1) & 1], p, (p.tiles - 1 - next.tile) * kTileB, lane);
    }
    if (warp == kWarps - 2 && turn > 0) add_runs(last_tile, last_c0);
    __syncthreads();
    copy(sh.unit[(turn + 1) & 1], turn + 1);
    // states again, b <- the one before each row; dz; then the rows' gradients, last row first
    Vals<V> se = splat<V>(0.f), sr = se, si = se;
    const int64_t row_at = row0 * p.dim + ch;
    auto walk = [&](auto inner) {
      constexpr bool IN = decltype(inner)::value;
      auto at = [&](void* q, int j) {
        return reinterpret_cast<char*>(static_cast<T*>(q) + row_at) + (uint64_t)(uint32_t)p.dim * (uint32_t)(j * sizeof(T));
      };
      h = get<V>(fw_H[warp], lane);
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (!IN && (bits.start >> j & 1)) h = initial(j);
        const Vals<V> before = h;
        h = fma_of(a[j], h, b[j]);
        b[j] = before;
        if constexpr (Z) {
          if (IN || j < n)
            store_of<T>(at(p.dz, j), 0, IN || (bits.live >> j & 1) ? mul_of(dq[j], h) : splat<V>(0.f));
        }
      }
      Vals<V> C = get<V>(sh.runs.H[warp], lane);
#pragma unroll
      for (int j = R - 2; j >= 0; j -= 2) {
        Vals<V> g[2], e[2], dx[2], dr[2], di[2];
#pragma unroll
        for (int q = 1; q >= 0; --q) {
          g[q] = !IN && (bits.last >> (j + q) & 1) ? dy[j + q] : add_of(C, dy[j + q]);
          C = mul_of(a[j + q], g[q]);
          if (!IN && p.dinit && ok && (bits.start >> (j + q) & 1)) {
            float f[V];
            vals_to(C, f);
            store_state<V>(p.dinit, (int64_t)rows.n[warp * R + j + q] * p.dim + ch, f, false);
          }
        }
        const Vals<V> x[2] = {row(inner, 0, j), row(inner, 0, j + 1)}, r[2] = {row(inner, 1, j), row(inner, 1, j + 1)};
        const Vals<V> i[2] = {row(inner, 2, j), row(inner, 2, j + 1)};
        const Vals<V> a2[2] = {a[j], a[j + 1]}, h2[2] = {b[j], b[j + 1]};
        grads_of<T>(x, r, i, c, a2, h2, g, e, dx, dr, di);
#pragma unroll
        for (int q = 1; q >= 0; --q) {
          if (!IN && !(bits.live >> (j + q) & 1)) e[q] = dx[q] = dr[q] = di[q] = splat<V>(0.f);
          se = add_of(se, e[q]), sr = add_of(sr, dr[q]), si = add_of(si, di[q]);
          if (IN || j + q < n) {
            store_of<T>(at(p.dx, j + q), 0, dx[q]);
            store_of<T>(at(p.dr, j + q), 0, dr[q]);
            store_of<T>(at(p.di, j + q), 0, di[q]);
          }
        }
      }
    };
    if (within) walk(std::true_type{});
    else walk(std::false_type{});
    put<V>(sums[0][warp], lane, se);
    put<V>(sums[1][warp], lane, sr);
    put<V>(sums[2][warp], lane, si);
    last_tile = tile, last_c0 = c0;
  }
  __syncthreads();
  if (warp == kWarps - 2 && last_tile >= 0) add_runs(last_tile, last_c0);
  ptx::cp_async_wait_all();
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
  float* gates;              // [3][dim], written
  const float *A_log, *r_bias, *i_bias;
  float bias_scale;
  const void* src;           // NULL: zeros
  void* dst;                 // NULL: nothing
  int32_t src_bf16, dst_bf16;
};
__global__ void __launch_bounds__(256) linrec_setup_kernel(SetupParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t k = at; k < p.count; k += step) p.words[k] = kUnset;
  if (blockIdx.x == 0) {
    const bool bad = __syncthreads_or(p.cu && bad_seqlens(p.cu, p.N, p.total, threadIdx.x, 256));
    if (threadIdx.x < 32) p.status[threadIdx.x] = threadIdx.x == 0 && bad ? kDevStatusBadSeqlens : 0u;
  }
  for (int64_t d = at; d < p.dim; d += step) {
    p.gates[d] = scan::rate_of(p.A_log[d]);
    p.gates[p.dim + d] = p.r_bias ? p.bias_scale * p.r_bias[d] : 0.f;
    p.gates[2 * (int64_t)p.dim + d] = p.i_bias ? p.bias_scale * p.i_bias[d] : 0.f;
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
size_t join_bytes(int64_t total, int32_t dim, int rows) {  // what tiles publish
  const size_t tiles = (size_t)tiles_of(total, rows);
  return up256(tiles * dim * 8) + up256(tiles / kGroup * dim * 8) + up256(tiles / kGroup * dim * 4);
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

// `lanes`: the channels that a thread can read at a time, 1, 2 or 4, by the rows' alignment;
// `tma`: whether tensor maps can describe them.
kda_status check_linrec(const kda_linrec_problem* q, LinrecParams& p, int& lanes, bool& tma) {
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
  lanes = 4, tma = true;
  while (lanes > 1 && q->dim % lanes) lanes /= 2;
  for (int k = 0; k < 4; ++k) {
    if (!al_to(row[k], e)) return KDA_ERR_MISALIGNED;
    while (lanes > 1 && (!al_to(row[k], lanes * e) || stride[k] % lanes)) lanes /= 2;
    tma = tma && al_to(row[k], 16) && stride[k] * e % 16 == 0;
  }
  if (!al_to(q->A_log, 4) || !al_to(q->r_bias, 4) || !al_to(q->i_bias, 4) ||
      !al_to(q->initial_state, se) || !al_to(q->cu_seqlens, 8))
    return KDA_ERR_MISALIGNED;
  p.x = q->x, p.r = q->r, p.i = q->i, p.z = q->z;
  p.x_s = (uint32_t)q->x_stride, p.r_s = (uint32_t)q->r_stride, p.i_s = (uint32_t)q->i_stride;
  p.z_s = (uint32_t)stride[3];
  p.A_log = q->A_log, p.r_bias = q->r_bias, p.i_bias = q->i_bias;
  p.init = q->initial_state, p.state_bf16 = q->state_dtype == KDA_STATE_BF16;
  p.stall = q->debug_stall;
  return KDA_OK;
}
void lanes_for(int& lanes, const void* p, size_t e) {  // contiguous rows
  while (lanes > 1 && !al_to(p, lanes * e)) lanes /= 2;
}

// Tiles and channel blocks of a pass, and its part of the workspace.
bool plan_pass(LinrecParams& p, int lanes, int rows, uint8_t*& ws) {
  p.tiles = tiles_of(p.total, rows);
  p.blocks = (p.dim + 32 * lanes - 1) / (32 * lanes);
  p.agg = reinterpret_cast<uint64_t*>(ws);
  p.group_agg = reinterpret_cast<uint64_t*>(ws + up256((size_t)p.tiles * p.dim * 8));
  p.ends = reinterpret_cast<unsigned*>(reinterpret_cast<uint8_t*>(p.group_agg) +
                                       up256((size_t)(p.tiles / kGroup) * p.dim * 8));
  ws += join_bytes(p.total, p.dim, rows);
  const bool whole = !p.cu && p.T > 0 && p.T % rows == 0;
  p.units = (unsigned)(p.tiles * p.blocks);
  p.strips = whole ? (unsigned)(p.total / p.T) : 1u;
  p.strip_tiles = whole ? (unsigned)(p.T / rows) : (unsigned)p.tiles;
  return p.tiles * p.blocks < (int64_t(1) << 31);
}

cudaError_t launch_setup(const LinrecParams& p, bool f32, void* words, size_t bytes, const void* src, bool src_bf16,
                         void* dst, bool dst_bf16, cudaStream_t stream) {
  SetupParams s = {};
  s.status = p.status, s.words = static_cast<uint64_t*>(words), s.count = (int64_t)(bytes / 8);
  s.cu = p.cu, s.T = p.T, s.total = p.total, s.N = p.N, s.dim = p.dim;
  s.gates = p.gates, s.A_log = p.A_log, s.r_bias = p.r_bias, s.i_bias = p.i_bias;
  s.bias_scale = f32 ? kBiasScale32 : kBiasScale16;
  s.src = src, s.dst = dst, s.src_bf16 = src_bf16, s.dst_bf16 = dst_bf16;
  const int64_t want = (s.count + 1023) / 1024 + (dst && p.cu ? p.N : 1);
  linrec_setup_kernel<<<(unsigned)(want < 608 ? want : 608), 256, 0, stream>>>(s);
  return cudaGetLastError();
}

// A launch whose blocks may start while the one before it, always one of ours, still runs: they wait
// for its end before they read anything of it (512 tokens of 1,024 channels 9.4 to 8.8 us, 2,048 of 4,096
// 28.9 to 27.9).
template <typename... A>
cudaError_t launch_behind(void (*kernel)(A...), unsigned grid, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid), c.blockDim = dim3(32 * kWarps), c.dynamicSmemBytes = smem, c.stream = stream;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}
template <typename K>
cudaError_t launch_tiles(K kernel, bool (&done)[64], int smem, int blocks, const LinrecParams& p, cudaStream_t stream) {
  int sms = 0;
  if (sm_count(&sms) != KDA_OK) return cudaErrorUnknown;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  return launch_behind(kernel, std::min(p.units, (unsigned)(blocks * sms)), smem, stream, p);
}
template <typename T>
cudaError_t rows_map(CUtensorMap* m, const void* p, const LinrecParams& q, uint32_t stride, int channels) {
  const uint64_t dims[2] = {(uint64_t)q.dim, (uint64_t)q.total}, strides[1] = {(uint64_t)stride * sizeof(T)};
  const uint32_t box[2] = {(uint32_t)channels, (uint32_t)kRowsF};
  return encode_tiled_map(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p,
                          dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}
template <typename T, int V, bool OUT>
cudaError_t launch_fwd_of(const LinrecParams& p, bool tma, cudaStream_t stream) {
  LinrecMaps maps = {};
  const int smem = (p.z && OUT ? 4 : 3) * Slots<T, V, kRowsF>::kArray;
  int sms = 0;
  if (sm_count(&sms) != KDA_OK) return cudaErrorUnknown;
  const unsigned grid = std::min(p.units, (unsigned)(kFwdBlocks<V> * sms));
  cudaError_t e = cudaSuccess;
  if constexpr (V * sizeof(T) == 4) {
    if (tma) {
      static bool done[64];
      e = rows_map<T>(&maps.x, p.x, p, p.x_s, 32 * V);
      if (e == cudaSuccess) e = rows_map<T>(&maps.r, p.r, p, p.r_s, 32 * V);
      if (e == cudaSuccess) e = rows_map<T>(&maps.i, p.i, p, p.i_s, 32 * V);
      if (e == cudaSuccess) e = rows_map<T>(&maps.z, p.z, p, p.z_s, 32 * V);
      auto kernel = linrec_fwd_kernel<T, V, OUT, true>;
      if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), 4 * Slots<T, V, kRowsF>::kArray, done);
      if (e != cudaSuccess) return e;
      return launch_behind(kernel, grid, smem, stream, p, maps);
    }
  }
  static bool done[64];
  auto kernel = linrec_fwd_kernel<T, V, OUT, false>;
  e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), 4 * Slots<T, V, kRowsF>::kArray, done);
  if (e != cudaSuccess) return e;
  return launch_behind(kernel, grid, smem, stream, p, maps);
}
template <typename T, int V>
cudaError_t launch_bwd_of(const LinrecParams& p, cudaStream_t stream) {
  using S = Slots<T, V, kRowsB>;
  constexpr int smem = 2 * (5 * S::kArray + S::kGates);
  static bool done[2][64];
  return p.z ? launch_tiles(linrec_bwd_kernel<T, V, true>, done[1], smem, 2, p, stream)
             : launch_tiles(linrec_bwd_kernel<T, V, false>, done[0], smem, 2, p, stream);
}

// Channels per thread: 4 bytes of a row where its alignment allows.
int lanes_of(int lanes, bool f32) { return f32 ? 1 : std::min(lanes, 2); }
template <bool OUT>
cudaError_t launch_fwd(const LinrecParams& p, bool f32, int lanes, bool tma, cudaStream_t stream) {
  return f32          ? launch_fwd_of<float, 1, OUT>(p, tma, stream)
         : lanes == 2 ? launch_fwd_of<bf16, 2, OUT>(p, tma, stream)
                      : launch_fwd_of<bf16, 1, OUT>(p, tma, stream);
}

size_t states_bytes(int64_t total, int32_t dim) {
  return (size_t)(total / KDA_LINREC_CHUNK + 1) * dim * sizeof(float);
}
size_t gates_bytes(int32_t dim) { return up256((size_t)dim * 3 * sizeof(float)); }
size_t fwd_bytes(const LinrecParams& p) {
  return KDA_STATUS_BYTES + gates_bytes(p.dim) + join_bytes(p.total, p.dim, kTileF);
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
  *bytes = KDA_STATUS_BYTES + gates_bytes(p.dim) + join_bytes(p.total, p.dim, kTileB) +
           up256((size_t)tiles * 3 * p.dim * sizeof(float));
  if (!have_states)
    *bytes += join_bytes(p.total, p.dim, kTileF) + up256(states_bytes(p.total, p.dim));
  return KDA_OK;
}

kda_status kda_linrec_fwd(const kda_linrec_problem* problem, void* out, void* final_state,
                          void* chunk_states, size_t chunk_states_bytes, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  LinrecParams p = {};
  int lanes = 1;
  bool tma = false;
  kda_status st = check_linrec(problem, p, lanes, tma);
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
  lanes_for(lanes, out, f32 ? 4 : 2);
  p.out = out, p.fin = final_state, p.states = static_cast<float*>(chunk_states);
  p.status = static_cast<unsigned*>(workspace);
  if (step) {
    if (workspace && cudaMemsetAsync(workspace, 0, 4, stream) != cudaSuccess) return KDA_ERR_CUDA;
    lanes_for(lanes, p.init, p.state_bf16 ? 2 : 4);
    lanes_for(lanes, p.fin, p.state_bf16 ? 2 : 4);
    const int V = lanes == 2 ? 1 : lanes;
    const int64_t threads = (int64_t)p.N * (p.dim / V), blocks = (threads + 255) / 256;
    if (blocks >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
    p.units = threads < (int64_t(1) << 31);
    auto kernel = f32 ? (V == 4 ? linrec_step_kernel<float, 4> : linrec_step_kernel<float, 1>)
                      : (V == 4 ? linrec_step_kernel<bf16, 4> : linrec_step_kernel<bf16, 1>);
    kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES;
  p.gates = reinterpret_cast<float*>(ws), ws += gates_bytes(p.dim);
  lanes = lanes_of(lanes, f32);
  if (!plan_pass(p, lanes, kTileF, ws)) return KDA_ERR_INVALID_SHAPE;
  p.ticket = p.status + 1;
  cudaError_t e = launch_setup(p, f32, p.agg, join_bytes(p.total, p.dim, kTileF), p.init, p.state_bf16,
                               p.fin == p.init ? nullptr : p.fin, p.state_bf16, stream);
  if (e == cudaSuccess && p.total > 0) e = launch_fwd<true>(p, f32, lanes, tma, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_linrec_bwd(const kda_linrec_problem* problem, const void* dout, const void* dfinal_state,
                          const void* chunk_states, size_t chunk_states_bytes, void* dx, void* dr,
                          void* di, void* dz, float* dA_log, float* dr_bias, float* di_bias,
                          float* dinitial_state, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  using namespace kda;
  LinrecParams p = {};
  int lanes = 1;
  bool tma = false;
  kda_status st = check_linrec(problem, p, lanes, tma);
  if (st != KDA_OK) return st;
  const bool f32 = problem->dtype == KDA_ROW_FP32;
  const size_t e = f32 ? 4 : 2;
  if (!dA_log || !workspace || (p.total > 0 && (!dout || !dx || !dr || !di || (p.z && !dz))))
    return KDA_ERR_NULL_POINTER;
  for (const void* q : {dout, (const void*)dx, (const void*)dr, (const void*)di, (const void*)dz}) {
    if (!al_to(q, e)) return KDA_ERR_MISALIGNED;
    lanes_for(lanes, q, e);
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
  p.gates = reinterpret_cast<float*>(ws), ws += gates_bytes(p.dim);
  uint8_t* const published_at = ws;
  LinrecParams f = p;
  f.stall = 0;
  const int back = lanes_of(lanes, f32);
  bool fits = plan_pass(p, back, kTileB, ws);
  if (!chunk_states) fits = fits && plan_pass(f, lanes_of(lanes, f32), kTileF, ws);
  if (!fits) return KDA_ERR_INVALID_SHAPE;
  const size_t published_bytes = (size_t)(ws - published_at);
  p.part = reinterpret_cast<float*>(ws);
  ws += up256((size_t)p.tiles * 3 * p.dim * sizeof(float));
  p.states = const_cast<float*>(static_cast<const float*>(chunk_states));
  if (!chunk_states) p.states = f.states = reinterpret_cast<float*>(ws);
  p.ticket = p.status + 1, f.ticket = p.status + 2;
  p.dout = dout, p.dfin = dfinal_state;
  p.dx = dx, p.dr = dr, p.di = di, p.dz = dz, p.dinit = dinitial_state;
  cudaError_t err = launch_setup(p, f32, published_at, published_bytes, dfinal_state, p.state_bf16,
                                 dinitial_state, false, stream);
  if (err == cudaSuccess && p.total > 0) {
    if (!chunk_states) err = launch_fwd<false>(f, f32, lanes_of(lanes, f32), tma, stream);
    if (err == cudaSuccess)
      err = f32     ? launch_bwd_of<float, 1>(p, stream)
            : back == 2 ? launch_bwd_of<bf16, 2>(p, stream)
                    : launch_bwd_of<bf16, 1>(p, stream);
  }
  if (err == cudaSuccess)
    err = launch_column_sums(p.part, p.tiles, 3 * (int64_t)p.dim, 3 * (int64_t)p.dim, p.dim, p.dim, dA_log,
                             dr_bias, di_bias, stream);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
