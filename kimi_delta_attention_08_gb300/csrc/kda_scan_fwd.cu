// kda_scan_fwd.cu -- the selective state space scan, forward: prompts, packed prompts and
// single tokens.
//
//   delta = softplus(dt + dt_bias),  h_t = 2^(delta A2) h_{t-1} + (delta x) B_t,
//   y = C_t . h_t + D x,  out = y silu(z),     A2 = -exp(A_log) log2 e
//
// Per (token, channel, state) this takes one exponential and four fp32 operations, against
// 8 bytes of rows per (token, channel) in bf16, so at 16 states it is bound by the FMA and
// special function pipes and the issue of their instructions, not by HBM.  The state never
// leaves the registers: a thread walks all tokens of its sequence (or segment).  Every
// (token, channel)'s softplus is computed once, by the lane that loads its rows, and handed
// to the channel's other lanes; the rows of the next 16 tokens are in flight meanwhile.  The
// dot product over a channel's lanes is reduced for as many tokens at a time as there are
// lanes, so each lane ends up with the tokens that it loaded.
//
// 8 sequences of 4,096 tokens, 4,096 channels, 16 states in bf16 take 783 us (1.4 TB/s; the
// exponentials alone 230 us, those and the packed operations 290; fp32 rows 797 us; 8 states
// 749, 32 states 1,513); one of 65,536 tokens
// and five of 1,024 with 1,024 channels, which has to be cut, 633 us.
//
// Where the channels alone do not fill the GPU, sequences are cut into segments: a first
// pass computes each segment's end state from zero and its sum of delta, a second carries
// the states over the segments (the decay over a segment is 2^(A2 sum delta)), and the
// main pass starts every segment from its state.
#include <cstring>

#include "kda_scan.cuh"

namespace kda {
namespace {

using namespace scan;

enum ScanPass { kOutputs, kStatesOnly, kReverse };

// A thread holds 8 states of two neighbouring channels, as pairs of fp32 values that the
// packed operations take: with everything about 27 instructions per 4 states of a warp's
// channels (4 states a thread, with the rows staged in shared memory: 31 to 35 and 884 us
// for the 784 above; 16 states a thread: 887).  Of U tokens
// loaded together, each of a channel pair's LPC lanes owns OWN: it loads their rows,
// computes their steps, hands those round by shuffles, ends up with their dot products and
// writes their outputs.  Shared memory only carries B and C, each value twice.
template <int NS>
struct FwdShape {
  static constexpr int SP = 8, LPC = NS / SP, NT = 64, CH = 2 * NT / LPC;
  static constexpr int TB = 16;                  // tokens of B and C staged at once
  static constexpr int U = LPC == 8 ? 8 : 4, OWN = U / LPC;
  static constexpr int BV = 2 * TB * NS / NT;    // elements of B and C per thread ...
  static constexpr int BW = BV < 8 ? BV : 8;     // ... in vectors of BW
};

// PASS kOutputs: the main pass.  kStatesOnly: states only (of every block, or the end of a
// segment).  kReverse: the backward's like pass over segments, from their last token to
// their first, of the gradient: g <- 2^(delta A2) (g + dy C) with dy = dout silu(z).
template <typename T, int NS, bool VEC, int PASS>
__global__ void __launch_bounds__(FwdShape<NS>::NT, PASS == kOutputs ? 4 : 5) scan_fwd_kernel(const ScanParams p) {
  constexpr bool OUT = PASS == kOutputs, REV = PASS == kReverse;
  using S = FwdShape<NS>;
  constexpr int SP = S::SP, LPC = S::LPC, NT = S::NT, CH = S::CH, TB = S::TB, U = S::U;
  constexpr int OWN = S::OWN, BW = S::BW, BN = S::BV / BW;
  __shared__ __align__(16) pair s_bc[2][2][TB][NS];  // [buffer][B, C]

  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned tiles = (unsigned)p.tiles;
  const int64_t slot = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x % tiles);
  if (blockIdx.x == 0 && tid < 32 && p.status) {
    if (p.cu) check_seqlens(p.cu, p.N, p.total, p.status, kDevStatusBadSeqlens);
    else if (tid == 0) *p.status = 0u;
  }
  const Segment u = find_unit(p, slot);
  if (!u.live) return;
  const bool prescan = !OUT && p.prescan;
  // the last segment's end starts no segment; nothing before the first asks for its gradient
  if (prescan && (REV ? u.first : u.last)) return;
  const int grp = tile / p.tiles_per_group;
  const int l = lane_part<LPC>(lane);
  // the thread's channels within the group, cg and cg + 1; `left` of them exist
  const int cg = (tile % p.tiles_per_group) * CH + 2 * (tid / 32 * (32 / LPC) + lane_channel<LPC>(lane));
  const int left = min(2, p.per - cg);
  const int64_t ch = (int64_t)grp * p.per + (left > 0 ? cg : 0);
  const int64_t st_at = ch * NS + l * SP;              // state offset within [dim][NS]
  const int64_t st_seq = (int64_t)p.dim * NS;
  auto per_channel = [&](const float* v) {
    return pr(v && left > 0 ? __ldg(v + ch) : 0.f, v && left > 1 ? __ldg(v + ch + 1) : 0.f);
  };
  const pair bias = per_channel(p.dt_bias), skip = per_channel(OUT ? p.D : nullptr);

  pair A2[SP], h[SP];
  {
    float a[2][SP], v[2][SP];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int i = 0; i < SP; ++i) a[q][i] = v[q][i] = 0.f;
      if (q < left) {
        load_rates<SP>(a[q], p.A_log, st_at + q * NS);
        if (REV) {
          if (u.last && p.dfin) load_state<SP>(v[q], p.dfin, u.n * st_seq + st_at + q * NS, p.state_bf16);
        } else if (p.seg_state && !prescan) load_state<SP>(v[q], p.seg_state, slot * st_seq + st_at + q * NS, false);
        else if (u.first && p.init) load_state<SP>(v[q], p.init, u.n * st_seq + st_at + q * NS, p.state_bf16);
      }
    }
#pragma unroll
    for (int i = 0; i < SP; ++i) A2[i] = pr(a[0][i], a[1][i]), h[i] = pr(v[0][i], v[1][i]);
  }
  auto put_state = [&](void* to, int64_t at, bool b16) {
    float v[2][SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) v[0][i] = un(h[i]).x, v[1][i] = un(h[i]).y;
    if (left > 0) store_state<SP>(to, at, v[0], b16);
    if (left > 1) store_state<SP>(to, at + NS, v[1], b16);
  };
  const int tokens = (int)(u.t1 - u.t0);
  pair sum_delta = 0;

  // B and C of a block: vector q * NT + tid of [B, C][TB][NS]
  Raw<T, BW> rbc[BN];
  auto fetch_bc = [&](int t0) {
#pragma unroll
    for (int q = 0; q < BN; ++q) {
      const int e = (q * NT + tid) * BW, m = e / (TB * NS), tok = e / NS % TB, n = e % NS;
      rbc[q] = Raw<T, BW>{};
      if (t0 + tok < tokens && (OUT || m == (REV ? 1 : 0))) {
        const int64_t t = REV ? u.t1 - 1 - t0 - tok : u.t0 + t0 + tok;
        const T* const row = m == 0 ? static_cast<const T*>(p.B) + t * p.b_s
                                    : static_cast<const T*>(p.C) + t * p.c_s;
        load_row<T, BW, VEC>(rbc[q], row + grp * NS + n, 1, BW);
      }
    }
  };
  auto put_bc = [&](int buf) {
#pragma unroll
    for (int q = 0; q < BN; ++q) {
      float v[BW];
      unpack(rbc[q], v);
      float4* const to = reinterpret_cast<float4*>(&s_bc[buf][0][0][0] + (q * NT + tid) * BW);
#pragma unroll
      for (int i = 0; i < BW; i += 2) to[i / 2] = make_float4(v[i], v[i], v[i + 1], v[i + 1]);
    }
  };
  // the rows of the lane's own tokens; one past the end has dt = -infinity, a step of zero
  constexpr int DIR = REV ? -1 : 1;
  const int64_t own0 = REV ? u.t1 - 1 - l * OWN : u.t0 + l * OWN;
  const int64_t x_s = DIR * (REV ? (int64_t)p.dim : p.x_s), t_s = DIR * p.dt_s, z_s = DIR * p.z_s;
  const T* px = static_cast<const T*>(REV ? p.dout : p.x) + own0 * (DIR * x_s) + ch;
  const T* pt = static_cast<const T*>(p.dt) + own0 * p.dt_s + ch;
  const T* pz = static_cast<const T*>(p.z) + own0 * p.z_s + ch;
  T* po = static_cast<T*>(p.out) + (u.t0 + l * OWN) * p.dim + ch;
  constexpr int G = TB / U;  // groups of U tokens in flight: a block's worth
  Raw<T, 2> rx[G][OWN], rt[G][OWN], rz[G][OWN], none;
  const float minus_inf[2] = {-INFINITY, -INFINITY};
  pack(none, minus_inf);
  auto fetch = [&](int g, int t) {
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      rx[g][k] = rz[g][k] = Raw<T, 2>{};
      rt[g][k] = none;
      if (t + l * OWN + k < tokens && left > 0) {
        load_row<T, 2, VEC>(rx[g][k], px + k * x_s, 1, left);
        load_row<T, 2, VEC>(rt[g][k], pt + k * t_s, 1, left);
        if ((OUT || REV) && p.z) load_row<T, 2, VEC>(rz[g][k], pz + k * z_s, 1, left);
      }
    }
    px += U * x_s, pt += U * t_s;
    if ((OUT || REV) && p.z) pz += U * z_s;
  };
  auto as_pair = [](const Raw<T, 2>& r) {
    float f[2];
    unpack(r, f);
    return pr(f[0], f[1]);
  };
  // the lane of these channels that owns token k of U
  auto owner = [&](int k) {
    const int part = k / OWN;
    return LPC == 1 ? lane : (lane & (64 / LPC - 2)) | (part & 1) | (part >> 1) * (64 / LPC);
  };
  float* chunk = p.chunk_states
                     ? p.chunk_states + (u.bos / kScanBlock + u.n + (u.t0 - u.bos) / kScanBlock) * st_seq
                     : nullptr;

  fetch_bc(0);
#pragma unroll
  for (int g = 0; g < G; ++g) fetch(g, g * U);
  put_bc(0);
  __syncthreads();
  for (int t0 = 0, buf = 0; t0 < tokens; t0 += TB, buf ^= 1) {
    fetch_bc(t0 + TB);
    if (chunk && t0 % kScanBlock == 0) {
      put_state(chunk, st_at, false);
      chunk += st_seq;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int j0 = g * U;
      if (t0 + j0 >= tokens) break;
      pair delta[OWN], dx[OWN], xv[OWN], zv[OWN];
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        pair ex;
        xv[k] = as_pair(rx[g][k]);
        if (OUT && p.z) zv[k] = as_pair(rz[g][k]);
        delta[k] = softplus(padd(as_pair(rt[g][k]), bias), ex);
        if (REV) dx[k] = p.z ? pmul(xv[k], silu<T>(as_pair(rz[g][k]))) : xv[k];  // dy
        else dx[k] = pmul(delta[k], xv[k]);
        if (!OUT) sum_delta = padd(sum_delta, delta[k]);
      }
      fetch(g, t0 + TB + j0);
      pair y[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const pair d = LPC == 1 ? delta[k % OWN] : __shfl_sync(0xffffffffu, delta[k % OWN], owner(k));
        const pair m = LPC == 1 ? dx[k % OWN] : __shfl_sync(0xffffffffu, dx[k % OWN], owner(k));
        const pair* const b = &s_bc[buf][REV ? 1 : 0][j0 + k][l * SP];
        const pair* const cc = &s_bc[buf][1][j0 + k][l * SP];
        pair acc[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
          const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(b + i);
          if constexpr (REV) {
            h[i] = pmul(decay(d, A2[i]), pfma(m, b2.x, h[i]));
            h[i + 1] = pmul(decay(d, A2[i + 1]), pfma(m, b2.y, h[i + 1]));
            continue;
          }
          h[i] = advance(h[i], A2[i], d, m, b2.x);
          h[i + 1] = advance(h[i + 1], A2[i + 1], d, m, b2.y);
          if (OUT) {
            const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(cc + i);
            acc[0] = i ? pfma(c2.x, h[i], acc[0]) : pmul(c2.x, h[i]);
            acc[1] = i ? pfma(c2.y, h[i + 1], acc[1]) : pmul(c2.y, h[i + 1]);
          }
        }
        if (OUT) y[k] = padd(acc[0], acc[1]);
      }
      if (!OUT) continue;
      int off = 0;  // l * OWN
      reduce_states<U, LPC>(y, lane, off);
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        y[k] = pfma(skip, xv[k], y[k]);
        if (p.z) y[k] = pmul(y[k], silu<T>(zv[k]));
        const float o[2] = {un(y[k]).x, un(y[k]).y};
        if (t0 + j0 + l * OWN + k < tokens && left > 0)
          store_row<T, 2, VEC>(po + (int64_t)k * p.dim, o, 1, left);
      }
      po += (int64_t)U * p.dim;
    }
    put_bc(buf ^ 1);
    __syncthreads();
  }
  if (prescan) {
    int off = 0;
    if constexpr (LPC > 1) reduce_states<1, LPC>(&sum_delta, lane, off);
    put_state(p.seg_state, slot * st_seq + st_at, false);
    if (l == 0 && left > 0) p.seg_sum[slot * p.dim + ch] = un(sum_delta).x;
    if (l == 0 && left > 1) p.seg_sum[slot * p.dim + ch + 1] = un(sum_delta).y;
  } else if (OUT && u.last && p.fin) {
    put_state(p.fin, u.n * st_seq + st_at, p.state_bf16);
  }
}

// Carries the states over a sequence's segments: in place, the end of segment s (from
// zero; the first from the initial state) becomes the start of segment s.
__global__ void scan_carry_kernel(const ScanParams p, int state) {
  const int64_t st_seq = (int64_t)p.dim * state;
  const int64_t blocks = (st_seq + blockDim.x - 1) / blockDim.x;  // per sequence
  const int n = (int)(blockIdx.x / blocks);
  const int64_t i = (blockIdx.x % blocks) * blockDim.x + threadIdx.x;
  if (i >= st_seq) return;
  int64_t bos, eos;
  seq_bounds(p, n, bos, eos);
  const int64_t ns = (eos - bos + p.seg_len - 1) / p.seg_len, slot = first_slot(p, n);
  const float A2 = rate_of(__ldg(p.A_log + i));
  float h = 0.f;
  if (p.init)
    h = p.state_bf16 ? to_f(static_cast<const bf16*>(p.init)[n * st_seq + i])
                     : static_cast<const float*>(p.init)[n * st_seq + i];
  const int64_t ch = i / state;
  if (ns == 0) p.seg_state[slot * st_seq + i] = h;
  constexpr int kAhead = 8;  // segments whose loads are in flight
  for (int64_t s = 0; s < ns; s += kAhead) {
    float e[kAhead], d[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool ok = s + k + 1 < ns;
      e[k] = ok ? p.seg_state[(slot + s + k) * st_seq + i] : 0.f;
      d[k] = ok ? p.seg_sum[(slot + s + k) * p.dim + ch] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (s + k >= ns) break;
      p.seg_state[(slot + s + k) * st_seq + i] = h;
      h = s + k == 0 ? e[k] : fmaf(exp2f(A2 * d[k]), h, e[k]);
    }
  }
}

// Single tokens and prompts of a few: bound by HBM through the states.  A thread holds 4
// states of a channel (a warp's lie in a row) for kStepSeqs sequences, whose states and rows
// are all in flight at once.  Of these sequences each of a channel's lanes owns OWN: it
// reads their rows, computes their steps, hands those to the others, ends up with their
// dot products and writes their outputs.  256 sequences of 4,096 channels and 16 fp32 states
// take 24.9 us (5.7 TB/s) in blocks of 7 per SM; with 8 it spills (29.2), with 5 too few
// loads are in flight (36).  Before the rates were computed behind the last load it took
// 33.1; with fp32 rows, whose kernels spill 64 bytes, it takes 31.5 us; one thread for all 16 states
// of a channel reads 64 bytes apart (36.8); CTAs that
// stay, with the next states on their way into shared memory, take 32 to 43.
constexpr int kStepSeqs = 4;
constexpr int kStepTokens = 8;  // the longest such prompt

template <typename T, int NS, bool VEC>
__global__ void __launch_bounds__(128, NS == 8 ? 6 : 7) scan_step_kernel(const ScanParams p) {
  constexpr int SP = 4, LPC = NS / SP, OWN = LPC >= 4 ? 1 : 2, OWNERS = kStepSeqs / OWN;
  const int lane = threadIdx.x & 31;
  const unsigned tiles = (unsigned)p.tiles;  // 32-bit divisions: 64-bit ones cost as much as a token
  const unsigned i = blockIdx.x % tiles * blockDim.x + threadIdx.x;
  const int n0 = (int)(blockIdx.x / tiles) * kStepSeqs;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = 0u;
  const bool mine = i / LPC < (unsigned)p.dim;
  const int ch = mine ? (int)(i / LPC) : 0, l = (int)(i % LPC);
  const int grp = p.groups == 1 ? 0 : ch / p.per;
  const int first = l % OWNERS * OWN;  // the sequences it owns
  const int64_t st_at = (int64_t)ch * NS + l * SP, st_seq = (int64_t)p.dim * NS;
  // everything that the first token needs is asked for before anything is waited for
  const int nq = min(kStepSeqs, p.N - n0);  // the others repeat the last one's rows
  float v[kStepSeqs][SP] = {};
  int64_t at = n0 * st_seq + st_at;
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q, at += st_seq)
    if (p.init && q < nq) load_state<SP>(v[q], p.init, at, p.state_bf16);
  const int T_ = (int)p.T;
  const int64_t t0 = (int64_t)n0 * T_;
  const T *px[OWN], *pt[OWN], *pz[OWN];
#pragma unroll
  for (int k = 0; k < OWN; ++k) {
    const int64_t t = t0 + (int64_t)min(first + k, nq - 1) * T_;
    px[k] = static_cast<const T*>(p.x) + t * p.x_s + ch;
    pt[k] = static_cast<const T*>(p.dt) + t * p.dt_s + ch;
    pz[k] = static_cast<const T*>(p.z) + t * p.z_s + ch;
  }
  const T* pb = static_cast<const T*>(p.B) + t0 * p.b_s + grp * NS + l * SP;
  const T* pc = static_cast<const T*>(p.C) + t0 * p.c_s + grp * NS + l * SP;
  const int64_t b_step = T_ * p.b_s, c_step = T_ * p.c_s;
  Raw<T, 1> rx[OWN], rt[OWN], rz[OWN];
  Raw<T, SP> rb[kStepSeqs], rc[kStepSeqs];
  auto rows = [&] {  // of the next token
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      load_row<T, 1, false>(rx[k], px[k], 1, 1);
      load_row<T, 1, false>(rt[k], pt[k], 1, 1);
      rz[k] = Raw<T, 1>{};
      if (p.z) load_row<T, 1, false>(rz[k], pz[k], 1, 1);
      px[k] += p.x_s, pt[k] += p.dt_s, pz[k] += p.z_s;
    }
    const T *qb = pb, *qc = pc;
#pragma unroll
    for (int q = 0; q < kStepSeqs; ++q) {
      load_row<T, SP, VEC>(rb[q], qb, 1, SP);
      load_row<T, SP, VEC>(rc[q], qc, 1, SP);
      if (q + 1 < nq) qb += b_step, qc += c_step;
    }
    pb += p.b_s, pc += p.c_s;
  };
  rows();
  float log_a[SP];
#pragma unroll
  for (int i = 0; i < SP; ++i) log_a[i] = __ldg(p.A_log + st_at + i);
  const float bias = p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f, D = p.D ? __ldg(p.D + ch) : 0.f;
  pair h[kStepSeqs][2];
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q) h[q][0] = pr(v[q][0], v[q][1]), h[q][1] = pr(v[q][2], v[q][3]);
  const pair A2[2] = {pr(rate_of(log_a[0]), rate_of(log_a[1])), pr(rate_of(log_a[2]), rate_of(log_a[3]))};
  T* po = static_cast<T*>(p.out) + (t0 + (int64_t)first * T_) * p.dim + ch;
  for (int j = 0;; ++j) {
    float x[OWN], z[OWN], delta[OWN], dx[OWN];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      float f[1], ex;
      unpack(rx[k], f);
      x[k] = f[0];
      unpack(rz[k], f);
      z[k] = f[0];
      unpack(rt[k], f);
      delta[k] = softplus(f[0] + bias, ex);
      dx[k] = delta[k] * x[k];
    }
    float y[kStepSeqs];
#pragma unroll
    for (int q = 0; q < kStepSeqs; ++q) {
      const int from = (lane & ~(OWNERS - 1)) | q / OWN;
      const pair d = pr(__shfl_sync(0xffffffffu, delta[q % OWN], from));
      const pair m = pr(__shfl_sync(0xffffffffu, dx[q % OWN], from));
      float b[SP], c[SP];
      unpack(rb[q], b);
      unpack(rc[q], c);
      h[q][0] = advance(h[q][0], A2[0], d, m, pr(b[0], b[1]));
      h[q][1] = advance(h[q][1], A2[1], d, m, pr(b[2], b[3]));
      const float2 s = un(pfma(pr(c[2], c[3]), h[q][1], pmul(pr(c[0], c[1]), h[q][0])));
      y[q] = s.x + s.y;
    }
    int off = 0;  // first
    reduce_scatter<kStepSeqs, OWNERS / 2, 1>(y, lane, off);
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
#pragma unroll
      for (int o = OWNERS; o < LPC; o <<= 1) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
      y[k] = fmaf(D, x[k], y[k]);
      if (p.z) y[k] *= z[k] * sigmoid<T>(z[k]);
      if (mine && l < OWNERS && first + k < nq) po[(int64_t)(k * T_ + j) * p.dim] = from_f<T>(y[k]);
    }
    if (j + 1 >= T_) break;
    rows();
  }
  if (!p.fin || !mine) return;
  at = n0 * st_seq + st_at;
#pragma unroll
  for (int q = 0; q < kStepSeqs; ++q, at += st_seq) {
    const float f[SP] = {un(h[q][0]).x, un(h[q][0]).y, un(h[q][1]).x, un(h[q][1]).y};
    if (q < nq) store_state<SP>(p.fin, at, f, p.state_bf16);
  }
}

template <typename T, bool VEC, int PASS>
cudaError_t launch_main(const ScanParams& p, int state, cudaStream_t stream) {
  const int64_t grid = p.slots * p.tiles;
  if (grid == 0) return cudaSuccess;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)grid;
  constexpr int NT = FwdShape<16>::NT;
  switch (state) {
    case 8: scan_fwd_kernel<T, 8, VEC, PASS><<<g, NT, 0, stream>>>(p); break;
    case 16: scan_fwd_kernel<T, 16, VEC, PASS><<<g, NT, 0, stream>>>(p); break;
    case 32: scan_fwd_kernel<T, 32, VEC, PASS><<<g, NT, 0, stream>>>(p); break;
    default: scan_fwd_kernel<T, 64, VEC, PASS><<<g, NT, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

template <int PASS>
cudaError_t launch_pass(const ScanParams& p, int state, bool f32, bool vec, cudaStream_t stream) {
  if (f32) return vec ? launch_main<float, true, PASS>(p, state, stream)
                      : launch_main<float, false, PASS>(p, state, stream);
  return vec ? launch_main<bf16, true, PASS>(p, state, stream)
             : launch_main<bf16, false, PASS>(p, state, stream);
}

template <typename T, bool VEC>
cudaError_t launch_step(ScanParams p, int state, cudaStream_t stream) {
  p.tiles = ((int64_t)p.dim * (state / 4) + 127) / 128;
  const int64_t grid = p.tiles * (((int64_t)p.N + kStepSeqs - 1) / kStepSeqs);
  if (grid == 0) return cudaSuccess;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)grid;
  switch (state) {
    case 8: scan_step_kernel<T, 8, VEC><<<g, 128, 0, stream>>>(p); break;
    case 16: scan_step_kernel<T, 16, VEC><<<g, 128, 0, stream>>>(p); break;
    case 32: scan_step_kernel<T, 32, VEC><<<g, 128, 0, stream>>>(p); break;
    default: scan_step_kernel<T, 64, VEC><<<g, 128, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

namespace scan {

// A unit is one CTA's walk over one segment; an SM holds `resident` of them at a time.  Units
// are as long as one another, so they run in turns over the GPU, and sequences are cut so
// that they nearly fill a whole number of turns, with segments of 128 tokens at least.
// (Training at 4 sequences of 4,096 tokens, 4,096 channels, 256 units if whole: cut into 7
// pieces, 3.9 turns of the backward, it takes 1.70 ms; into 4, which take a third turn for
// the last eighth, 1.96 ms.)
constexpr int64_t kMinSegment = 128;

int64_t scan_whole_units(const ScanParams& p, int64_t tiles) { return p.cu ? tiles : tiles * p.N; }

ScanPlan scan_plan(const ScanParams& p, int64_t tiles, int64_t resident, bool cut) {
  const bool packed = p.cu != nullptr;
  const int64_t N = p.N, T = p.T, total = p.total;
  ScanPlan r = {0, N};
  if (!cut || total == 0) return r;
  const int64_t whole = scan_whole_units(p, tiles), turn = kSms * resident;
  const int64_t turns_whole = (whole + turn - 1) / turn;
  int64_t pieces = 0;
  double best = 0.0;
  for (int64_t turns = turns_whole + 2; turns <= turns_whole + 7 && best < 0.95; ++turns) {
    const int64_t room = turn * turns, n = room / whole;
    const double fill = (double)(n * whole) / (double)room;
    if (fill > best) best = fill, pieces = n;
  }
  const int64_t span = packed ? total : T;
  int64_t len = (span + pieces - 1) / pieces;
  len = (len + kScanBlock - 1) / kScanBlock * kScanBlock;
  if (len < kMinSegment) len = kMinSegment;
  if (!packed && len >= T) return r;
  r.seg_len = len;
  r.slots = total / len + N;
  return r;
}

// Counted with 4 CTAs of two warps on an SM; with 16 and more states 5 fit in bf16, but segments
// for 5 take as long (2 sequences of 4,096 tokens and channels, 16 states, 323 / 317 us, 5 735 /
// 740).  Cutting costs half the main pass once more, while a GPU with half of that room taken
// still runs at 7 tenths of its rate, so sequences stay whole from a part of the room on: 6
// tenths with 8 states, whose CTA is the slowest alone, 4 with 16 and 32, 3 with 64, whose first
// pass is as long as the main one.  Sequences of 4,096 tokens and channels, whole / cut: 8
// states, 9 (47 %) 924 / 857 us, 11 (58 %) 1,051 / 974, 12 (63 %) 1,052 / 1,092; 16 states, 3
// (32 %) 568 / 468, 4 (42 %) 572 / 598; 32 states, 1 (21 %) 517 / 317, 2 (42 %) 535 / 579; 64
// states, 1 of 2,048 channels (21 %) 443 / 411, 1 of 3,200 (33 %) 557 / 606.
void scan_fwd_plan(ScanParams& p, int state) {
  const int ch = 1024 / state;  // FwdShape::CH
  p.tiles_per_group = (p.per + ch - 1) / ch;
  p.tiles = (int64_t)p.tiles_per_group * p.groups;
  const int64_t tenths = state == 8 ? 6 : state == 64 ? 3 : 4;
  const ScanPlan r = scan_plan(p, p.tiles, 4, 10 * scan_whole_units(p, p.tiles) < tenths * 4 * kSms);
  p.seg_len = r.seg_len, p.slots = r.slots;
}

size_t fwd_ws_bytes(const ScanParams& p, int state) {
  return p.seg_len ? (size_t)p.slots * p.dim * (state + 1) * sizeof(float) : 0;
}

void carve_fwd(ScanParams& p, int state, void* ws) {
  p.seg_state = static_cast<float*>(ws);
  p.seg_sum = p.seg_state + p.slots * p.dim * state;
}

kda_status check_scan_sizes(const kda_scan_problem* q, ScanParams& s) {
  if (!q) return KDA_ERR_NULL_POINTER;
  const int64_t B = q->batch, T = q->T, lim = int64_t(1) << 31;
  if (B < 1 || T < 0 || B >= lim || T >= lim || B * T >= lim || q->dim < 1 || q->groups < 1 ||
      q->dim % q->groups != 0 ||
      (q->state != 8 && q->state != 16 && q->state != 32 && q->state != 64))
    return KDA_ERR_INVALID_SHAPE;
  int32_t N = q->N;
  if (q->cu_seqlens) {
    if (B != 1 || N < 1) return KDA_ERR_INVALID_SHAPE;
  } else {
    N = (int32_t)B;
  }
  std::memset(&s, 0, sizeof(s));
  s.cu = q->cu_seqlens, s.T = T, s.total = B * T;
  s.N = N, s.dim = q->dim, s.groups = q->groups, s.per = q->dim / q->groups;
  return KDA_OK;
}

kda_status check_scan(const kda_scan_problem* q, ScanParams& s, bool& vec) {
  const kda_status sizes = check_scan_sizes(q, s);
  if (sizes != KDA_OK) return sizes;
  if (!q->A_log) return KDA_ERR_NULL_POINTER;
  const int64_t gw = (int64_t)q->groups * q->state, lim = int64_t(1) << 31;
  for (int64_t st : {q->x_stride - q->dim, q->dt_stride - q->dim,
                     q->z ? q->z_stride - q->dim : 0, q->B_stride - gw, q->C_stride - gw})
    if (st < 0 || st >= lim) return KDA_ERR_INVALID_SHAPE;
  if ((q->dtype != KDA_ROW_BF16 && q->dtype != KDA_ROW_FP32) ||
      (q->state_dtype != KDA_STATE_FP32 && q->state_dtype != KDA_STATE_BF16))
    return KDA_ERR_INVALID_ARG;
  if (s.total > 0 && (!q->x || !q->dt || !q->B || !q->C)) return KDA_ERR_NULL_POINTER;
  const size_t e = q->dtype == KDA_ROW_FP32 ? 4 : 2;
  const void* row[5] = {q->x, q->dt, q->z, q->B, q->C};
  const int64_t stride[5] = {q->x_stride, q->dt_stride, q->z ? q->z_stride : 0, q->B_stride,
                             q->C_stride};
  vec = (q->dim / q->groups) % 8 == 0;
  for (int i = 0; i < 5; ++i) {
    if (!al_to(row[i], e)) return KDA_ERR_MISALIGNED;
    vec = vec && al_to(row[i], 16) && stride[i] * e % 16 == 0;
  }
  if (!al_to(q->A_log, 4) || !al_to(q->D, 4) || !al_to(q->dt_bias, 4) ||
      !al_to(q->initial_state, 16) || !al_to(q->cu_seqlens, 8))
    return KDA_ERR_MISALIGNED;
  s.x = q->x, s.dt = q->dt, s.z = q->z, s.B = q->B, s.C = q->C;
  s.x_s = q->x_stride, s.dt_s = q->dt_stride, s.z_s = q->z_stride;
  s.b_s = q->B_stride, s.c_s = q->C_stride;
  s.A_log = q->A_log, s.D = q->D, s.dt_bias = q->dt_bias;
  s.init = q->initial_state, s.state_bf16 = q->state_dtype == KDA_STATE_BF16;
  return KDA_OK;
}

__global__ void scan_status_kernel(const int64_t* cu, int N, int64_t total, unsigned* status) {
  check_seqlens(cu, N, total, status, kDevStatusBadSeqlens);
}

cudaError_t seqlens_status(const ScanParams& p, unsigned* status, cudaStream_t stream) {
  if (!p.cu) return cudaMemsetAsync(status, 0, sizeof(unsigned), stream);
  scan_status_kernel<<<1, 32, 0, stream>>>(p.cu, p.N, p.total, status);
  return cudaGetLastError();
}

// The reverse pass over segments; its tiles are the forward's.
cudaError_t launch_scan_rev(ScanParams p, int state, bool f32, bool vec, cudaStream_t stream) {
  const int64_t seg_len = p.seg_len, slots = p.slots;
  scan_fwd_plan(p, state);
  p.seg_len = seg_len, p.slots = slots;
  p.prescan = 1;
  p.chunk_states = nullptr;
  p.status = nullptr;
  return launch_pass<kReverse>(p, state, f32, vec, stream);
}

// The forward's own tiles and segments, the first two passes where sequences are cut, and
// the main pass.  p.seg_state holds the workspace's state region.
cudaError_t launch_scan_fwd(ScanParams p, int state, bool f32, bool vec, bool out,
                            cudaStream_t stream) {
  float* const ws_state = p.seg_state;
  float* const ws_sum = p.seg_sum;
  unsigned* const status = p.status;
  cudaError_t e = cudaSuccess;
  p.seg_state = nullptr;
  if (p.seg_len) {
    ScanParams q = p;
    q.seg_state = ws_state, q.seg_sum = ws_sum;
    q.chunk_states = nullptr;
    q.prescan = 1;
    e = launch_pass<kStatesOnly>(q, state, f32, vec, stream);
    if (e != cudaSuccess) return e;
    const int64_t grid = ((int64_t)p.dim * state + 127) / 128 * p.N;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    scan_carry_kernel<<<(unsigned)grid, 128, 0, stream>>>(q, state);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.seg_state = ws_state;
  }
  p.status = p.seg_len ? nullptr : status;
  return out ? launch_pass<kOutputs>(p, state, f32, vec, stream)
             : launch_pass<kStatesOnly>(p, state, f32, vec, stream);
}

}  // namespace scan
}  // namespace kda

extern "C" {

kda_status kda_scan_get_states_size(int64_t total_tokens, int32_t N, int32_t dim, int32_t state,
                                    size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  if (total_tokens < 0 || total_tokens >= (int64_t(1) << 31) || N < 0 || dim < 1 || state < 1)
    return KDA_ERR_INVALID_SHAPE;
  *bytes = ((size_t)(total_tokens / KDA_SCAN_CHUNK) + N + 1) * dim * state * sizeof(float);
  return KDA_OK;
}

kda_status kda_scan_get_workspace_size(const kda_scan_problem* problem, size_t* bytes) {
  using namespace kda;
  if (!bytes) return KDA_ERR_NULL_POINTER;
  scan::ScanParams p;
  const kda_status st = scan::check_scan_sizes(problem, p);
  if (st != KDA_OK) return st;
  scan::scan_fwd_plan(p, problem->state);
  *bytes = KDA_STATUS_BYTES + scan::fwd_ws_bytes(p, problem->state);
  return KDA_OK;
}

kda_status kda_scan_fwd(const kda_scan_problem* problem, void* out, void* final_state,
                        void* chunk_states, size_t chunk_states_bytes, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  scan::ScanParams p;
  bool vec = false;
  kda_status st = scan::check_scan(problem, p, vec);
  if (st != KDA_OK) return st;
  const bool f32 = problem->dtype == KDA_ROW_FP32;
  if (p.total > 0 && !out) return KDA_ERR_NULL_POINTER;
  if (!al_to(out, f32 ? 4 : 2) || !al_to(final_state, 16) || !al_to(chunk_states, 16) ||
      !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  const int state = problem->state;
  if (chunk_states) {
    size_t need = 0;
    kda_scan_get_states_size(p.total, p.N, p.dim, state, &need);
    if (chunk_states_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  }
  const bool step = !p.cu && p.T > 0 && p.T <= kStepTokens && !chunk_states;
  scan::scan_fwd_plan(p, problem->state);
  if (step) p.seg_len = 0;
  const size_t need = scan::fwd_ws_bytes(p, state);
  if (need > 0 && !workspace) return KDA_ERR_NULL_POINTER;
  if (workspace && workspace_bytes < KDA_STATUS_BYTES + need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  p.out = out, p.fin = final_state, p.chunk_states = static_cast<float*>(chunk_states);
  p.status = static_cast<unsigned*>(workspace);
  if (need > 0) scan::carve_fwd(p, state, static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
  vec = vec && al_to(out, 16);
  cudaError_t e;
  if (step)
    e = f32 ? (vec ? launch_step<float, true>(p, state, stream)
                   : launch_step<float, false>(p, state, stream))
            : (vec ? launch_step<scan::bf16, true>(p, state, stream)
                   : launch_step<scan::bf16, false>(p, state, stream));
  else
    e = scan::launch_scan_fwd(p, state, f32, vec, true, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
