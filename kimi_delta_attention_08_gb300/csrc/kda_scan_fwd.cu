// kda_scan_fwd.cu -- the selective state space scan, forward: prompts, packed prompts and
// single tokens.
//
//   delta = softplus(dt + dt_bias),  h_t = 2^(delta A2) h_{t-1} + (delta x) B_t,
//   y = C_t . h_t + D x,  out = y silu(z),     A2 = -exp(A_log) log2 e
//
// Per (token, channel, state) this takes one exponential and four fp32 operations, against
// 8 bytes of rows per (token, channel) in bf16, so at 16 states it is bound by the special
// function and FMA pipes, not by HBM.  The state never leaves the registers: a thread
// walks all tokens of its sequence (or segment).  Blocks of 32 tokens are staged through
// shared memory: every (token, channel)'s softplus is computed once by the thread that
// loads it, and the next block's rows are in flight meanwhile.  The dot product over a
// channel's lanes is reduced for as many tokens at a time as there are lanes, so each lane
// ends up with one token's sum.
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

constexpr int kCh = 32;      // channels per CTA
constexpr int kYPitch = 40;  // floats per token of the y tile: spreads 4 tokens over the banks

// A thread's staged elements: SN vectors of SV channels, vector q of token tok(q).
template <int NT>
struct Stage {
  static constexpr int EPT = kScanBlock * kCh / NT;
  static constexpr int SV = EPT < 8 ? EPT : 8;
  static constexpr int SN = EPT / SV;
  static constexpr int PER_ROW = kCh / SV;
};

template <typename T, int NS, bool VEC, bool OUT>
__global__ void __launch_bounds__(kCh * NS / kStates<NS>)
    scan_fwd_kernel(const ScanParams p) {
  constexpr int SP = kStates<NS>, LPC = NS / SP, NT = kCh * LPC;
  using S = Stage<NT>;
  constexpr int SV = S::SV, SN = S::SN, PER_ROW = S::PER_ROW;
  __shared__ float2 s_dx[kScanBlock][kCh];  // delta, delta x
  __shared__ __align__(16) float s_b[kScanBlock][NS];
  __shared__ __align__(16) float s_c[OUT ? kScanBlock : 1][NS];
  __shared__ __align__(16) float s_y[OUT ? kScanBlock : 1][kYPitch];

  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t slot = blockIdx.x / p.tiles;
  const int tile = (int)(blockIdx.x % p.tiles);
  if (blockIdx.x == 0 && tid < 32 && p.status) {
    if (p.cu) check_seqlens(p.cu, p.N, p.total, p.status, kDevStatusBadSeqlens);
    else if (tid == 0) *p.status = 0u;
  }
  const Segment u = find_unit(p, slot);
  if (!u.live) return;
  const bool prescan = !OUT && p.prescan;
  if (prescan && u.last) return;  // its end starts no segment
  const int grp = tile / p.tiles_per_group;
  const int c_lo = (tile % p.tiles_per_group) * kCh;     // within the group
  const int c_n = min(kCh, p.per - c_lo);
  const int64_t ch0 = (int64_t)grp * p.per + c_lo;       // first channel of the tile
  const int c = tid / LPC, l = tid % LPC;
  const bool mine = c < c_n;
  const int64_t st_at = (ch0 + c) * NS + l * SP;         // state offset within [dim][NS]
  const int64_t st_seq = (int64_t)p.dim * NS;

  float A2[SP], h[SP];
#pragma unroll
  for (int i = 0; i < SP; ++i) A2[i] = h[i] = 0.f;
  if (mine) {
    load_rates<SP>(A2, p.A_log, st_at);
    if (p.seg_state && !prescan) load_state<SP>(h, p.seg_state, slot * st_seq + st_at, false);
    else if (u.first && p.init) load_state<SP>(h, p.init, u.n * st_seq + st_at, p.state_bf16);
  }
  float sum_delta = 0.f;

  // the staged channels of this thread
  const int sc = VEC ? (tid % PER_ROW) * SV : tid % PER_ROW;   // first channel
  const int sstep = VEC ? 1 : PER_ROW;
  const int sleft = VEC ? (sc < c_n ? kCh : 0) : c_n - sc;
  float bias[SV], dsk[SV];
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    const int cc = sc + i * sstep;
    bias[i] = cc < c_n && p.dt_bias ? __ldg(p.dt_bias + ch0 + cc) : 0.f;
    dsk[i] = OUT && cc < c_n && p.D ? __ldg(p.D + ch0 + cc) : 0.f;
  }
  Raw<T, SV> rx[SN], rt[SN], rz[SN];
  Raw<T, SP> rb, rc;
  auto fetch = [&](int64_t t0) {
#pragma unroll
    for (int q = 0; q < SN; ++q) {
      const int64_t t = t0 + (q * NT + tid) / PER_ROW;
      rx[q] = rt[q] = rz[q] = Raw<T, SV>{};
      if (t >= u.t1 || sleft <= 0) continue;
      load_row<T, SV, VEC>(rx[q], static_cast<const T*>(p.x) + t * p.x_s + ch0 + sc, sstep, (int64_t)sleft);
      load_row<T, SV, VEC>(rt[q], static_cast<const T*>(p.dt) + t * p.dt_s + ch0 + sc, sstep, (int64_t)sleft);
      if (OUT && p.z)
        load_row<T, SV, VEC>(rz[q], static_cast<const T*>(p.z) + t * p.z_s + ch0 + sc, sstep, (int64_t)sleft);
    }
    rb = rc = Raw<T, SP>{};
    const int64_t t = t0 + tid / LPC;  // the thread's channel index doubles as a token
    if (t < u.t1) {
      load_row<T, SP, VEC>(rb, static_cast<const T*>(p.B) + t * p.b_s + grp * NS + l * SP, 1, SP);
      if (OUT) load_row<T, SP, VEC>(rc, static_cast<const T*>(p.C) + t * p.c_s + grp * NS + l * SP, 1, SP);
    }
  };
  fetch(u.t0);
  for (int64_t t0 = u.t0; t0 < u.t1; t0 += kScanBlock) {
    const int nt = (int)min((int64_t)kScanBlock, u.t1 - t0);
    // tokens past nt are staged as zero steps, which leave the state as it is
#pragma unroll
    for (int q = 0; q < SN; ++q) {
      const int tok = (q * NT + tid) / PER_ROW;
      float xv[SV], tv[SV];
      unpack(rx[q], xv);
      unpack(rt[q], tv);
#pragma unroll
      for (int i = 0; i < SV; ++i) {
        float sig, d = softplus(tv[i] + bias[i], sig);
        if (tok >= nt) d = 0.f;
        s_dx[tok][sc + i * sstep] = make_float2(d, d * xv[i]);
      }
    }
    {
      float v[SP];
      unpack(rb, v);
#pragma unroll
      for (int i = 0; i < SP; ++i) s_b[tid / LPC][l * SP + i] = v[i];
      if (OUT) {
        unpack(rc, v);
#pragma unroll
        for (int i = 0; i < SP; ++i) s_c[tid / LPC][l * SP + i] = v[i];
      }
    }
    Raw<T, SV> cx[SN], cz[SN];
#pragma unroll
    for (int q = 0; q < SN; ++q) cx[q] = rx[q], cz[q] = rz[q];
    __syncthreads();
    if (t0 + kScanBlock < u.t1) fetch(t0 + kScanBlock);
    if (p.chunk_states && mine) {
      const int64_t chunk = u.bos / kScanBlock + u.n + (t0 - u.bos) / kScanBlock;
      store_state<SP>(p.chunk_states, chunk * st_seq + st_at, h, false);
    }
    for (int j0 = 0; j0 < nt; j0 += LPC) {
      float y[LPC];
#pragma unroll
      for (int k = 0; k < LPC; ++k) {
        const float2 d = s_dx[j0 + k][c];
        float2 acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
          const float2 b2 = *reinterpret_cast<const float2*>(&s_b[j0 + k][l * SP + i]);
          const float2 e = ptx::f2mul(make_float2(d.x, d.x), make_float2(A2[i], A2[i + 1]));
          const float2 a = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
          const float2 hn = ptx::f2fma(a, make_float2(h[i], h[i + 1]),
                                       ptx::f2mul(make_float2(d.y, d.y), b2));
          h[i] = hn.x, h[i + 1] = hn.y;
          if (OUT)
            acc = ptx::f2fma(*reinterpret_cast<const float2*>(&s_c[j0 + k][l * SP + i]), hn, acc);
        }
        if (OUT) y[k] = acc.x + acc.y;
        else sum_delta += d.x;
      }
      if (OUT) {
        int off = 0;
        reduce_scatter<LPC, LPC / 2, 1>(y, lane, off);
        s_y[j0 + off][c] = y[0];
      }
    }
    __syncthreads();
    if (OUT) {
#pragma unroll
      for (int q = 0; q < SN; ++q) {
        const int tok = (q * NT + tid) / PER_ROW;
        if (tok >= nt || sleft <= 0) continue;
        float xv[SV], zv[SV], o[SV];
        unpack(cx[q], xv);
        unpack(cz[q], zv);
#pragma unroll
        for (int i = 0; i < SV; ++i) {
          o[i] = fmaf(dsk[i], xv[i], s_y[tok][sc + i * sstep]);
          if (p.z) o[i] *= zv[i] * sigmoid(zv[i]);
        }
        store_row<T, SV, VEC>(static_cast<T*>(p.out) + (t0 + tok) * p.dim + ch0 + sc, o, sstep,
                              (int64_t)sleft);
      }
    }
  }
  if (!mine) return;
  if (prescan) {
    store_state<SP>(p.seg_state, slot * st_seq + st_at, h, false);
    if (l == 0) p.seg_sum[slot * p.dim + ch0 + c] = sum_delta;
  } else if (OUT && u.last && p.fin) {
    store_state<SP>(p.fin, u.n * st_seq + st_at, h, p.state_bf16);
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
  const float A2 = -expf(__ldg(p.A_log + i)) * kLog2e;
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

// Single tokens and prompts of a few: no staging.  A thread loads its states of one
// (sequence, channel), walks the tokens and writes the states back; bound by HBM through
// the states, whose loads and stores are contiguous over the warp.
template <typename T, int NS>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams p) {
  constexpr int SP = kStates<NS>, LPC = NS / SP;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i == 0 && p.status) *p.status = 0u;
  const int64_t per_seq = (int64_t)p.dim * LPC;
  const bool mine = i < p.N * per_seq;
  const int n = mine ? (int)(i / per_seq) : p.N - 1;
  const int64_t r = mine ? i % per_seq : 0;
  const int64_t ch = r / LPC;
  const int l = (int)(r % LPC), grp = (int)(ch / p.per);
  const int64_t st_at = n * (int64_t)p.dim * NS + ch * NS + l * SP;
  float A2[SP], h[SP];
#pragma unroll
  for (int k = 0; k < SP; ++k) h[k] = 0.f;
  if (p.init && mine) load_state<SP>(h, p.init, st_at, p.state_bf16);
  load_rates<SP>(A2, p.A_log, ch * NS + l * SP);
  const float bias = p.dt_bias ? __ldg(p.dt_bias + ch) : 0.f, D = p.D ? __ldg(p.D + ch) : 0.f;
  for (int64_t t = n * p.T; t < (n + 1) * p.T; ++t) {
    const float x = to_f(static_cast<const T*>(p.x)[t * p.x_s + ch]);
    float sig;
    const float d = softplus(to_f(static_cast<const T*>(p.dt)[t * p.dt_s + ch]) + bias, sig);
    const T* B = static_cast<const T*>(p.B) + t * p.b_s + grp * NS + l * SP;
    const T* C = static_cast<const T*>(p.C) + t * p.c_s + grp * NS + l * SP;
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < SP; ++k) {
      h[k] = fmaf(ptx::ex2_approx(d * A2[k]), h[k], d * x * to_f(B[k]));
      y = fmaf(to_f(C[k]), h[k], y);
    }
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (l == 0 && mine) {
      y = fmaf(D, x, y);
      if (p.z) {
        const float z = to_f(static_cast<const T*>(p.z)[t * p.z_s + ch]);
        y *= z * sigmoid(z);
      }
      static_cast<T*>(p.out)[t * p.dim + ch] = from_f<T>(y);
    }
  }
  if (p.fin && mine) store_state<SP>(p.fin, st_at, h, p.state_bf16);
}

template <typename T, bool VEC, bool OUT>
cudaError_t launch_main(const ScanParams& p, int state, cudaStream_t stream) {
  const int64_t grid = p.slots * p.tiles;
  if (grid == 0) return cudaSuccess;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)grid;
  switch (state) {
    case 8: scan_fwd_kernel<T, 8, VEC, OUT><<<g, kCh * 2, 0, stream>>>(p); break;
    case 16: scan_fwd_kernel<T, 16, VEC, OUT><<<g, kCh * 4, 0, stream>>>(p); break;
    case 32: scan_fwd_kernel<T, 32, VEC, OUT><<<g, kCh * 4, 0, stream>>>(p); break;
    default: scan_fwd_kernel<T, 64, VEC, OUT><<<g, kCh * 8, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

template <bool OUT>
cudaError_t launch_pass(const ScanParams& p, int state, bool f32, bool vec, cudaStream_t stream) {
  if (f32) return vec ? launch_main<float, true, OUT>(p, state, stream)
                      : launch_main<float, false, OUT>(p, state, stream);
  return vec ? launch_main<bf16, true, OUT>(p, state, stream)
             : launch_main<bf16, false, OUT>(p, state, stream);
}

template <typename T>
cudaError_t launch_step(const ScanParams& p, int state, cudaStream_t stream) {
  const int lpc = state >= 32 ? state / 8 : state / 4;
  const int64_t grid = ((int64_t)p.N * p.dim * lpc + 255) / 256;
  if (grid == 0) return cudaSuccess;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned g = (unsigned)grid;
  switch (state) {
    case 8: scan_step_kernel<T, 8><<<g, 256, 0, stream>>>(p); break;
    case 16: scan_step_kernel<T, 16><<<g, 256, 0, stream>>>(p); break;
    case 32: scan_step_kernel<T, 32><<<g, 256, 0, stream>>>(p); break;
    default: scan_step_kernel<T, 64><<<g, 256, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

constexpr int kStepTokens = 8;  // longest prompt of the single-token kernel

bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

namespace scan {

// A unit is one CTA's walk over one segment; sequences are cut until there are about 8 CTAs
// of 128 threads for each SM, but not below 256 tokens.
constexpr int64_t kMinSegment = 256;
constexpr int64_t kSms = 152;

ScanPlan scan_plan(const ScanParams& p, int64_t tiles, int64_t ctas_per_sm) {
  const bool packed = p.cu != nullptr;
  const int64_t N = p.N, T = p.T, total = p.total;
  ScanPlan r = {0, N};
  const int64_t want = kSms * ctas_per_sm;
  const int64_t whole = packed ? tiles : tiles * N;        // CTAs that surely run side by side
  if (whole * 4 >= want * 3 || total == 0) return r;
  const int64_t pieces = (want + whole - 1) / whole;
  const int64_t span = packed ? total : T;
  int64_t len = (span + pieces - 1) / pieces;
  len = (len + kScanBlock - 1) / kScanBlock * kScanBlock;
  if (len < kMinSegment) len = kMinSegment;
  if (!packed && len >= T) return r;
  r.seg_len = len;
  r.slots = total / len + N;
  return r;
}

void scan_fwd_plan(ScanParams& p) {
  p.tiles_per_group = (p.per + kCh - 1) / kCh;
  p.tiles = (int64_t)p.tiles_per_group * p.groups;
  // 8 CTAs of 128 threads: all that an SM holds at the kernel's registers
  const ScanPlan r = scan_plan(p, p.tiles, 8);
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
  if (cu) check_seqlens(cu, N, total, status, kDevStatusBadSeqlens);
  else if (threadIdx.x == 0) *status = 0u;
}

cudaError_t seqlens_status(const ScanParams& p, unsigned* status, cudaStream_t stream) {
  if (!p.cu) return cudaMemsetAsync(status, 0, sizeof(unsigned), stream);
  scan_status_kernel<<<1, 32, 0, stream>>>(p.cu, p.N, p.total, status);
  return cudaGetLastError();
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
    e = launch_pass<false>(q, state, f32, vec, stream);
    if (e != cudaSuccess) return e;
    const int64_t grid = ((int64_t)p.dim * state + 127) / 128 * p.N;
    if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
    scan_carry_kernel<<<(unsigned)grid, 128, 0, stream>>>(q, state);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.seg_state = ws_state;
  }
  p.status = p.seg_len ? nullptr : status;
  return out ? launch_pass<true>(p, state, f32, vec, stream)
             : launch_pass<false>(p, state, f32, vec, stream);
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
  scan::scan_fwd_plan(p);
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
  scan::scan_fwd_plan(p);
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
    e = f32 ? launch_step<float>(p, state, stream) : launch_step<bf16>(p, state, stream);
  else
    e = scan::launch_scan_fwd(p, state, f32, vec, true, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
