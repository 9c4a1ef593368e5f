// kda_scan.cuh -- what the scan's forward and backward share: the division of the
// (tokens, channels, states) space over threads, the segments of a split scan and the
// reductions across lanes.
//
// A thread holds SP states of a channel pair in registers (the single-token kernel: of one
// channel), and a warp 32 / LPC of these with LPC = state / SP lanes each: bit 0 of the lane
// and its top bits choose the states' part, the bits between them the channels.  So two
// neighbouring lanes always share a channel, and a quarter of the warp reads two addresses
// of B and C: a 16-byte read from shared memory then takes 2.1 cycles, and one of 8 bytes by
// channel 1.1, where other orders of the same lanes take 4 and 2 (measured).  A CTA holds CH
// channels of one group and walks the tokens of a sequence or a segment.
//
// Segments.  A sequence is cut into segments of seg_len tokens (0: not cut).  Segment s of
// sequence n has slot floor(bos_n / seg_len) + n + s: distinct for all segments of all
// sequences and below total / seg_len + N.
#pragma once

#include <cfloat>

#include "kda_internal.h"
#include "kda_rows.cuh"
#include "../../include/kda_layer.h"

namespace kda {
namespace scan {

using namespace rows;

constexpr int kScanBlock = KDA_SCAN_CHUNK;  // 32 tokens: one saved state each, the backward's block

struct ScanParams {
  const void *x, *dt, *z, *B, *C, *dout;
  int64_t x_s, dt_s, z_s, b_s, c_s;
  const float *A_log, *D, *dt_bias;
  const void *init, *dfin;
  int32_t state_bf16, prescan;
  const int64_t* cu;
  int64_t T, total;
  int32_t N, dim, groups, per;   // per: channels per group
  int32_t tiles_per_group;
  int64_t tiles, slots, seg_len;
  void *out, *fin;
  float* chunk_states;
  float* seg_state;              // [slots][dim][state]: ends, then starts, of segments
  float* seg_sum;                // [slots][dim]: sum of delta
  unsigned* status;
  void *dx, *ddt, *dz;           // backward
  float *part_bc, *part_par;     // [tiles][total][2][state], [slots][dim][state + 2]
  float* dinit;
};

// What a unit (one slot, one channel tile) works on.
struct Segment {
  int n;              // sequence
  int64_t bos, eos;   // its tokens
  int64_t t0, t1;     // the segment's tokens
  bool first, last;   // of the sequence
  bool live;          // false: an unused slot
};

__device__ __forceinline__ void seq_bounds(const ScanParams& p, int n, int64_t& bos, int64_t& eos) {
  if (p.cu) {
    bos = __ldg(p.cu + n);
    eos = __ldg(p.cu + n + 1);
    bos = bos < 0 ? 0 : bos > p.total ? p.total : bos;
    eos = eos > p.total ? p.total : eos < bos ? bos : eos;
  } else {
    bos = (int64_t)n * p.T;
    eos = bos + p.T;
  }
}

__device__ __forceinline__ int64_t first_slot(const ScanParams& p, int n) {
  int64_t bos, eos;
  seq_bounds(p, n, bos, eos);
  return p.seg_len ? bos / p.seg_len + n : n;
}

// All lanes of a warp together (a search of 32 pivots a step, as find_sequence).
__device__ __forceinline__ Segment find_unit(const ScanParams& p, int64_t slot) {
  Segment u;
  int64_t s = 0;
  if (p.seg_len == 0) {
    u.n = (int)slot;
  } else {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = p.N;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + lane * step;
      const bool le = at < hi && first_slot(p, at) <= slot;
      const unsigned m = __ballot_sync(0xffffffffu, le) | 1u;
      const int k = 31 - __clz(m);
      hi = min(hi, lo + (k + 1) * step);
      lo = lo + k * step;
    }
    u.n = lo;
    s = slot - first_slot(p, lo);
  }
  seq_bounds(p, u.n, u.bos, u.eos);
  const int64_t len = p.seg_len ? p.seg_len : u.eos - u.bos;
  u.t0 = u.bos + s * len;
  u.live = s >= 0 && (s == 0 || u.t0 < u.eos);
  u.t1 = u.t0 + len < u.eos ? u.t0 + len : u.eos;
  u.first = s == 0;
  u.last = u.t1 == u.eos;
  return u;
}

// softplus(v) = max(v, 0) + log1p(u), u = exp(-|v|) in (0, 1], with the relative accuracy
// that small steps need: log1p(u) = u P(u), P of degree 8 with P(0) = 1, fitted to
// log1p(u) / u on [0, 1] by reweighted least squares to an even relative error (3.3e-8;
// 1.4e-7 at most and 7e-9 on average as evaluated in fp32).  No reciprocal: that costs as
// much as two exponentials.
__device__ __forceinline__ pair softplus(pair v, pair& u) {
  const float2 w = un(v);
  u = pr(ptx::ex2_approx(-fabsf(w.x) * kLog2e), ptx::ex2_approx(-fabsf(w.y) * kLog2e));
  pair s = pfma(pr(0.00536481664f), u, pr(-0.0300657619f));
  s = pfma(s, u, pr(0.0792044848f));
  s = pfma(s, u, pr(-0.137537986f));
  s = pfma(s, u, pr(0.191536531f));
  s = pfma(s, u, pr(-0.248571634f));
  s = pfma(s, u, pr(0.33321324f));
  s = pfma(s, u, pr(-0.499996483f));
  s = pfma(s, u, pr(1.0f));
  return pfma(u, s, pr(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v, float& u) {
  pair w;
  const float r = un(softplus(pr(v, 0.f), w)).x;
  u = un(w).x;
  return r;
}
// Its derivative sigmoid(v) from the same u.
__device__ __forceinline__ float softplus_slope(float v, float u) {
  const float r = ptx::rcp_approx(1.0f + u);
  return v >= 0.f ? r : u * r;
}

// A lane's channel within the warp and its states' part.
template <int LPC>
__device__ __forceinline__ int lane_channel(int lane) {
  return LPC == 1 ? lane : (lane >> 1) % (32 / LPC);
}
template <int LPC>
__device__ __forceinline__ int lane_part(int lane) {
  return LPC == 1 ? 0 : (lane & 1) | (lane / (64 / LPC) << 1);
}

// The decay 2^(delta A2) of two channels.  The hardware's exponential lies 1.8e-8 low on
// average where its result is in (1/2, 1) (measured over 4 million points in each of
// several ranges), and long products of decays multiply that up, so the exponent is raised
// by as much.  A step of zero still leaves exactly 1.  At no cost this takes the error of
// the decay rates' gradient from 1.0e-6 to 3.8e-7 (16,384 tokens of 1,024 channels).
__device__ __forceinline__ pair decay(pair delta, pair A2) {
  return pex2(pfma(delta, A2, pr(2.5e-8f)));
}

// h <- 2^(delta A2) h + (delta x) B for a state of two channels; b = (B, B).
__device__ __forceinline__ pair advance(pair h, pair A2, pair delta, pair dx, pair b) {
  return pfma(decay(delta, A2), h, pmul(dx, b));
}

__device__ __forceinline__ float sum_of(float a, float b) { return a + b; }
__device__ __forceinline__ pair sum_of(pair a, pair b) { return padd(a, b); }

// v[0 .. L) summed over the lanes that differ in the bits from `BIT` down to `LOW`: each
// step the lanes of a pair keep one half of the values each.  Afterwards the thread holds
// max(L / 2^steps, 1) sums, those from value `off` on (all lanes of a group hold the same
// one where values ran out).  V: float, or a pair of them.
template <int L, int BIT, int LOW, typename V>
__device__ __forceinline__ void reduce_scatter(V* v, int lane, int& off) {
  if constexpr (BIT >= LOW) {
    if constexpr (L > 1) {
      const bool up = lane & BIT;
#pragma unroll
      for (int i = 0; i < L / 2; ++i) {
        const V give = up ? v[i] : v[i + L / 2];
        const V keep = up ? v[i + L / 2] : v[i];
        v[i] = sum_of(keep, __shfl_xor_sync(0xffffffffu, give, BIT));
      }
      off += up ? L / 2 : 0;
      reduce_scatter<L / 2, BIT / 2, LOW>(v, lane, off);
    } else {
      v[0] = sum_of(v[0], __shfl_xor_sync(0xffffffffu, v[0], BIT));
      reduce_scatter<1, BIT / 2, LOW>(v, lane, off);
    }
  }
}

// The same over a channel's lanes.
template <int L, int LPC, typename V>
__device__ __forceinline__ void reduce_states(V* v, int lane, int& off) {
  if constexpr (LPC > 2) reduce_scatter<L, 16, 64 / LPC>(v, lane, off);
  constexpr int ROUNDS = LPC > 1 ? LPC / 2 : 1, LEFT = L / ROUNDS > 1 ? L / ROUNDS : 1;
  if constexpr (LPC > 1) reduce_scatter<LEFT, 1, 1>(v, lane, off);
}

template <int SP>
__device__ __forceinline__ void load_state(float (&h)[SP], const void* p, int64_t at, bool b16) {
#pragma unroll
  for (int i = 0; i < SP; i += 4) {
    if (b16) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at + i);
      h[i] = lo_bf16(w.x), h[i + 1] = hi_bf16(w.x), h[i + 2] = lo_bf16(w.y), h[i + 3] = hi_bf16(w.y);
    } else {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + i);
      h[i] = v.x, h[i + 1] = v.y, h[i + 2] = v.z, h[i + 3] = v.w;
    }
  }
}
template <int SP>
__device__ __forceinline__ void store_state(void* p, int64_t at, const float (&h)[SP], bool b16) {
#pragma unroll
  for (int i = 0; i < SP; i += 4) {
    if (b16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at + i) =
          make_uint2(pack_bf16(h[i], h[i + 1]), pack_bf16(h[i + 2], h[i + 3]));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at + i) =
          make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
  }
}

// Decay rates in base 2: A2 = -exp(A_log) log2 e, so that exp(-delta exp(A_log)) = 2^(delta A2).
// exp(v) = 2^(v log2 e) with the product's rounding error put back: 2^e (1 + e' ln 2); not
// where that error is no number because v or the result is infinite.  An infinite rate
// becomes the largest finite one, so that a step of zero still leaves 1.
__device__ __forceinline__ float rate_of(float v) {
  const float hi = v * kLog2e;
  const float lo = fmaf(v, kLog2eRest, fmaf(v, kLog2e, -hi));
  const float e = ptx::ex2_approx(hi);
  const float r = fmaf(e, lo * kLn2, e);
  const float a = -kLog2e * (fabsf(r) < INFINITY ? r : e);
  return a < -FLT_MAX ? -FLT_MAX : a;
}
template <int SP>
__device__ __forceinline__ void load_rates(float (&a)[SP], const float* A_log, int64_t at) {
#pragma unroll
  for (int i = 0; i < SP; ++i) a[i] = rate_of(__ldg(A_log + at + i));
}

constexpr int64_t kSms = 152;  // a GB300's: a workspace's size is asked for without a device

// How sequences are cut (seg_len 0: not at all) for a pass over `tiles` channel tiles whose
// SMs hold `resident` CTAs; and the CTAs that run side by side without cutting.
struct ScanPlan {
  int64_t seg_len, slots;
};
ScanPlan scan_plan(const ScanParams& p, int64_t tiles, int64_t resident, bool cut);
int64_t scan_whole_units(const ScanParams& p, int64_t tiles);

// The checks of sizes and of arguments that the entry points share; they fill the
// problem's part of `s`, and whether every row starts on 16 bytes.
kda_status check_scan_sizes(const kda_scan_problem* q, ScanParams& s);
kda_status check_scan(const kda_scan_problem* q, ScanParams& s, bool& vec);

// The status word from a check of cu_seqlens.
cudaError_t seqlens_status(const ScanParams& p, unsigned* status, cudaStream_t stream);

// The forward's tiles and plan, the bytes it needs for segments and their place.
void scan_fwd_plan(ScanParams& p, int state);
size_t fwd_ws_bytes(const ScanParams& p, int state);
void carve_fwd(ScanParams& p, int state, void* ws);
// All its passes (out: the main pass writes outputs, else saved states only).
cudaError_t launch_scan_fwd(ScanParams p, int state, bool f32, bool vec, bool out,
                            cudaStream_t stream);

// The gradient that leaves each segment at its start, from a zero gradient at its end (the
// last one's: dfinal_state), into p.seg_state, and the segment's sum of delta.
cudaError_t launch_scan_rev(ScanParams p, int state, bool f32, bool vec, cudaStream_t stream);

}  // namespace scan
}  // namespace kda
