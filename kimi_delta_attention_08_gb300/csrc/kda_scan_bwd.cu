// kda_scan_bwd.cu -- the selective state space scan, backward.
//
// With g_t the gradient of h_t, a_t = 2^(delta_t A2), dy = dout silu(z):
//   g_t = dy_t C_t + a_{t+1} g_{t+1}        (from dfinal_state after the last token)
//   dC_t = sum_d dy_t h_t                    dB_t = sum_d (delta_t x_t) g_t
//   q_t = sum_n g_t B_t,  s_t = sum_n (g_t a_t h_{t-1}) A
//   dx = delta q + dy D,  ddt = (x q + s) sigmoid(dt + dt_bias),  dA_log = A sum_t delta g a h_{t-1}
//   dz = dout (y + D x) silu'(z),  dD = sum dy x,  ddt_bias = sum ddt,  dinitial = a_1 g_1
//
// The states h come from the forward's saved state of every 32-token block.  A CTA walks
// its blocks from the last to the first: from a block's saved state it runs forward once,
// keeping a checkpoint every SB tokens in shared memory, then takes the SB-token pieces in
// reverse, recomputing a piece's decays and states into registers and running the reverse
// recurrence over them.  Sums over a channel's states go across its lanes; the sums over
// channels that dB and dC need go across the warp's channels by halving exchanges, over
// the CTA's warps through shared memory and over the channel tiles through a partial
// buffer that a second launch adds up, all in a fixed order.
//
// Per (token, channel, state) this takes two exponentials and about 20 fp32 operations, so
// it is bound by the FMA and issue pipes.  As in the forward, sequences are cut into
// segments where channels alone do not fill the GPU: a reverse pass computes each
// segment's gradient at its start from a zero gradient at its end, and a second carries
// the gradients over the segments.
#include <cstring>

#include "kda_scan.cuh"

namespace kda {
namespace {

using namespace scan;

constexpr int kRevCh = 32;

template <int NS>
constexpr int kStates = NS >= 32 ? 8 : 4;
template <int NS>
constexpr int kBwdCh = NS == 64 ? 32 : 64;

template <typename T, int NS>
struct BwdShape {
  static constexpr int CH = kBwdCh<NS>;
  static constexpr int SP = kStates<NS>, LPC = NS / SP, NT = CH * LPC, NW = NT / 32;
  static constexpr int SB = 32 / SP, NSB = kScanBlock / SB;   // tokens per piece, pieces
  static constexpr int CL = 32 / LPC;                         // channels per warp
  static constexpr int EPT = kScanBlock * CH / NT, SV = EPT < 8 ? EPT : 8, SN = EPT / SV;
  static constexpr int PER_ROW = CH / SV;
  // shared memory, in floats
  static constexpr int DX = 0;                                // float2 [32][CH]: delta, delta x,
                                                              // then q and s of done tokens
  static constexpr int DY = DX + 2 * kScanBlock * CH;         // [32][CH]: dy, then y
  static constexpr int SB_ = DY + kScanBlock * CH;            // B [32][NS]
  static constexpr int SC_ = SB_ + kScanBlock * NS;           // C [32][NS]
  static constexpr int PART = SC_ + kScanBlock * NS;          // [NW][SB][2 NS]
  static constexpr int CKPT = PART + NW * SB * 2 * NS;        // [NSB - 1][NT][SP]
  static constexpr int FLOATS = CKPT + (NSB - 1) * NT * SP;
};

template <typename T, int NS, bool VEC>
__global__ void __launch_bounds__(BwdShape<T, NS>::NT, 2) scan_bwd_kernel(const ScanParams p) {
  using H = BwdShape<T, NS>;
  constexpr int CH = H::CH, SP = H::SP, LPC = H::LPC, NT = H::NT, NW = H::NW, SB = H::SB;
  constexpr int NSB = H::NSB, SV = H::SV, SN = H::SN, PER_ROW = H::PER_ROW;
  extern __shared__ __align__(16) float sm[];
  float2(*s_dx)[CH] = reinterpret_cast<float2(*)[CH]>(sm + H::DX);
  float(*s_dy)[CH] = reinterpret_cast<float(*)[CH]>(sm + H::DY);
  float(*s_b)[NS] = reinterpret_cast<float(*)[NS]>(sm + H::SB_);
  float(*s_c)[NS] = reinterpret_cast<float(*)[NS]>(sm + H::SC_);
  float* const s_part = sm + H::PART;
  float* const s_ck = sm + H::CKPT;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t st_seq = (int64_t)p.dim * NS;
  if ((int64_t)blockIdx.x >= p.slots * p.tiles) {  // zero gradients behind the last sequence
    const int64_t i0 = __ldg(p.cu + p.N), blk = (int64_t)blockIdx.x - p.slots * p.tiles;
    const int64_t nb = (int64_t)gridDim.x - p.slots * p.tiles;
    for (int64_t i = (i0 < 0 ? 0 : i0) * p.dim + blk * NT + tid; i < p.total * p.dim; i += nb * NT) {
      static_cast<T*>(p.dx)[i] = from_f<T>(0.f);
      static_cast<T*>(p.ddt)[i] = from_f<T>(0.f);
      if (p.dz) static_cast<T*>(p.dz)[i] = from_f<T>(0.f);
    }
    return;
  }
  const int64_t slot = blockIdx.x / p.tiles;
  const int tile = (int)(blockIdx.x % p.tiles);
  const Segment u = find_unit(p, slot);
  const int grp = tile / p.tiles_per_group;
  const int c_lo = (tile % p.tiles_per_group) * CH;
  const int c_n = min(CH, p.per - c_lo);
  const int64_t ch0 = (int64_t)grp * p.per + c_lo;
  const int c = tid / LPC, l = tid % LPC;
  const bool mine = c < c_n;
  const int64_t st_at = (ch0 + c) * NS + l * SP;

  float A2[SP], g[SP], dA[SP], h0[SP];
#pragma unroll
  for (int i = 0; i < SP; ++i) A2[i] = g[i] = dA[i] = 0.f;
  if (mine) {
    load_rates<SP>(A2, p.A_log, st_at);
    if (u.live && u.last) {
      if (p.dfin) load_state<SP>(g, p.dfin, u.n * st_seq + st_at, p.state_bf16);
    } else if (u.live) {
      load_state<SP>(g, p.seg_state, slot * st_seq + st_at, false);
    }
  }
  const int sc = VEC ? (tid % PER_ROW) * SV : tid % PER_ROW;
  const int sstep = VEC ? 1 : PER_ROW;
  const int64_t sleft = VEC ? (sc < c_n ? CH : 0) : c_n - sc;
  float bias[SV], dsk[SV], sum_d[SV], sum_b[SV];
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    const int cc = sc + i * sstep;
    bias[i] = cc < c_n && p.dt_bias ? __ldg(p.dt_bias + ch0 + cc) : 0.f;
    dsk[i] = cc < c_n && p.D ? __ldg(p.D + ch0 + cc) : 0.f;
    sum_d[i] = sum_b[i] = 0.f;
  }

  const int64_t blocks = u.live ? (u.t1 - u.t0 + kScanBlock - 1) / kScanBlock : 0;
  for (int64_t blk = blocks - 1; blk >= 0; --blk) {
    const int64_t t0 = u.t0 + blk * kScanBlock;
    const int nt = (int)min((int64_t)kScanBlock, u.t1 - t0);
    // ---- stage the block; tokens past nt are zero steps with zero gradients
#pragma unroll
    for (int q = 0; q < SN; ++q) {
      const int tok = (q * NT + tid) / PER_ROW;
      Raw<T, SV> rx = {}, rt = {}, rz = {}, ro = {};
      const int64_t t = t0 + tok;
      if (tok < nt && sleft > 0) {
        load_row<T, SV, VEC>(rx, static_cast<const T*>(p.x) + t * p.x_s + ch0 + sc, sstep, sleft);
        load_row<T, SV, VEC>(rt, static_cast<const T*>(p.dt) + t * p.dt_s + ch0 + sc, sstep, sleft);
        if (p.z)
          load_row<T, SV, VEC>(rz, static_cast<const T*>(p.z) + t * p.z_s + ch0 + sc, sstep, sleft);
        load_row<T, SV, VEC>(ro, static_cast<const T*>(p.dout) + t * p.dim + ch0 + sc, sstep, sleft);
      }
      float xv[SV], tv[SV], zv[SV], ov[SV];
      unpack(rx, xv);
      unpack(rt, tv);
      unpack(rz, zv);
      unpack(ro, ov);
#pragma unroll
      for (int i = 0; i < SV; ++i) {
        float ex, d = softplus(tv[i] + bias[i], ex);
        if (tok >= nt) d = 0.f;
        s_dx[tok][sc + i * sstep] = make_float2(d, d * xv[i]);
        s_dy[tok][sc + i * sstep] = p.z ? ov[i] * zv[i] * sigmoid(zv[i]) : ov[i];
      }
    }
    if (tid < kScanBlock * LPC) {
      const int tok = tid / LPC;
      Raw<T, SP> rb = {}, rc = {};
      if (tok < nt) {
        load_row<T, SP, VEC>(rb, static_cast<const T*>(p.B) + (t0 + tok) * p.b_s + grp * NS + l * SP, 1, SP);
        load_row<T, SP, VEC>(rc, static_cast<const T*>(p.C) + (t0 + tok) * p.c_s + grp * NS + l * SP, 1, SP);
      }
      float v[SP];
      unpack(rb, v);
#pragma unroll
      for (int i = 0; i < SP; ++i) s_b[tok][l * SP + i] = v[i];
      unpack(rc, v);
#pragma unroll
      for (int i = 0; i < SP; ++i) s_c[tok][l * SP + i] = v[i];
    }
    if (mine) {
      const int64_t chunk = u.bos / kScanBlock + u.n + (t0 - u.bos) / kScanBlock;
      load_state<SP>(h0, p.chunk_states, chunk * st_seq + st_at, false);
    } else {
#pragma unroll
      for (int i = 0; i < SP; ++i) h0[i] = 0.f;
    }
    __syncthreads();

    // ---- forward over the block: a checkpoint before every piece but the first
    const int pieces = (nt + SB - 1) / SB;
    float h[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) h[i] = h0[i];
    auto step = [&](int tok, float (&a)[SP]) {
      const float2 d = s_dx[tok][c];
#pragma unroll
      for (int i = 0; i < SP; i += 2) {
        const float2 b2 = *reinterpret_cast<const float2*>(&s_b[tok][l * SP + i]);
        const float2 e = ptx::f2mul(make_float2(d.x, d.x), make_float2(A2[i], A2[i + 1]));
        a[i] = ptx::ex2_approx(e.x), a[i + 1] = ptx::ex2_approx(e.y);
        const float2 hn = ptx::f2fma(make_float2(a[i], a[i + 1]), make_float2(h[i], h[i + 1]),
                                     ptx::f2mul(make_float2(d.y, d.y), b2));
        h[i] = hn.x, h[i + 1] = hn.y;
      }
    };
    for (int k = 0; k + 1 < pieces; ++k) {
      float a[SP];
#pragma unroll
      for (int j = 0; j < SB; ++j) step(k * SB + j, a);
#pragma unroll
      for (int i = 0; i < SP; i += 4)
        *reinterpret_cast<float4*>(&s_ck[(k * NT + tid) * SP + i]) =
            make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    }
    // ---- the pieces in reverse
    for (int k = pieces - 1; k >= 0; --k) {
#pragma unroll
      for (int i = 0; i < SP; ++i) h[i] = k ? s_ck[((k - 1) * NT + tid) * SP + i] : h0[i];
      float a[SB][SP], hp[SB][SP];
#pragma unroll
      for (int j = 0; j < SB; ++j) {
#pragma unroll
        for (int i = 0; i < SP; ++i) hp[j][i] = h[i];
        step(k * SB + j, a[j]);
      }
      constexpr int L = SB < LPC ? SB : LPC;   // tokens whose state sums are reduced together
      constexpr int GT = 16 / (2 * SP);        // tokens whose channel sums are
      float qv[L], sv[L], yv[L], bc[16];
#pragma unroll
      for (int j = SB - 1; j >= 0; --j) {
        const int tok = k * SB + j;
        const float2 d = s_dx[tok][c];
        const float dy = s_dy[tok][c];
        float2 q2 = make_float2(0.f, 0.f), s2 = q2, y2 = q2;
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
          const float2 b2 = *reinterpret_cast<const float2*>(&s_b[tok][l * SP + i]);
          const float2 c2 = *reinterpret_cast<const float2*>(&s_c[tok][l * SP + i]);
          const float2 ht = j == SB - 1 ? make_float2(h[i], h[i + 1])
                                        : make_float2(hp[(j + 1) % SB][i], hp[(j + 1) % SB][i + 1]);
          float2 g2 = ptx::f2fma(make_float2(dy, dy), c2, make_float2(g[i], g[i + 1]));
          const float2 vb = ptx::f2mul(make_float2(d.y, d.y), g2);
          const float2 vc = ptx::f2mul(make_float2(dy, dy), ht);
          const int at = (j % GT) * 2 * SP + i;
          bc[at] = vb.x, bc[at + 1] = vb.y;
          bc[at + SP] = vc.x, bc[at + SP + 1] = vc.y;
          q2 = ptx::f2fma(g2, b2, q2);
          y2 = ptx::f2fma(c2, ht, y2);
          g2 = ptx::f2mul(g2, make_float2(a[j][i], a[j][i + 1]));
          const float2 w2 = ptx::f2mul(g2, make_float2(hp[j][i], hp[j][i + 1]));
          s2 = ptx::f2fma(w2, make_float2(A2[i], A2[i + 1]), s2);
          const float2 da = ptx::f2fma(w2, make_float2(d.x, d.x), make_float2(dA[i], dA[i + 1]));
          dA[i] = da.x, dA[i + 1] = da.y;
          g[i] = g2.x, g[i + 1] = g2.y;
        }
        qv[j % L] = q2.x + q2.y, sv[j % L] = s2.x + s2.y, yv[j % L] = y2.x + y2.y;
        if (j % GT == 0) {  // sums over the warp's channels
          int off = 0;
          reduce_scatter<16, 16, LPC>(bc, lane, off);
          constexpr int LEFT = 16 / H::CL > 0 ? 16 / H::CL : 1;
#pragma unroll
          for (int i = 0; i < LEFT; ++i) {
            const int o = off + i;
            const int tk = j + o / (2 * SP), kind = o / SP % 2;
            s_part[(warp * SB + tk) * 2 * NS + kind * NS + l * SP + o % SP] = bc[i];
          }
        }
        if (j % L == 0) {  // sums over the channel's states: one token per lane
          int off = 0;
          reduce_scatter<L, LPC / 2, 1>(qv, lane, off);
          off = 0;
          reduce_scatter<L, LPC / 2, 1>(sv, lane, off);
          off = 0;
          reduce_scatter<L, LPC / 2, 1>(yv, lane, off);
          __syncwarp();  // the channel's lanes are done with these tokens
          s_dx[k * SB + j + off][c] = make_float2(qv[0], sv[0] * kLn2);
          s_dy[k * SB + j + off][c] = yv[0];
        }
      }
      __syncthreads();
      for (int e = tid; e < SB * 2 * NS; e += NT) {  // over the CTA's warps
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += s_part[w * SB * 2 * NS + e];
        const int tk = k * SB + e / (2 * NS);
        if (tk < nt) p.part_bc[((int64_t)tile * p.total + t0 + tk) * 2 * NS + e % (2 * NS)] = v;
      }
      __syncthreads();
    }
    // ---- the gradients of the block's rows
#pragma unroll
    for (int q = 0; q < SN; ++q) {
      const int tok = (q * NT + tid) / PER_ROW;
      const int64_t t = t0 + tok;
      if (tok >= nt || sleft <= 0) continue;
      Raw<T, SV> rx = {}, rt = {}, rz = {}, ro = {};
      load_row<T, SV, VEC>(rx, static_cast<const T*>(p.x) + t * p.x_s + ch0 + sc, sstep, sleft);
      load_row<T, SV, VEC>(rt, static_cast<const T*>(p.dt) + t * p.dt_s + ch0 + sc, sstep, sleft);
      if (p.z)
        load_row<T, SV, VEC>(rz, static_cast<const T*>(p.z) + t * p.z_s + ch0 + sc, sstep, sleft);
      load_row<T, SV, VEC>(ro, static_cast<const T*>(p.dout) + t * p.dim + ch0 + sc, sstep, sleft);
      float xv[SV], tv[SV], zv[SV], ov[SV], dx[SV], dt[SV], dz[SV];
      unpack(rx, xv);
      unpack(rt, tv);
      unpack(rz, zv);
      unpack(ro, ov);
#pragma unroll
      for (int i = 0; i < SV; ++i) {
        const float2 qs = s_dx[tok][sc + i * sstep];
        float ex;
        const float d = softplus(tv[i] + bias[i], ex);
        const float sig = softplus_slope(tv[i] + bias[i], ex);
        float dy = ov[i];
        dz[i] = 0.f;
        if (p.z) {
          const float sz = sigmoid(zv[i]);
          dy *= zv[i] * sz;
          const float y = fmaf(dsk[i], xv[i], s_dy[tok][sc + i * sstep]);
          dz[i] = ov[i] * y * sz * fmaf(zv[i], 1.f - sz, 1.f);
        }
        dx[i] = fmaf(d, qs.x, dy * dsk[i]);
        dt[i] = fmaf(xv[i], qs.x, qs.y) * sig;
        sum_d[i] = fmaf(dy, xv[i], sum_d[i]);
        sum_b[i] += dt[i];
      }
      const int64_t at = t * p.dim + ch0 + sc;
      store_row<T, SV, VEC>(static_cast<T*>(p.dx) + at, dx, sstep, sleft);
      store_row<T, SV, VEC>(static_cast<T*>(p.ddt) + at, dt, sstep, sleft);
      if (p.dz) store_row<T, SV, VEC>(static_cast<T*>(p.dz) + at, dz, sstep, sleft);
    }
    __syncthreads();
  }
  // ---- what is summed over tokens: a partial row per slot
  float* const par = p.part_par + slot * (int64_t)p.dim * (NS + 2);
  if (mine) {
#pragma unroll
    for (int i = 0; i < SP; ++i) par[st_at + i] = dA[i] * A2[i] * kLn2;
    if (u.live && u.first && p.dinit) store_state<SP>(p.dinit, u.n * st_seq + st_at, g, false);
  }
  float(*s_red)[CH] = reinterpret_cast<float(*)[CH]>(sm);  // [NT / PER_ROW][CH], twice
  constexpr int ROWS = NT / PER_ROW;
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    s_red[tid / PER_ROW][sc + i * sstep] = sum_d[i];
    s_red[ROWS + tid / PER_ROW][sc + i * sstep] = sum_b[i];
  }
  __syncthreads();
  for (int e = tid; e < 2 * CH; e += NT) {
    const int cc = e % CH, k = e / CH;
    float v = 0.f;
    for (int r = 0; r < ROWS; ++r) v += s_red[k * ROWS + r][cc];
    if (cc < c_n) par[st_seq + k * (int64_t)p.dim + ch0 + cc] = v;
  }
}

// The gradient that leaves a segment at its start, from a zero gradient at its end (the
// last segment: from dfinal_state), and the segment's sum of delta.
template <typename T, int NS, bool VEC>
__global__ void __launch_bounds__(kRevCh * NS / kStates<NS>)
    scan_rev_kernel(const ScanParams p) {
  constexpr int SP = kStates<NS>, LPC = NS / SP, CH = kRevCh, NT = CH * LPC;
  constexpr int EPT = kScanBlock * CH / NT, SV = EPT < 8 ? EPT : 8, SN = EPT / SV;
  constexpr int PER_ROW = CH / SV;
  __shared__ float2 s_d[kScanBlock][CH];  // delta, dy
  __shared__ __align__(16) float s_c[kScanBlock][NS];
  const int tid = threadIdx.x;
  const int tpg = (p.per + CH - 1) / CH;
  const int64_t tiles = (int64_t)tpg * p.groups;
  const int64_t slot = blockIdx.x / tiles;
  const int tile = (int)(blockIdx.x % tiles);
  const Segment u = find_unit(p, slot);
  if (!u.live || u.first) return;  // nothing before the first segment asks for its gradient
  const int grp = tile / tpg, c_lo = (tile % tpg) * CH, c_n = min(CH, p.per - c_lo);
  const int64_t ch0 = (int64_t)grp * p.per + c_lo, st_seq = (int64_t)p.dim * NS;
  const int c = tid / LPC, l = tid % LPC;
  const bool mine = c < c_n;
  const int64_t st_at = (ch0 + c) * NS + l * SP;
  float A2[SP], g[SP], sum_delta = 0.f;
#pragma unroll
  for (int i = 0; i < SP; ++i) A2[i] = g[i] = 0.f;
  if (mine) {
    load_rates<SP>(A2, p.A_log, st_at);
    if (u.last && p.dfin) load_state<SP>(g, p.dfin, u.n * st_seq + st_at, p.state_bf16);
  }
  const int sc = VEC ? (tid % PER_ROW) * SV : tid % PER_ROW;
  const int sstep = VEC ? 1 : PER_ROW;
  const int64_t sleft = VEC ? (sc < c_n ? CH : 0) : c_n - sc;
  for (int64_t blk = (u.t1 - u.t0 + kScanBlock - 1) / kScanBlock - 1; blk >= 0; --blk) {
    const int64_t t0 = u.t0 + blk * kScanBlock;
    const int nt = (int)min((int64_t)kScanBlock, u.t1 - t0);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < SN; ++q) {
      const int tok = (q * NT + tid) / PER_ROW;
      Raw<T, SV> rt = {}, rz = {}, ro = {};
      const int64_t t = t0 + tok;
      if (tok < nt && sleft > 0) {
        load_row<T, SV, VEC>(rt, static_cast<const T*>(p.dt) + t * p.dt_s + ch0 + sc, sstep, sleft);
        if (p.z)
          load_row<T, SV, VEC>(rz, static_cast<const T*>(p.z) + t * p.z_s + ch0 + sc, sstep, sleft);
        load_row<T, SV, VEC>(ro, static_cast<const T*>(p.dout) + t * p.dim + ch0 + sc, sstep, sleft);
      }
      float tv[SV], zv[SV], ov[SV];
      unpack(rt, tv);
      unpack(rz, zv);
      unpack(ro, ov);
#pragma unroll
      for (int i = 0; i < SV; ++i) {
        const int cc = sc + i * sstep;
        float ex;
        const float d =
            softplus(tv[i] + (cc < c_n && p.dt_bias ? __ldg(p.dt_bias + ch0 + cc) : 0.f), ex);
        s_d[tok][cc] = make_float2(tok < nt ? d : 0.f,
                                   p.z ? ov[i] * zv[i] * sigmoid(zv[i]) : ov[i]);
      }
    }
    {
      const int tok = tid / LPC;
      Raw<T, SP> rc = {};
      if (tok < nt)
        load_row<T, SP, VEC>(rc, static_cast<const T*>(p.C) + (t0 + tok) * p.c_s + grp * NS + l * SP, 1, SP);
      float v[SP];
      unpack(rc, v);
#pragma unroll
      for (int i = 0; i < SP; ++i) s_c[tok][l * SP + i] = v[i];
    }
    __syncthreads();
#pragma unroll 4
    for (int tok = kScanBlock - 1; tok >= 0; --tok) {
      const float2 d = s_d[tok][c];
      sum_delta += d.x;
#pragma unroll
      for (int i = 0; i < SP; i += 2) {
        const float2 c2 = *reinterpret_cast<const float2*>(&s_c[tok][l * SP + i]);
        const float2 e = ptx::f2mul(make_float2(d.x, d.x), make_float2(A2[i], A2[i + 1]));
        const float2 a = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
        const float2 gn = ptx::f2mul(
            a, ptx::f2fma(make_float2(d.y, d.y), c2, make_float2(g[i], g[i + 1])));
        g[i] = gn.x, g[i + 1] = gn.y;
      }
    }
  }
  if (!mine) return;
  store_state<SP>(p.seg_state, slot * st_seq + st_at, g, false);
  if (l == 0) p.seg_sum[slot * p.dim + ch0 + c] = sum_delta;
}

// Carries the gradients over a sequence's segments, last to first: in place, the gradient
// leaving segment s becomes the one entering it from behind (0 for the last, which starts
// from dfinal_state itself).
__global__ void scan_rev_carry_kernel(const ScanParams p, int state) {
  const int64_t st_seq = (int64_t)p.dim * state;
  const int64_t blocks = (st_seq + blockDim.x - 1) / blockDim.x;
  const int n = (int)(blockIdx.x / blocks);
  const int64_t i = (blockIdx.x % blocks) * blockDim.x + threadIdx.x;
  if (i >= st_seq) return;
  int64_t bos, eos;
  seq_bounds(p, n, bos, eos);
  const int64_t ns = (eos - bos + p.seg_len - 1) / p.seg_len, slot = first_slot(p, n);
  const float A2 = rate_of(__ldg(p.A_log + i));
  const int64_t ch = i / state;
  float g = 0.f;
  constexpr int kAhead = 8;
  for (int64_t s = ns - 1; s >= 0; s -= kAhead) {
    float e[kAhead], d[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool ok = s - k > 0;
      e[k] = ok ? p.seg_state[(slot + s - k) * st_seq + i] : 0.f;
      d[k] = ok ? p.seg_sum[(slot + s - k) * p.dim + ch] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (s - k < 0) break;
      p.seg_state[(slot + s - k) * st_seq + i] = g;
      g = s - k == ns - 1 ? e[k] : fmaf(exp2f(A2 * d[k]), g, e[k]);
    }
  }
}

// dB and dC: the partial sums of a group's channel tiles, added in their order; zeros for
// the tokens of no sequence.
template <typename T>
__global__ void scan_bc_kernel(const ScanParams p, int state, T* dB, T* dC) {
  const int w = 2 * state;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;  // over [total][groups][w]
  if (i >= p.total * p.groups * w) return;
  const int e = (int)(i % w);
  const int grp = (int)(i / w % p.groups);
  const int64_t t = i / ((int64_t)w * p.groups);
  float v = 0.f;
  if (!p.cu || t < __ldg(p.cu + p.N)) {
#pragma unroll 8
    for (int k = 0; k < p.tiles_per_group; ++k)
      v += p.part_bc[((int64_t)(grp * p.tiles_per_group + k) * p.total + t) * w + e];
  }
  T* out = e < state ? dB : dC;
  out[(t * p.groups + grp) * state + e % state] = from_f<T>(v);
}

template <typename T, int NS, bool VEC>
cudaError_t launch_bwd_ns(const ScanParams& p, int64_t tail, cudaStream_t stream) {
  using H = BwdShape<T, NS>;
  static bool done[64];
  const int bytes = H::FLOATS * (int)sizeof(float);
  const cudaError_t e = ensure_smem_attr(
      reinterpret_cast<const void*>(scan_bwd_kernel<T, NS, VEC>), bytes, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = p.slots * p.tiles + tail;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  if (grid > 0) scan_bwd_kernel<T, NS, VEC><<<(unsigned)grid, H::NT, bytes, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int NS, bool VEC>
cudaError_t launch_rev_ns(const ScanParams& p, cudaStream_t stream) {
  const int64_t grid = (int64_t)((p.per + kRevCh - 1) / kRevCh) * p.groups * p.slots;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  scan_rev_kernel<T, NS, VEC>
      <<<(unsigned)grid, kRevCh * NS / kStates<NS>, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch_bwd(const ScanParams& p, int state, bool rev, int64_t tail, cudaStream_t s) {
  switch (state) {
    case 8: return rev ? launch_rev_ns<T, 8, VEC>(p, s) : launch_bwd_ns<T, 8, VEC>(p, tail, s);
    case 16: return rev ? launch_rev_ns<T, 16, VEC>(p, s) : launch_bwd_ns<T, 16, VEC>(p, tail, s);
    case 32: return rev ? launch_rev_ns<T, 32, VEC>(p, s) : launch_bwd_ns<T, 32, VEC>(p, tail, s);
    default: return rev ? launch_rev_ns<T, 64, VEC>(p, s) : launch_bwd_ns<T, 64, VEC>(p, tail, s);
  }
}

cudaError_t launch_bwd_pass(const ScanParams& p, int state, bool f32, bool vec, bool rev,
                            int64_t tail, cudaStream_t s) {
  if (f32) return vec ? launch_bwd<float, true>(p, state, rev, tail, s)
                      : launch_bwd<float, false>(p, state, rev, tail, s);
  return vec ? launch_bwd<bf16, true>(p, state, rev, tail, s)
             : launch_bwd<bf16, false>(p, state, rev, tail, s);
}

bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The backward's tiles and plan, and its workspace: offsets behind the status word.
struct BwdLayout {
  size_t fwd, states, seg, bc, par, total;
};

BwdLayout bwd_layout(ScanParams& p, int state, bool have_states) {
  BwdLayout w;
  size_t at = KDA_STATUS_BYTES;
  ScanParams f = p;
  scan_fwd_plan(f, state);
  w.fwd = at;
  if (!have_states) at = up256(at + fwd_ws_bytes(f, state));
  w.states = at;
  size_t n = 0;
  kda_scan_get_states_size(p.total, p.N, p.dim, state, &n);
  if (!have_states) at = up256(at + n);
  const int ch = state == 64 ? kBwdCh<64> : kBwdCh<16>;
  p.tiles_per_group = (p.per + ch - 1) / ch;
  p.tiles = (int64_t)p.tiles_per_group * p.groups;
  // 2 CTAs of 256 threads per SM at the kernel's registers and shared memory
  const ScanPlan r = scan_plan(p, p.tiles, 1, 2);
  p.seg_len = r.seg_len, p.slots = r.slots;
  w.seg = at;
  if (p.seg_len) at = up256(at + (size_t)p.slots * p.dim * (state + 1) * sizeof(float));
  w.bc = at;
  at = up256(at + (size_t)p.tiles * p.total * 2 * state * sizeof(float));
  w.par = at;
  at += (size_t)p.slots * p.dim * (state + 2) * sizeof(float);
  w.total = at;
  return w;
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_scan_bwd_get_workspace_size(const kda_scan_problem* problem, int32_t have_states,
                                           size_t* bytes) {
  using namespace kda;
  if (!bytes) return KDA_ERR_NULL_POINTER;
  scan::ScanParams p;
  const kda_status st = scan::check_scan_sizes(problem, p);
  if (st != KDA_OK) return st;
  *bytes = bwd_layout(p, problem->state, have_states != 0).total;
  return KDA_OK;
}

kda_status kda_scan_bwd(const kda_scan_problem* problem, const void* dout,
                        const void* dfinal_state, const void* chunk_states,
                        size_t chunk_states_bytes, void* dx, void* ddt, void* dz, void* dB,
                        void* dC, float* dA_log, float* dD, float* ddt_bias,
                        float* dinitial_state, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  using namespace kda;
  scan::ScanParams p;
  bool vec = false;
  kda_status st = scan::check_scan(problem, p, vec);
  if (st != KDA_OK) return st;
  const bool f32 = problem->dtype == KDA_ROW_FP32;
  const size_t e = f32 ? 4 : 2;
  const int state = problem->state;
  if (!workspace || !dA_log || (p.total > 0 && (!dout || !dx || !ddt || !dB || !dC)))
    return KDA_ERR_NULL_POINTER;
  if ((dz && !p.z) || (dD && !p.D) || (ddt_bias && !p.dt_bias)) return KDA_ERR_INVALID_ARG;
  if (!al_to(dout, e) || !al_to(dx, e) || !al_to(ddt, e) || !al_to(dz, e) || !al_to(dB, e) ||
      !al_to(dC, e) || !al_to(dA_log, 4) || !al_to(dD, 4) || !al_to(ddt_bias, 4) ||
      !al_to(dfinal_state, 16) || !al_to(dinitial_state, 16) || !al_to(chunk_states, 16) ||
      !al_to(workspace, 128))
    return KDA_ERR_MISALIGNED;
  if (chunk_states) {
    size_t need = 0;
    kda_scan_get_states_size(p.total, p.N, p.dim, state, &need);
    if (chunk_states_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  }
  scan::ScanParams f = p;
  const BwdLayout w = bwd_layout(p, state, chunk_states != nullptr);
  if (workspace_bytes < w.total) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  vec = vec && al_to(dout, 16) && al_to(dx, 16) && al_to(ddt, 16) && al_to(dz, 16);
  if (!chunk_states) {
    scan::scan_fwd_plan(f, state);
    scan::carve_fwd(f, state, ws + w.fwd);
    f.chunk_states = reinterpret_cast<float*>(ws + w.states);
    if (scan::launch_scan_fwd(f, state, f32, vec, false, stream) != cudaSuccess)
      return KDA_ERR_CUDA;
  }
  p.chunk_states = chunk_states ? static_cast<float*>(const_cast<void*>(chunk_states))
                                : reinterpret_cast<float*>(ws + w.states);
  p.dout = dout, p.dfin = dfinal_state, p.dx = dx, p.ddt = ddt, p.dz = dz;
  p.dinit = dinitial_state;
  p.part_bc = reinterpret_cast<float*>(ws + w.bc);
  p.part_par = reinterpret_cast<float*>(ws + w.par);
  if (p.seg_len) {
    p.seg_state = reinterpret_cast<float*>(ws + w.seg);
    p.seg_sum = p.seg_state + p.slots * p.dim * state;
    if (launch_bwd_pass(p, state, f32, vec, true, 0, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const int64_t grid = ((int64_t)p.dim * state + 127) / 128 * p.N;
    if (grid >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
    scan_rev_carry_kernel<<<(unsigned)grid, 128, 0, stream>>>(p, state);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  }
  if (launch_bwd_pass(p, state, f32, vec, false, p.cu ? 32 : 0, stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  if (p.total > 0) {
    const int64_t grid = (p.total * p.groups * 2 * state + 255) / 256;
    if (f32)
      scan_bc_kernel<float><<<(unsigned)grid, 256, 0, stream>>>(
          p, state, static_cast<float*>(dB), static_cast<float*>(dC));
    else
      scan_bc_kernel<scan::bf16><<<(unsigned)grid, 256, 0, stream>>>(
          p, state, static_cast<scan::bf16*>(dB), static_cast<scan::bf16*>(dC));
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  }
  const int64_t n = (int64_t)p.dim * state;
  if (launch_column_sums(p.part_par, p.slots, n + 2 * (int64_t)p.dim, n, p.dim, dA_log, dD,
                         ddt_bias, stream) != cudaSuccess ||
      seqlens_status(p, static_cast<unsigned*>(workspace), stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"
