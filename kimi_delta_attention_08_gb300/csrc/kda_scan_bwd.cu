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
// Per (token, channel, state) this takes two exponentials and 15 multiply-adds, in packed
// pairs of channels, and about as many other instructions (shared-memory reads, the sums over
// channels and over states), so it is bound by the rate at which a scheduler issues: about
// 0.5 instructions a clock, a packed one taking two or three.  4 sequences of 4,096 tokens,
// 4,096 channels, 16 states in bf16: 1.69 ms, 2.27 with the forward that saves the states
// (0.65 TB/s; fp32 2.41); the exponentials alone would take 0.23 ms.  At 168 registers the
// kernels for 8 and 16 states spill 68 to 128 bytes.  As in the forward, sequences are cut
// into segments where channels alone do not fill the GPU: a reverse pass computes each
// segment's gradient at its start from a zero gradient at its end, and a second launch
// carries the gradients over the segments.
#include <cstring>

#include "kda_scan.cuh"

namespace kda {
namespace {

using namespace scan;

// Floats of a slot's row of partial sums [dim][state], [dim], [dim]: whole 16-byte units.
__host__ __device__ __forceinline__ int64_t par_pitch(int64_t dim, int state) {
  return (dim * (state + 2) + 3) / 4 * 4;
}

// A thread holds SP states of two neighbouring channels, as pairs.
template <typename T, int NS>
struct BwdShape {
  static constexpr int SP = 4, LPC = NS / SP, NT = NS >= 32 ? 256 : 128, NW = NT / 32;
  static constexpr int CL = 32 / LPC;                         // channel pairs per warp
  static constexpr int CH = 2 * CL * NW;                      // channels per CTA
  static constexpr int SB = 4, NSB = kScanBlock / SB;         // tokens per piece, pieces
  static constexpr int EPT = kScanBlock * CH / NT, SV = EPT < 8 ? EPT : 8, SN = EPT / SV;
  static constexpr int PER_ROW = CH / SV;
  static constexpr int BV = kScanBlock * NS / NT;             // of B and of C staged per thread
  // shared memory, in floats
  static constexpr int DX = 0;                                // [32][CH / 2] of (delta, delta',
                                                              // delta x, delta' x'), then (q, q',
                                                              // s, s') of done tokens
  static constexpr int DY = DX + 2 * kScanBlock * CH;         // [32][CH]: dy, then y
  static constexpr int SB_ = DY + kScanBlock * CH;            // B [32][NS], each value twice
  static constexpr int SC_ = SB_ + 2 * kScanBlock * NS;       // C
  static constexpr int PART = SC_ + 2 * kScanBlock * NS;      // [2][NW][SB][2 NS]
  static constexpr int CKPT = PART + 2 * NW * SB * 2 * NS;        // [NSB - 1][2][NT] of 4
  static constexpr int SUMA = CKPT + (NSB - 1) * 2 * 4 * NT;  // [2][NT] of 4
  static constexpr int FLOATS = SUMA + 2 * 4 * NT;
  // CTAs on an SM, by registers (12 warps) and by shared memory: 2 with 8 states, 3 with 16, 1
  // with 32 and 64
  static constexpr int BY_SMEM = 228 * 1024 / (FLOATS * 4 + 1024);
  static constexpr int RESIDENT = 384 / NT < BY_SMEM ? 384 / NT : BY_SMEM;
};

// The channels of a CTA and the CTAs on an SM.
struct BwdFit {
  int channels, resident;
};
template <int NS>
BwdFit bwd_fit_of() {
  return {BwdShape<float, NS>::CH, BwdShape<float, NS>::RESIDENT};
}
BwdFit bwd_fit(int state) {
  return state == 8 ? bwd_fit_of<8>() : state == 16 ? bwd_fit_of<16>() : state == 32 ? bwd_fit_of<32>()
                                                                                     : bwd_fit_of<64>();
}

// Where the 16 bytes of a channel pair lie in a token's row of DX: exchanged within groups
// of four, so that the staging writes (neighbouring lanes 64 bytes apart, two rows in 8
// lanes) use every bank once, as the reads do anyway.
__device__ __forceinline__ int pair_unit(int tok, int u) {
  return u ^ ((u >> 3 & 1) | (tok & 1) << 1);
}

template <typename T, int NS, bool VEC>
__global__ void __launch_bounds__(BwdShape<T, NS>::NT, 384 / BwdShape<T, NS>::NT)
    scan_bwd_kernel(const ScanParams p) {
  using H = BwdShape<T, NS>;
  constexpr int CH = H::CH, SP = H::SP, LPC = H::LPC, NT = H::NT, NW = H::NW, SB = H::SB;
  constexpr int CL = H::CL, SV = H::SV, SN = H::SN, PER_ROW = H::PER_ROW, BV = H::BV;
  extern __shared__ __align__(16) float sm[];
  float4(*s_dx)[CH / 2] = reinterpret_cast<float4(*)[CH / 2]>(sm + H::DX);
  float(*s_dy)[CH] = reinterpret_cast<float(*)[CH]>(sm + H::DY);
  pair(*s_b)[NS] = reinterpret_cast<pair(*)[NS]>(sm + H::SB_);
  pair(*s_c)[NS] = reinterpret_cast<pair(*)[NS]>(sm + H::SC_);
  float* const s_part = sm + H::PART;
  float4* const s_ck = reinterpret_cast<float4*>(sm + H::CKPT);
  float4* const s_da = reinterpret_cast<float4*>(sm + H::SUMA);

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
  const int64_t slot = blockIdx.x / (unsigned)p.tiles;
  const int tile = (int)(blockIdx.x % (unsigned)p.tiles);
  const Segment u = find_unit(p, slot);
  const int grp = tile / p.tiles_per_group;
  const int c_lo = (tile % p.tiles_per_group) * CH;
  const int c_n = min(CH, p.per - c_lo);
  const int64_t ch0 = (int64_t)grp * p.per + c_lo;
  const int cp = warp * CL + lane_channel<LPC>(lane), l = lane_part<LPC>(lane);
  const int left = max(0, min(2, c_n - 2 * cp));  // channels of the thread's pair that exist
  const int64_t st_at = (ch0 + 2 * cp) * NS + l * SP;

  // a state array of the thread's two channels, from [dim][NS]
  auto get_pairs = [&](pair (&v)[SP], const void* from, int64_t at, bool b16) {
    float f[2][SP] = {};
    if (left > 0) load_state<SP>(f[0], from, at + st_at, b16);
    if (left > 1) load_state<SP>(f[1], from, at + st_at + NS, b16);
#pragma unroll
    for (int i = 0; i < SP; ++i) v[i] = pr(f[0][i], f[1][i]);
  };
  pair A2[SP], g[SP], h0[SP];
  {
    float a[2][SP] = {};
    if (left > 0) load_rates<SP>(a[0], p.A_log, st_at);
    if (left > 1) load_rates<SP>(a[1], p.A_log, st_at + NS);
#pragma unroll
    for (int i = 0; i < SP; ++i) A2[i] = pr(a[0][i], a[1][i]), g[i] = 0;
  }
  if (u.live && u.last) {
    if (p.dfin) get_pairs(g, p.dfin, u.n * st_seq, p.state_bf16);
  } else if (u.live) {
    get_pairs(g, p.seg_state, slot * st_seq, false);
  }
  s_da[tid] = s_da[NT + tid] = make_float4(0.f, 0.f, 0.f, 0.f);  // read by this thread alone
  const int sc = VEC ? (tid % PER_ROW) * SV : tid % PER_ROW;
  const int sstep = VEC ? 1 : PER_ROW;
  const int64_t sleft = VEC ? (sc < c_n ? CH : 0) : c_n - sc;
  const int btok = tid / (NS / BV), bn = tid % (NS / BV) * BV;
  float bias[SV], dsk[SV], sum_d[SV], sum_b[SV];
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    const int cc = sc + i * sstep;
    bias[i] = cc < c_n && p.dt_bias ? __ldg(p.dt_bias + ch0 + cc) : 0.f;
    dsk[i] = cc < c_n && p.D ? __ldg(p.D + ch0 + cc) : 0.f;
    sum_d[i] = sum_b[i] = 0.f;
  }
  const int u_even = pair_unit(0, cp), u_odd = pair_unit(1, cp);

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
      for (int i = 0; i < SV; i += 2) {
        pair ex;
        pair d = softplus(padd(pr(tv[i], tv[i + 1]), pr(bias[i], bias[i + 1])), ex);
        d = tok < nt ? d : 0;
        const pair m = pmul(d, pr(xv[i], xv[i + 1]));
        pair dy = pr(ov[i], ov[i + 1]);
        if (p.z) dy = pmul(dy, silu<T>(pr(zv[i], zv[i + 1])));
        if constexpr (VEC) {
          *reinterpret_cast<ulonglong2*>(&s_dx[tok][pair_unit(tok, (sc + i) / 2)]) = make_ulonglong2(d, m);
          *reinterpret_cast<pair*>(&s_dy[tok][sc + i]) = dy;
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int cc = sc + (i + k) * sstep;
            float* const unit = &s_dx[tok][pair_unit(tok, cc / 2)].x;
            unit[cc & 1] = k ? un(d).y : un(d).x;
            unit[2 + (cc & 1)] = k ? un(m).y : un(m).x;
            s_dy[tok][cc] = k ? un(dy).y : un(dy).x;
          }
        }
      }
    }
    {
      Raw<T, BV> rb = {}, rc = {};
      if (btok < nt) {
        load_row<T, BV, VEC>(rb, static_cast<const T*>(p.B) + (t0 + btok) * p.b_s + grp * NS + bn, 1, BV);
        load_row<T, BV, VEC>(rc, static_cast<const T*>(p.C) + (t0 + btok) * p.c_s + grp * NS + bn, 1, BV);
      }
      float v[BV];
      unpack(rb, v);
#pragma unroll
      for (int i = 0; i < BV; ++i) s_b[btok][bn + i] = pr(v[i]);
      unpack(rc, v);
#pragma unroll
      for (int i = 0; i < BV; ++i) s_c[btok][bn + i] = pr(v[i]);
    }
    get_pairs(h0, p.chunk_states, (u.bos / kScanBlock + u.n + (t0 - u.bos) / kScanBlock) * st_seq, false);
    __syncthreads();

    // ---- forward over the block: a checkpoint before every piece but the first
    const int pieces = (nt + SB - 1) / SB;
    pair h[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) h[i] = h0[i];
    auto step = [&](int tok, int unit, pair (&a)[SP]) {
      const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s_dx[tok][unit]);
#pragma unroll
      for (int i = 0; i < SP; i += 2) {
        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(&s_b[tok][l * SP + i]);
        a[i] = decay(d.x, A2[i]), a[i + 1] = decay(d.x, A2[i + 1]);
        h[i] = pfma(a[i], h[i], pmul(d.y, b2.x));
        h[i + 1] = pfma(a[i + 1], h[i + 1], pmul(d.y, b2.y));
      }
    };
    for (int k = 0; k + 1 < pieces; ++k) {
      pair a[SP];
#pragma unroll
      for (int j = 0; j < SB; ++j) step(k * SB + j, j & 1 ? u_odd : u_even, a);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<ulonglong2*>(&s_ck[(k * 2 + q) * NT + tid]) = make_ulonglong2(h[2 * q], h[2 * q + 1]);
    }
    // ---- the pieces in reverse
    pair dA[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) dA[i] = 0;
    for (int k = pieces - 1; k >= 0; --k) {
      if (k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s_ck[((k - 1) * 2 + q) * NT + tid]);
          h[2 * q] = v.x, h[2 * q + 1] = v.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < SP; ++i) h[i] = h0[i];
      }
      float* const part = s_part + (k & 1) * NW * SB * 2 * NS;
      pair a[SB][SP], hp[SB][SP];
#pragma unroll
      for (int j = 0; j < SB; ++j) {
#pragma unroll
        for (int i = 0; i < SP; ++i) hp[j][i] = h[i];
        step(k * SB + j, j & 1 ? u_odd : u_even, a[j]);
      }
      pair qv[SB], sv[SB], yv[SB];
#pragma unroll
      for (int j = SB - 1; j >= 0; --j) {
        const int tok = k * SB + j;
        const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(&s_dx[tok][j & 1 ? u_odd : u_even]);
        const pair dy = *reinterpret_cast<const pair*>(&s_dy[tok][2 * cp]);
        float bc[2 * SP];
        pair q2 = 0, s2 = 0, y2 = 0;
#pragma unroll
        for (int i = 0; i < SP; i += 2) {
          const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(&s_b[tok][l * SP + i]);
          const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(&s_c[tok][l * SP + i]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int n = i + e;
            const pair bn2 = e ? b2.y : b2.x, cn2 = e ? c2.y : c2.x;
            const pair ht = j == SB - 1 ? h[n] : hp[(j + 1) % SB][n];
            pair gn = pfma(dy, cn2, g[n]);
            const float2 vb = un(pmul(d.y, gn)), vc = un(pmul(dy, ht));
            bc[n] = vb.x + vb.y, bc[SP + n] = vc.x + vc.y;
            q2 = n ? pfma(gn, bn2, q2) : pmul(gn, bn2);
            y2 = n ? pfma(cn2, ht, y2) : pmul(cn2, ht);
            gn = pmul(gn, a[j][n]);
            const pair w = pmul(gn, hp[j][n]);
            s2 = n ? pfma(w, A2[n], s2) : pmul(w, A2[n]);
            dA[n] = pfma(w, d.x, dA[n]);
            g[n] = gn;
          }
        }
        qv[j] = q2, sv[j] = s2, yv[j] = y2;
        // over the warp's channels: lane bits 1 .. CL (see lane_channel)
        int off = 0;
        reduce_scatter<2 * SP, CL, 2>(bc, lane, off);
        constexpr int LEFT = 2 * SP / CL > 0 ? 2 * SP / CL : 1;
#pragma unroll
        for (int i = 0; i < LEFT; ++i) {
          const int o = off + i;
          part[(warp * SB + j) * 2 * NS + o / SP * NS + l * SP + o % SP] = bc[i];
        }
      }
      // over the channels' states: a token per lane
      constexpr int TOK = LPC < SB ? SB / LPC : 1;
      int off = 0;
      reduce_states<SB, LPC>(qv, lane, off);
      off = 0;
      reduce_states<SB, LPC>(sv, lane, off);
      off = 0;
      reduce_states<SB, LPC>(yv, lane, off);
      __syncwarp();  // the pair's lanes are done with these tokens
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
        const int tok = k * SB + off + j;
        *reinterpret_cast<ulonglong2*>(&s_dx[tok][pair_unit(tok, cp)]) =
            make_ulonglong2(qv[j], pmul(sv[j], pr(kLn2)));
        *reinterpret_cast<pair*>(&s_dy[tok][2 * cp]) = yv[j];
      }
      __syncthreads();
      for (int e = tid; e < SB * 2 * NS; e += NT) {  // over the CTA's warps
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) v += part[w * SB * 2 * NS + e];
        const int tk = k * SB + e / (2 * NS);
        if (tk < nt) p.part_bc[((int64_t)tile * p.total + t0 + tk) * 2 * NS + e % (2 * NS)] = v;
      }
    }
    __syncthreads();
    // a block's share of dA joins the rest in one addition
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ulonglong2* const to = reinterpret_cast<ulonglong2*>(&s_da[q * NT + tid]);
      const ulonglong2 v = *to;
      *to = make_ulonglong2(padd(v.x, dA[2 * q]), padd(v.y, dA[2 * q + 1]));
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
      for (int i = 0; i < SV; i += 2) {
        pair qi, si, yi;
        if constexpr (VEC) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s_dx[tok][pair_unit(tok, (sc + i) / 2)]);
          qi = v.x, si = v.y;
          yi = *reinterpret_cast<const pair*>(&s_dy[tok][sc + i]);
        } else {
          const int c0 = sc + i * sstep, c1 = c0 + sstep;
          const float* const u0 = &s_dx[tok][pair_unit(tok, c0 / 2)].x;
          const float* const u1 = &s_dx[tok][pair_unit(tok, c1 / 2)].x;
          qi = pr(u0[c0 & 1], u1[c1 & 1]), si = pr(u0[2 + (c0 & 1)], u1[2 + (c1 & 1)]);
          yi = pr(s_dy[tok][c0], s_dy[tok][c1]);
        }
        const pair x2 = pr(xv[i], xv[i + 1]), o2 = pr(ov[i], ov[i + 1]);
        const pair v = padd(pr(tv[i], tv[i + 1]), pr(bias[i], bias[i + 1]));
        pair ex, dy = o2, dz2 = 0;
        const pair d = softplus(v, ex);
        const pair sig = pr(softplus_slope(un(v).x, un(ex).x), softplus_slope(un(v).y, un(ex).y));
        const pair sk = pr(dsk[i], dsk[i + 1]);
        if (p.z) {
          const pair z2 = pr(zv[i], zv[i + 1]), sz = sigmoid<T>(z2), zs = pmul(z2, sz);
          dy = pmul(o2, zs);
          dz2 = pmul(pmul(o2, pfma(sk, x2, yi)), silu_slope(z2, sz));
        }
        const pair dx2 = pfma(d, qi, pmul(dy, sk)), dt2 = pmul(pfma(x2, qi, si), sig);
        const float2 sd = un(pmul(dy, x2));
        sum_d[i] += sd.x, sum_d[i + 1] += sd.y;
        dx[i] = un(dx2).x, dx[i + 1] = un(dx2).y;
        dt[i] = un(dt2).x, dt[i + 1] = un(dt2).y;
        dz[i] = un(dz2).x, dz[i + 1] = un(dz2).y;
        sum_b[i] += dt[i], sum_b[i + 1] += dt[i + 1];
      }
      const int64_t at = t * p.dim + ch0 + sc;
      store_row<T, SV, VEC>(static_cast<T*>(p.dx) + at, dx, sstep, sleft);
      store_row<T, SV, VEC>(static_cast<T*>(p.ddt) + at, dt, sstep, sleft);
      if (p.dz) store_row<T, SV, VEC>(static_cast<T*>(p.dz) + at, dz, sstep, sleft);
    }
    __syncthreads();
  }
  // ---- what is summed over tokens: a partial row per slot
  float* const par = p.part_par + slot * par_pitch(p.dim, NS);
  {
    float f[2][SP], gi[2][SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s_da[i / 2 * NT + tid]);
      const float2 da = un(pmul(i & 1 ? v.y : v.x, pmul(A2[i], pr(kLn2))));
      f[0][i] = da.x, f[1][i] = da.y;
      gi[0][i] = un(g[i]).x, gi[1][i] = un(g[i]).y;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (q >= left) break;
      store_state<SP>(par, st_at + q * NS, f[q], false);
      if (u.live && u.first && p.dinit) store_state<SP>(p.dinit, u.n * st_seq + st_at + q * NS, gi[q], false);
    }
  }
  __syncthreads();
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

template <typename T, bool VEC>
cudaError_t launch_bwd(const ScanParams& p, int state, int64_t tail, cudaStream_t s) {
  switch (state) {
    case 8: return launch_bwd_ns<T, 8, VEC>(p, tail, s);
    case 16: return launch_bwd_ns<T, 16, VEC>(p, tail, s);
    case 32: return launch_bwd_ns<T, 32, VEC>(p, tail, s);
    default: return launch_bwd_ns<T, 64, VEC>(p, tail, s);
  }
}

cudaError_t launch_bwd_pass(const ScanParams& p, int state, bool f32, bool vec, int64_t tail,
                            cudaStream_t s) {
  if (f32) return vec ? launch_bwd<float, true>(p, state, tail, s)
                      : launch_bwd<float, false>(p, state, tail, s);
  return vec ? launch_bwd<bf16, true>(p, state, tail, s)
             : launch_bwd<bf16, false>(p, state, tail, s);
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
  const BwdFit fit = bwd_fit(state);
  p.tiles_per_group = (p.per + fit.channels - 1) / fit.channels;
  p.tiles = (int64_t)p.tiles_per_group * p.groups;
  // The reverse pass that cutting adds costs a seventh of the main one, so sequences stay whole
  // where they fill nearly all of the turns that they take: 85 % with three CTAs on an SM, 80 %
  // with fewer.  Sequences of 4,096 channels, whole / cut: 16 states, 4,096 tokens, 6 (84 %)
  // 2,580 / 2,510 us, 7 (98 %) 2,589 / 2,987; 8 states, 2,048 tokens, 7 (74 %) 1,247 / 1,089,
  // 8 (84 %) 1,243 / 1,303; 32 states, 5 (70 %) 2,456 / 2,169, 2 (84 %) 843 / 931; 64 states, 1
  // (84 %) 918 / 1,014.
  const int64_t whole = scan_whole_units(p, p.tiles), turn = fit.resident * kSms;
  const int64_t enough = fit.resident == 3 ? 85 : 80;
  const bool cut = 100 * whole < enough * ((whole + turn - 1) / turn * turn);
  const ScanPlan r = scan_plan(p, p.tiles, fit.resident, cut);
  p.seg_len = r.seg_len, p.slots = r.slots;
  w.seg = at;
  if (p.seg_len) at = up256(at + (size_t)p.slots * p.dim * (state + 1) * sizeof(float));
  w.bc = at;
  at = up256(at + (size_t)p.tiles * p.total * 2 * state * sizeof(float));
  w.par = at;
  at += (size_t)p.slots * par_pitch(p.dim, state) * sizeof(float);
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
    if (scan::launch_scan_rev(p, state, f32, vec, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const int64_t grid = ((int64_t)p.dim * state + 127) / 128 * p.N;
    if (grid >= (int64_t(1) << 31)) return KDA_ERR_INVALID_SHAPE;
    scan_rev_carry_kernel<<<(unsigned)grid, 128, 0, stream>>>(p, state);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  }
  if (launch_bwd_pass(p, state, f32, vec, p.cu ? 32 : 0, stream) != cudaSuccess)
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
  if (launch_column_sums(p.part_par, p.slots, par_pitch(p.dim, state), n + 2 * (int64_t)p.dim, n,
                         p.dim, dA_log, dD, ddt_bias, stream) != cudaSuccess ||
      seqlens_status(p, static_cast<unsigned*>(workspace), stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return KDA_OK;
}

}  // extern "C"
