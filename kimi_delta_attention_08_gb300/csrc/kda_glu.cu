// kda_glu.cu -- the gated feed-forward product, forward and backward.
//
//   g = x Wg^T,  u = x Wu^T,  out = f(g) u                      (x: M x D, W: F x D)
//   dg = dout u f'(g),  du = dout f(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Four products on the tensor cores, one kernel.  A pair of CTAs computes 256 x 256 values in
// tensor memory, 128 rows each, as tcgen05.mma.cta_group::2 with M = N = 256: per 64
// values of the summed axis a CTA loads 16 KB of each operand by TMA where a CTA alone
// would load 48 KB, and reads half of B from its peer.  Forward, the 256 columns are 128 of
// the gate and the same 128 of the other projection, so both meet in one thread of the
// epilogue, and neither g nor u goes to memory; the recomputing backward multiplies dout in
// there.  dx sums over both projections in one accumulator.  Operands whose summed axis is
// not contiguous (W in dx, all of dW) are read as they lie, as MN-major tiles: nothing is
// transposed.  Two accumulators alternate, so the epilogue of a tile runs under the next
// one's products.
//
// Accumulation is fp32.  dg and du are rounded to bf16 between the two steps of the backward,
// since the tensor cores take bf16: their error, half a step of bf16 each and independent
// over the summed axis, adds as much to dx and dW as the outputs' own rounding.
//
// Where tiles of 128 columns would take a second turn and wider ones do not, they are 160 or 192 wide;
// the backward splits the sums of its last turn's tiles over the pairs left.
//
// 4,096 by 12,288: 32,768 rows forward 3.83 to 4.04 ms (1.63 to 1.72 PFLOP/s; the longer runs meet the
// power limit), 4,096 rows 468 us (1.76), 256 rows 44 us, 64 wide tiles on 76 pairs (4.6 TB/s of
// weights).  16,384 rows forward with kept pre-activations and backward 6.24 to 6.66 ms (1.49 to 1.58),
// backward that computes them again 6.17 to 6.36 ms (1.56 to 1.60).  The tensor pipe is active in 79 to 82 % of the cycles; operands arrive at 12 to 13
// TB/s from L2, which half the products would still need 2.9 ms for at 32,768 rows.
// One row 35 us, 32 rows 36.5 (5.8 TB/s of weights).
#include <algorithm>

#include "kda_internal.h"
#include "kda_rows.cuh"
#include "../../include/kda_layer.h"

namespace kda {
namespace {

using namespace rows;

constexpr int kTileM = 256, kTileN = 256, kTileK = 64, kStages = 6;
constexpr int kHalf = 128;                       // rows of A, columns of B in each CTA
constexpr uint32_t kOperand = kHalf * kTileK * 2, kStage = 2 * kOperand;  // bytes in a stage
constexpr int kEpilogueWarp = 4, kEpilogueWarps = 8;  // warps 4 .. 11
constexpr uint32_t kOut = 32 * 64;               // 32 rows by 32 columns of an output, on their way
constexpr uint32_t kSmem = kStages * kStage + kEpilogueWarps * 2 * kOut + 1024;
// Wide tiles, of which a pair has one: up to 192 columns of each projection, five stages of 40 KB,
// whose memory the outputs take when the products are done.
constexpr int kWide = 192, kWideStages = 5;
constexpr uint32_t kWideStage = kOperand + kWide * kTileK * 2;
static_assert(kWideStages * kWideStage + 1024 <= kSmem && kEpilogueWarps * 2 * kOut <= kWideStage, "");
constexpr uint64_t kWaitNs = 500000000ull;

// What a launch computes.
enum GluPass : int { kForward = 0, kRecompute = 1, kInput = 2, kWeights = 3 };

struct GluParams {
  CUtensorMap a[2], b[2];  // of the gate and the other projection, or one for both
  CUtensorMap o[3];        // outputs: out, g and u; dg and du; dx; or dWg and dWu
  int64_t M, N;            // of the output (columns: of one projection)
  int32_t k_blocks;        // of each of `sums` products that one tile adds up
  int32_t m_tiles, n_tiles;
  int32_t width;           // columns of each projection in a wide tile
  int32_t whole, splits;   // tiles from `whole` on are split over as many pairs
  float* parts;            // [tiles that are split][splits] sums
  unsigned* counts;        // [tiles that are split][2][kEpilogueWarps] parts that are there
  int32_t fn, stall;
  int32_t keep;            // whether g and u are outputs too
  int32_t ahead;           // whether the weights' gradients may start before dx ends
  unsigned* ready;         // set by dx when dg and du are there
  const bf16* dout;
  bf16* out;               // the forward's results again, for a wait that runs out
  uint16_t* pre;
  unsigned* status;
};

constexpr float kGelu = 1.5957691216057308f, kGeluCube = 0.044715f;  // sqrt(8 / pi)

// f(g) and f'(g).  gelu is its tanh form, g sigmoid(sqrt(8 / pi) (g + 0.044715 g^3)).  Its slope takes
// the square up to 2^96 only, from where on it meets a sigmoid of 0 or 1 and a slope of 0 in any
// case: infinity times that 0 would be no number.
__device__ __forceinline__ float act_of(float g, int fn) {
  if (fn == KDA_FN_GELU) return g * sigmoid<bf16>(kGelu * g * fmaf(kGeluCube * g, g, 1.f));
  const float s = sigmoid<bf16>(g);
  return fn == KDA_FN_SILU ? g * s : s;
}
__device__ __forceinline__ float act_of(float g, int fn, float& slope) {
  if (fn == KDA_FN_GELU) {
    const float c = fminf(kGeluCube * g * g, 0x1p96f);
    float t;
    const float s = sigmoid<bf16>(kGelu * g * (1.f + c), t);
    slope = fmaf(g * t, kGelu * fmaf(3.f, c, 1.f), s);
    return g * s;
  }
  float t;
  const float s = sigmoid<bf16>(g, t);
  slope = fn == KDA_FN_SILU ? fmaf(g, t, s) : t;
  return fn == KDA_FN_SILU ? g * s : s;
}

// Kept pre-activations: 16 bits each, 9 of fraction and 6 of exponent.  bf16's 7 bits of
// fraction would leave dx and dW 3.1e-3 from their 64-bit values where computing g and u
// again leaves 2.3e-3; these leave 2.4e-3.  Magnitudes up to 2^32; beyond that, and what is
// not finite, becomes NaN, and below 2^-30 the fraction shortens.  The fp32 value times 2^-96
// has its exponent in 6 bits, so what is kept is a part of its bits, rounded to even.
constexpr uint32_t kKeptNan = 0x7E01u;
__device__ __forceinline__ uint32_t keep_bits(float v) {
  const uint32_t b = __float_as_uint(v * 0x1p-96f), m = b & 0x7FFFFFFFu;
  const uint32_t r = (m + 0x1FFFu + (m >> 14 & 1u)) >> 14;
  return (b >> 16 & 0x8000u) | (r < 0x7E00u ? r : kKeptNan);
}
__device__ __forceinline__ float kept_value(uint32_t k) {
  const uint32_t m = k & 0x7FFFu;
  const float v = __uint_as_float((k & 0x8000u) << 16 | m << 14) * 0x1p96f;
  return m < 0x7E00u ? v : __uint_as_float(0x7FFFFFFFu);
}

// A pair's unit of work: a tile, or in the backward's last turn, which leaves pairs without a tile, a
// part of a tile's summed axis.
struct Unit {
  int tile, part, from, to;  // part: -1 for a whole tile
};
template <bool SPLITS>
__device__ __forceinline__ Unit unit_of(const GluParams& p, int u, int blocks) {
  if (!SPLITS || u < p.whole || p.splits == 1) return {u, -1, 0, blocks};
  const int v = u - p.whole, t = v / p.splits, part = v - t * p.splits;
  return {p.whole + t, part, (int)((int64_t)blocks * part / p.splits), (int)((int64_t)blocks * (part + 1) / p.splits)};
}

// A tile of the walk: groups of sixteen tiles down, so that the pairs at work share operands
// and a group's rows of A stay in L2 while it meets all of B.
__device__ __forceinline__ void tile_of(const GluParams& p, int t, int& m, int& n) {
  constexpr int kDown = 16;
  const int per = kDown * p.n_tiles, g = t / per, r = t % per;
  const int down = min(kDown, p.m_tiles - g * kDown);
  m = g * kDown + r % down, n = r / down;
}

__device__ __forceinline__ void store8(bf16* p, const float* f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

template <int PASS, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * (kEpilogueWarp + kEpilogueWarps), 1)
    glu_kernel(const __grid_constant__ GluParams p) {
  constexpr bool A_MN = PASS == kWeights, B_MN = PASS == kInput || PASS == kWeights;
  constexpr bool DUAL = PASS == kForward || PASS == kRecompute;
  constexpr int SUMS = PASS == kInput ? 2 : 1;
  constexpr int STAGES = WIDE ? kWideStages : kStages;
  constexpr uint32_t STAGE = WIDE ? kWideStage : kStage;
  extern __shared__ uint8_t raw[];
  uint8_t* const tiles = ptx::smem_align1024(raw);
  __shared__ uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2];
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = ptx::cluster_rank();
  const int total = p.whole + (p.m_tiles * p.n_tiles - p.whole) * p.splits;  // units
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int blocks = SUMS * p.k_blocks;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < STAGES; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
    for (int b = 0; b < 2; ++b) ptx::mbar_init(&tfull[b], 1), ptx::mbar_init(&tempty[b], 2 * kEpilogueWarps);
    ptx::fence_mbar_init();
  }
  if (warp == 2) ptx::tmem_alloc_pair(&tmem_at, 2 * kTileN);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
  // The backward's launches are in their places before the one ahead ends: dx waits for dg and du, and
  // the weights' gradients, which do not need dx, for dx, before their first tile or (`ahead`) their end.
  // What a launch wrote is promised to those that wait for it, so `ahead` takes dg and du from dx, which
  // did: dx says so by a word that it releases before it lets the next launch start, and the threads that
  // load acquire it; where it is not there they wait for the whole of dx.
  if (PASS == kInput || (PASS == kWeights && !p.ahead)) asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (PASS == kInput) {
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) ptx::st_release(p.ready, 1u);
      __syncthreads();
    }
  }
  if constexpr (PASS == kInput || PASS == kRecompute) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (PASS == kWeights) {
    if (p.ahead && warp == 0 && lane == 0) {
      if (ptx::ld_acquire(p.ready) == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
      ptx::fence_proxy_async_all();  // the loads are the asynchronous proxy's
    }
  }

  if (warp == 0 && lane == 0) {
    // loads: this CTA's half of both operands
    uint32_t stage = 0, parity = 1;
    bool ok = !p.stall;
    for (int t = first; t < total && ok; t += step) {
      const Unit u = unit_of<!DUAL>(p, t, blocks);
      int m, n;
      tile_of(p, u.tile, m, n);
      for (int kb = u.from; kb < u.to && ok; ++kb) {
        ok = ptx::mbar_wait(&empty[stage], parity, kWaitNs);
        if (!ok) break;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], WIDE ? 2 * (kOperand + (uint32_t)p.width * kTileK * 2) : 2 * kStage);
        const uint32_t bar = ptx::cluster_addr(&full[stage], 0);
        uint8_t* const A = tiles + stage * STAGE;
        uint8_t* const B = A + kOperand;
        const int part = SUMS == 2 && kb >= p.k_blocks, k0 = (kb - part * p.k_blocks) * kTileK;
        if constexpr (A_MN) {
          // tiles of the gate's gradient first, then of the other's
          const int half = p.m_tiles / 2, which = m >= half;
          const int at = (m - which * half) * kTileM + rank * kHalf;
          ptx::tma_load_2d_pair(A, &p.a[which], bar, at, k0);
          ptx::tma_load_2d_pair(A + kOperand / 2, &p.a[which], bar, at + 64, k0);
        } else {
          ptx::tma_load_2d_pair(A, &p.a[part], bar, k0, m * kTileM + (int)rank * kHalf);
        }
        if constexpr (B_MN) {
          const int at = n * kTileN + rank * kHalf;
          ptx::tma_load_2d_pair(B, &p.b[part], bar, at, k0);
          ptx::tma_load_2d_pair(B + kOperand / 2, &p.b[part], bar, at + 64, k0);
        } else {
          ptx::tma_load_2d_pair(B, &p.b[rank], bar, k0, n * (WIDE ? p.width : kHalf));
        }
        if (++stage == STAGES) stage = 0, parity ^= 1;
      }
    }
    // every stage is read before the pair may go
    for (int s = 0; s < STAGES && ok; ++s) {
      ok = ptx::mbar_wait(&empty[stage], parity, kWaitNs);
      if (++stage == STAGES) stage = 0, parity ^= 1;
    }
    if (!ok) failed = 1;
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // products of the pair
    constexpr uint32_t idesc = ptx::idesc_bf16_f32(kTileM, kTileN, A_MN, B_MN);
    const uint32_t rest = WIDE ? ptx::idesc_bf16_f32(kTileM, 2 * (p.width - kHalf), A_MN, B_MN) : 0;
    constexpr uint32_t a_step = A_MN ? 16 * 128 : 32, b_step = B_MN ? 16 * 128 : 32;
    uint32_t stage = 0, parity = 0, buf = 0, tparity = 1;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Unit u = unit_of<!DUAL>(p, t, blocks);
      ok = ptx::mbar_wait(&tempty[buf], tparity, kWaitNs);
      ptx::tc_fence_after();
      for (int kb = u.from; kb < u.to && ok; ++kb) {
        ok = ptx::mbar_wait(&full[stage], parity, kWaitNs);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t A = ptx::smem_u32(tiles + stage * STAGE), B = A + kOperand;
#pragma unroll
        for (int k = 0; k < kTileK / 16; ++k) {
          const uint64_t a_desc = ptx::sw128_desc(A + k * a_step, kOperand / 2, 1024);
          ptx::mma_bf16_ss_pair(tmem + buf * kTileN, a_desc, ptx::sw128_desc(B + k * b_step, kOperand / 2, 1024), idesc,
                                kb > u.from || k > 0);
          if constexpr (WIDE)  // the columns from the 129th on of both
            ptx::mma_bf16_ss_pair(tmem + kTileN, a_desc, ptx::sw128_desc(B + kOperand + k * b_step, kOperand / 2, 1024),
                                  rest, kb > u.from || k > 0);
        }
        ptx::mma_commit_pair(&empty[stage]);
        if (++stage == STAGES) stage = 0, parity ^= 1;
      }
      if (!ok) break;
      ptx::mma_commit_pair(&tfull[buf]);
      if (!WIDE) buf ^= 1;
      if (buf == 0) tparity ^= 1;
    }
    if (!ok) failed = 1;
  } else if (warp >= kEpilogueWarp) {
    // Two warps take the halves of the columns of 32 rows.  Values go 32 columns at a time through
    // shared memory and out by TMA, whole sectors at once; a thread's own stores of 16 bytes a
    // row took 4 % of the largest forward and a fifth of the smallest backward.
    constexpr int kColumns = (DUAL ? kHalf : kTileN) / 2;
    const int w = warp - kEpilogueWarp, quarter = w % 4, side = w / 4;
    // a wide tile's in turn: 160 columns have an odd number of 32
    const int first_c = side * (WIDE ? 32 : kColumns), step_c = WIDE ? 64 : 32;
    const int end_c = WIDE ? p.width : first_c + kColumns;
    uint8_t* const out = tiles + (WIDE ? 0 : kStages * kStage) + w * 2 * kOut;
    const uint64_t limit = kWaitNs + (uint64_t)blocks * 2000;  // a whole tile's sum may be long
    uint32_t buf = 0, parity = 0, turn = 0;
    bool ok = true;
    // 32 columns of the warp's rows: `packed(k)` is the pair of columns 2 k and 2 k + 1
    auto put = [&](const CUtensorMap* map, int64_t col, int64_t row0, int64_t rows, auto packed) {
      uint8_t* const at = out + (turn++ & 1) * kOut;
      if (lane == 0) ptx::tma_store_wait_read<1>();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k)  // 64-byte swizzle
        *reinterpret_cast<uint4*>(at + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) =
            make_uint4(packed(4 * k), packed(4 * k + 1), packed(4 * k + 2), packed(4 * k + 3));
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {  // a group for each turn, empty ones too: the wait above counts turns
        if (row0 < rows && col < p.N) ptx::tma_store_2d(map, at, (int)col, (int)row0);
        ptx::tma_store_commit();
      }
    };
    auto release = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::cluster_addr(&tempty[buf], 0));
      if (!WIDE) buf ^= 1;
      if (buf == 0) parity ^= 1;
    };
    for (int t = first; t < total; t += step) {
      const Unit u = unit_of<!DUAL>(p, t, blocks);
      int m, n;
      tile_of(p, u.tile, m, n);
      int64_t row0 = (int64_t)m * kTileM;
      int which = 0;
      if constexpr (PASS == kWeights) {
        const int half = p.m_tiles / 2;
        which = m >= half;
        row0 = (int64_t)(m - which * half) * kTileM;
      }
      row0 += rank * kHalf + quarter * 32;
      const int64_t col0 = (int64_t)n * (WIDE ? p.width : DUAL ? kHalf : kTileN);
      const uint32_t acc = tmem + buf * kTileN + ((uint32_t)(quarter * 32) << 16);
      uint4 d[4] = {};       // dout of 32 columns, asked for ahead
      auto load = [&](int c) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row0 + lane < p.M && col0 + c + 8 * k < p.N)
            d[k] = __ldg(reinterpret_cast<const uint4*>(p.dout + (row0 + lane) * p.N + col0 + c + 8 * k));
      };
      if constexpr (PASS == kRecompute) load(first_c);
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(&tfull[buf], parity, limit));
      if (!ok) break;
      ptx::tc_fence_after();
      // The parts of a split tile go to memory, and the warp whose part comes last adds them up, in
      // the order of the parts: nobody waits, and the sums are the same in every run.
      constexpr int kPart = kTileM * kTileN;
      const float* sums = nullptr;
      if constexpr (!DUAL) {
        if (u.part >= 0) {
          const int split = u.tile - p.whole;
          float* const mine =
              p.parts + (int64_t)split * p.splits * kPart + (rank * kEpilogueWarps + w) * 32 * kColumns + lane;
          float* to = mine + (int64_t)u.part * kPart;
#pragma unroll 1
          for (int c = 0; c < kColumns; c += 32, to += 32 * 32) {
            uint32_t v[32];
            ptx::tmem_ld32(acc + side * kColumns + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) to[k * 32] = __uint_as_float(v[k]);
          }
          release();
          __threadfence();
          __syncwarp();
          unsigned before = 0;
          if (lane == 0) before = atomicAdd(p.counts + (split * 2 + rank) * kEpilogueWarps + w, 1u);
          if (__shfl_sync(0xffffffffu, before, 0) != p.splits - 1) continue;
          __threadfence();
          sums = mine;
        }
      }
#pragma unroll 1
      for (int c = first_c; c < end_c; c += step_c) {
        uint32_t v[32];
        if (DUAL || !sums) ptx::tmem_ld32(acc + (WIDE && c >= kHalf ? kHalf : 0) + c, v);
        auto pack = [&](const uint32_t (&f)[32]) {
          return [&](int k) { return pack_bf16(__uint_as_float(f[2 * k]), __uint_as_float(f[2 * k + 1])); };
        };
        if constexpr (DUAL) {
          uint32_t q[32];
          ptx::tmem_ld32(acc + (WIDE && c >= kHalf ? p.width : kHalf) + c, q);
          ptx::tmem_wait_ld();
          if constexpr (PASS == kForward) {
            if (p.keep) {
              auto kept = [&](const uint32_t (&f)[32]) {
                return [&](int k) { return keep_bits(__uint_as_float(f[2 * k])) | keep_bits(__uint_as_float(f[2 * k + 1])) << 16; };
              };
              put(&p.o[1], col0 + c, row0, p.M, kept(v));
              put(&p.o[2], col0 + c, row0, p.M, kept(q));
            }
            put(&p.o[0], col0 + c, row0, p.M, [&](int k) {
              return pack_bf16(act_of(__uint_as_float(v[2 * k]), p.fn) * __uint_as_float(q[2 * k]),
                               act_of(__uint_as_float(v[2 * k + 1]), p.fn) * __uint_as_float(q[2 * k + 1]));
            });
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t dw = (&d[k / 8].x)[k / 2 % 4];
              const float dy = k & 1 ? hi_bf16(dw) : lo_bf16(dw);
              float slope;
              const float f = act_of(__uint_as_float(v[k]), p.fn, slope);
              v[k] = __float_as_uint(dy * __uint_as_float(q[k]) * slope);
              q[k] = __float_as_uint(dy * f);
            }
            if (c + step_c < end_c) load(c + step_c);
            put(&p.o[0], col0 + c, row0, p.M, pack(v));
            put(&p.o[1], col0 + c, row0, p.M, pack(q));
          }
        } else {
          if (sums) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0u;
            const float* from = sums + (c - first_c) * 32;
            for (int q = 0; q < p.splits; ++q, from += kPart)
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + __ldcg(from + k * 32));
          } else {
            ptx::tmem_wait_ld();
          }
          put(&p.o[which], col0 + c, row0, p.M, pack(v));
        }
      }
      if (DUAL || !sums) release();
    }
    if (lane == 0) ptx::tma_store_wait();
    if (!ok && lane == 0) failed = 1;
  }
  __syncwarp();
  __syncthreads();
  if (failed) {  // a wait ran out: what is in flight comes to rest before anything is freed
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevStatusTimeout);
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 2000000) {
    }
    if constexpr (PASS == kForward) {  // and, as the caller may read no status, this CTA's results become NaN
      const int64_t width = WIDE ? p.width : kHalf;
      for (int t = first; t < total; t += step) {
        int m, n;
        tile_of(p, t, m, n);
        const int64_t row0 = (int64_t)m * kTileM + rank * kHalf, col0 = n * width;
        for (int64_t e = threadIdx.x; e < kHalf * width; e += blockDim.x) {
          const int64_t row = row0 + e / width, col = col0 + e % width;
          if (row >= p.M || col >= p.N) continue;
          p.out[row * p.N + col] = __float2bfloat16_rn(__uint_as_float(0x7FFFFFFFu));
          if (p.keep) p.pre[row * 2 * p.N + col] = p.pre[(row * 2 + 1) * p.N + col] = (uint16_t)kKeptNan;
        }
      }
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp == 2) ptx::tmem_dealloc_pair(tmem, 2 * kTileN);
  if constexpr (PASS == kWeights) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------- few rows --
// The forward of up to kStepRows rows reads the weights once and is bound by that (128 rows 43
// us, 192 rows as wide tiles 44).  A CTA
// takes 64 rows of both weights as the 128 rows of A, and all of x as B's columns, so the tensor
// cores do no more work than the rows need; where the weights' rows alone do not fill the
// GPU, a cluster splits the summed axis and adds up through its shared memory, in the order
// of its CTAs.  Two CTAs fit an SM, each with 108 KB of weights and x in flight.
constexpr int kStepRows = 128, kStepTile = 64, kStepMaxSplit = 8;
constexpr uint32_t kStepRing = 110592, kStepSmem = kStepRing + 1024;
constexpr int kStepPitch = 132;                  // floats between two rows' sums

struct StepParams {
  CUtensorMap w[2], x;
  int32_t rows, cols;        // of x that exist; of the product, a multiple of 16
  int32_t hidden, k_blocks, splits, stages, fn, stall;
  bf16* out;
  uint16_t* pre;
  unsigned* status;
};

__global__ void __launch_bounds__(256, 2) glu_step_kernel(const __grid_constant__ StepParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* const ring = ptx::smem_align1024(raw);
  __shared__ uint64_t full[6], empty[6], done;
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = blockIdx.x % p.splits, f0 = blockIdx.x / p.splits * kStepTile;
  const int per = (p.k_blocks + p.splits - 1) / p.splits;
  const int first = split * per, last = min(p.k_blocks, first + per);
  const uint32_t stage_bytes = 2 * kStepTile * 128 + p.cols * 128;
  auto load = [&](int kb, int stage) {
    uint8_t* const A = ring + stage * stage_bytes;
    ptx::mbar_arrive_expect_tx(&full[stage], stage_bytes);
    ptx::tma_load_2d(A, &p.w[0], &full[stage], kb * kTileK, f0);
    ptx::tma_load_2d(A + kStepTile * 128, &p.w[1], &full[stage], kb * kTileK, f0);
    ptx::tma_load_2d(A + 2 * kStepTile * 128, &p.x, &full[stage], kb * kTileK, 0);
  };
  const int ahead = p.stall ? 0 : min(p.stages, last - first);  // loads that need not wait for anything
  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < p.stages; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
    ptx::mbar_init(&done, 1);
    ptx::fence_mbar_init();
    for (int s = 0; s < ahead; ++s) load(first + s, s);
  }
  if (warp == 2) {
    ptx::tmem_alloc(&tmem_at, 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
  if (warp == 0 && lane == 0) {
    bool ok = !p.stall;
    uint32_t stage = 0, parity = 0;
    for (int kb = first + ahead; kb < last && ok; ++kb) {
      ok = ptx::mbar_wait(&empty[stage], parity, kWaitNs);
      if (!ok) break;
      load(kb, stage);
      if (++stage == p.stages) stage = 0, parity ^= 1;
    }
    if (!ok) failed = 1;
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = ptx::idesc_bf16_f32(128, p.cols, 0, 0);
    bool ok = true;
    uint32_t stage = 0, parity = 0;
    for (int kb = first; kb < last; ++kb) {
      ok = ptx::mbar_wait(&full[stage], parity, kWaitNs);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t A = ptx::smem_u32(ring + stage * stage_bytes), B = A + 2 * kStepTile * 128;
#pragma unroll
      for (int k = 0; k < kTileK / 16; ++k)
        ptx::mma_bf16_ss(tmem, ptx::sw128_desc(A + k * 32, 16, 1024), ptx::sw128_desc(B + k * 32, 16, 1024), idesc,
                         kb > first || k > 0);
      ptx::mma_commit(&empty[stage]);
      if (++stage == p.stages) stage = 0, parity ^= 1;
    }
    ptx::mma_commit(&done);
    if (!ok) failed = 1;
  }
  __syncwarp();
  // this CTA's sums, [x's row][weights' row], where the ring was
  float* const sums = reinterpret_cast<float*>(ring);
  const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(&done, 0, 2 * kWaitNs));
  if (!ok && lane == 0) failed = 1;
  __syncthreads();
  if (failed) {  // a wait ran out: what is in flight comes to rest before its place is used
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kDevStatusTimeout);
    const uint64_t t0 = ptx::global_timer_ns();
    while (ptx::global_timer_ns() - t0 < 2000000) {
    }
  }
  ptx::tc_fence_after();
  if (warp >= 4) {
    const int f = (warp - 4) * 32 + lane;
    const bool bad = failed;  // no number then, as the caller may read no status
    for (int c = 0; c < p.cols; c += 16) {
      uint32_t v[16];
      ptx::tmem_ld16(tmem + ((uint32_t)((warp - 4) * 32) << 16) + c, v);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; ++k)
        sums[(c + k) * kStepPitch + f] = __uint_as_float(bad ? 0x7FFFFFFFu : first < last ? v[k] : 0u);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 2) ptx::tmem_dealloc(tmem, 128);
  // each CTA of the cluster adds up some of the rows: a warp a row, a lane two columns
  const int col = f0 + 2 * lane;
  for (int r = split * 8 + warp; r < p.rows; r += p.splits * 8) {
    float2 g = make_float2(0.f, 0.f), u = g;
    for (int q = 0; q < p.splits; ++q) {
      const uint32_t at = ptx::cluster_addr(sums + r * kStepPitch + 2 * lane, q);
      float2 v;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
      g.x += v.x, g.y += v.y;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at + 4 * kStepTile) : "memory");
      u.x += v.x, u.y += v.y;
    }
    if (col < p.hidden) {
      const int64_t at = (int64_t)r * p.hidden + col;
      *reinterpret_cast<uint32_t*>(p.out + at) = pack_bf16(act_of(g.x, p.fn) * u.x, act_of(g.y, p.fn) * u.y);
      if (p.pre) {
        uint16_t* const to = p.pre + (int64_t)r * 2 * p.hidden + col;
        *reinterpret_cast<uint32_t*>(to) = keep_bits(g.x) | keep_bits(g.y) << 16;
        *reinterpret_cast<uint32_t*>(to + p.hidden) = keep_bits(u.x) | keep_bits(u.y) << 16;
      }
    }
  }
  ptx::cluster_sync();
}

// dg and du from kept pre-activations, eight values a thread.
__global__ void __launch_bounds__(256) glu_slope_kernel(const uint16_t* pre, const bf16* dout, bf16* dg, bf16* du,
                                                        int64_t M, int64_t F, int fn) {
  const int64_t per = F / 8, n = M * per;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / per, col = e % per * 8;
    Raw<bf16, 8> rg, ru, rd;
    load_words(rg.w, pre + row * 2 * F + col);
    load_words(ru.w, pre + row * 2 * F + F + col);
    load_words(rd.w, dout + row * F + col);
    float g[8], u[8], d[8];
    unpack(rd, d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] = kept_value(rg.w[k / 2] >> (k % 2 * 16) & 0xFFFFu), u[k] = kept_value(ru.w[k / 2] >> (k % 2 * 16) & 0xFFFFu);
      float slope;
      const float f = act_of(g[k], fn, slope);
      g[k] = d[k] * u[k] * slope, u[k] = d[k] * f;
    }
    store8(dg + row * F + col, g);
    store8(du + row * F + col, u);
  }
}

// ------------------------------------------------------------------- host --
bool al_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// A map of an output of 16-bit values, its boxes 32 columns by 32 rows, 64-byte swizzled.
cudaError_t out_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)stride * 2};
  const uint32_t b[2] = {32, 32};
  return encode_tiled_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_64B);
}
// A map of bf16 [rows, cols] with boxes of 64 columns by `box` rows, 128-byte swizzled.
cudaError_t map_of(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride, uint32_t box) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)stride * 2};
  const uint32_t b[2] = {64, box};
  return encode_tiled_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, b,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

// How the backward splits its last turn's tiles: as often as pairs are left over, where a part has
// 16 steps of the summed axis at least and a tile 48.  A tile's parts cost a few us on their way
// through memory, a step 0.33 us.  Backward without and with: 100 rows of 4,096 by 12,288 243 and
// 168 us, 512 rows of 2,048 by 6,144 127 and 92, 16,384 rows of 1,000 by 2,728 521 and 453; parts of
// four steps lose up to 12 us at 1,024 hidden.  The forward's tiles stay
// whole: 256 rows, which read the weights at HBM's rate in either case, came to 53.1 us for 53.8,
// 512 rows of 2,048 by 6,144 to 32.7 for 29.2.
constexpr int64_t kPairs = 76;  // a GB300's: a workspace's size is asked for without a device
constexpr int64_t kMaxSplits = 8, kSplitBlocks = 48;
struct Split {
  int64_t whole, splits, split;  // tiles in whole turns; parts of each of the others; those
};
Split split_of(int64_t tiles, int64_t blocks) {
  Split s = {tiles / kPairs * kPairs, 1, tiles % kPairs};
  if (s.split > 0 && blocks >= kSplitBlocks) s.splits = std::max<int64_t>(1, std::min({kMaxSplits, kPairs / s.split, blocks / 16}));
  return s;
}
// Counters of the parts of dx's tiles, then of the weights'.
constexpr size_t kCounters = kPairs * 2 * kEpilogueWarps * sizeof(unsigned);
constexpr size_t kHeader = KDA_STATUS_BYTES + 2 * kCounters;
static_assert(kCounters % 256 == 0, "what follows is aligned");
// The backward's dg, du and parts of dx's tiles and of the weights', for any width of the rows.
size_t bwd_operand(int64_t M, int64_t F) { return up256((size_t)M * F * 2); }
size_t parts_bytes(int64_t blocks) { return blocks < kSplitBlocks ? 0 : (size_t)kPairs * kTileM * kTileN * sizeof(float); }
size_t bwd_bytes(int64_t M, int64_t F) {
  if (M == 0) return KDA_STATUS_BYTES;
  return kHeader + 2 * bwd_operand(M, F) + parts_bytes(2 * up(F, kTileK)) + parts_bytes(up(M, kTileK));
}

// counts: zeros.
template <int PASS, bool WIDE = false>
cudaError_t launch(GluParams& p, const Split& s, float* parts, unsigned* counts, cudaStream_t stream) {
  static bool done[64];
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(glu_kernel<PASS, WIDE>), kSmem, done);
  if (e != cudaSuccess) return e;
  int sms = 0;
  if (sm_count(&sms) != KDA_OK) return cudaErrorUnknown;
  p.whole = (int32_t)s.whole, p.splits = (int32_t)s.splits;
  p.parts = parts, p.counts = counts;
  const int64_t units = s.whole + s.split * p.splits, pairs = units < sms / 2 ? units : sms / 2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(2 * pairs)), c.blockDim = dim3(32 * (kEpilogueWarp + kEpilogueWarps));
  c.dynamicSmemBytes = kSmem, c.stream = stream;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a, c.numAttrs = PASS == kInput || PASS == kWeights;  // see glu_kernel
  return cudaLaunchKernelEx(&c, glu_kernel<PASS, WIDE>, p);
}

kda_status check_glu(const kda_glu_problem* q) {
  if (!q) return KDA_ERR_NULL_POINTER;
  const int64_t lim = int64_t(1) << 31;
  if (q->rows < 0 || q->rows >= lim || q->dim < 8 || q->hidden < 8 || q->dim % 8 || q->hidden % 8 ||
      q->x_stride < q->dim || q->x_stride >= lim || q->x_stride % 8)
    return KDA_ERR_INVALID_SHAPE;
  if (up(q->rows, kTileM) * up(q->hidden, kHalf) >= lim || up(q->rows, kTileM) * up(q->dim, kTileN) >= lim ||
      2 * up(q->hidden, kTileM) * up(q->dim, kTileN) >= lim)
    return KDA_ERR_INVALID_SHAPE;
  if (q->dtype != KDA_ROW_BF16 || (q->fn != KDA_FN_SILU && q->fn != KDA_FN_SIGMOID && q->fn != KDA_FN_GELU))
    return KDA_ERR_INVALID_ARG;
  if (!q->w_gate || !q->w_up || (q->rows > 0 && !q->x)) return KDA_ERR_NULL_POINTER;
  if (!al_to(q->x, 16) || !al_to(q->w_gate, 16) || !al_to(q->w_up, 16)) return KDA_ERR_MISALIGNED;
  return KDA_OK;
}

// Columns of each projection in a wide tile, or 0: where tiles of 128 need a second turn and wider ones
// do not.  256 rows of 4,096 by 12,288 as 96 tiles 54.6 us, as 64 wide ones 44.0; 512 rows of 2,048 by
// 6,144 30.0 and 24.5; 1,024 rows of 1,000 by 2,728 20.4 and 16.2.  Several turns of wide tiles, which
// have one accumulator, would put each one's epilogue after its products.
int wide_of(int64_t down, int64_t hidden) {
  int sms = 0;
  if (sm_count(&sms) != KDA_OK || down * up(hidden, kHalf) <= sms / 2) return 0;
  for (int w : {160, kWide})
    if (down * up(hidden, w) <= sms / 2) return w;
  return 0;
}

// The forward's tiles (also of the recomputing backward).
template <int PASS>
cudaError_t launch_dual(const kda_glu_problem* q, bf16* o0, bf16* o1, uint16_t* pre, const void* dout, unsigned* status,
                        cudaStream_t stream) {
  GluParams p = {};
  const int64_t down = up(q->rows, kTileM);
  const int wide = wide_of(down, q->hidden);
  p.width = wide ? wide : kHalf;
  cudaError_t e = map_of(&p.a[0], q->x, q->rows, q->dim, q->x_stride, kHalf);
  if (e == cudaSuccess) e = map_of(&p.b[0], q->w_gate, q->hidden, q->dim, q->dim, p.width);
  if (e == cudaSuccess) e = map_of(&p.b[1], q->w_up, q->hidden, q->dim, q->dim, p.width);
  if (e == cudaSuccess) e = out_map(&p.o[0], o0, q->rows, q->hidden, q->hidden);
  if (e == cudaSuccess && o1) e = out_map(&p.o[1], o1, q->rows, q->hidden, q->hidden);
  if (e == cudaSuccess && pre) {
    e = out_map(&p.o[1], pre, q->rows, q->hidden, 2 * (int64_t)q->hidden);
    if (e == cudaSuccess) e = out_map(&p.o[2], pre + q->hidden, q->rows, q->hidden, 2 * (int64_t)q->hidden);
  }
  if (e != cudaSuccess) return e;
  p.M = q->rows, p.N = q->hidden;
  p.k_blocks = (int32_t)up(q->dim, kTileK);
  p.m_tiles = (int32_t)down, p.n_tiles = (int32_t)up(q->hidden, p.width);
  p.fn = q->fn, p.stall = q->debug_stall, p.status = status;
  p.keep = pre != nullptr, p.dout = static_cast<const bf16*>(dout);
  p.out = o0, p.pre = pre;
  if (wide) return launch<PASS, true>(p, {(int64_t)p.m_tiles * p.n_tiles, 1, 0}, nullptr, nullptr, stream);
  return launch<PASS>(p, {(int64_t)p.m_tiles * p.n_tiles, 1, 0}, nullptr, nullptr, stream);
}

// Up to kStepRows rows.  As many CTAs share the summed axis as fit the GPU twice per SM, with four
// steps of 64 at least for each.
cudaError_t launch_step(const kda_glu_problem* q, bf16* out, uint16_t* pre, unsigned* status, cudaStream_t stream) {
  StepParams p = {};
  int sms = 0;
  if (sm_count(&sms) != KDA_OK) return cudaErrorUnknown;
  const int64_t tiles = up(q->hidden, kStepTile);
  p.rows = (int32_t)q->rows, p.cols = (int32_t)up(q->rows, 16) * 16;
  p.hidden = q->hidden, p.k_blocks = (int32_t)up(q->dim, kTileK);
  p.splits = 1;
  while (p.splits < kStepMaxSplit && tiles * p.splits * 2 <= 2 * sms && p.k_blocks >= 8 * p.splits) p.splits *= 2;
  p.stages = std::min(6, (int)(kStepRing / (2 * kStepTile * 128 + p.cols * 128)));
  p.fn = q->fn, p.stall = q->debug_stall, p.out = out, p.pre = pre, p.status = status;
  cudaError_t e = map_of(&p.w[0], q->w_gate, q->hidden, q->dim, q->dim, kStepTile);
  if (e == cudaSuccess) e = map_of(&p.w[1], q->w_up, q->hidden, q->dim, q->dim, kStepTile);
  if (e == cudaSuccess) e = map_of(&p.x, q->x, q->rows, q->dim, q->x_stride, p.cols);
  static bool done[64];
  if (e == cudaSuccess) e = ensure_smem_attr(reinterpret_cast<const void*>(glu_step_kernel), kStepSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(tiles * p.splits)), c.blockDim = dim3(256);
  c.dynamicSmemBytes = kStepSmem, c.stream = stream;
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = p.splits, a.val.clusterDim.y = a.val.clusterDim.z = 1;
  c.attrs = &a, c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, glu_step_kernel, p);
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_glu_fwd(const kda_glu_problem* problem, void* out, void* pre, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_glu(problem);
  if (st != KDA_OK) return st;
  if (problem->rows > 0 && !out) return KDA_ERR_NULL_POINTER;
  if (!al_to(out, 16) || !al_to(pre, 16) || !al_to(workspace, 128)) return KDA_ERR_MISALIGNED;
  if (workspace && workspace_bytes < KDA_STATUS_BYTES) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  unsigned* const status = static_cast<unsigned*>(workspace);
  if (status && cudaMemsetAsync(status, 0, 4, stream) != cudaSuccess) return KDA_ERR_CUDA;
  if (problem->rows == 0) return KDA_OK;
  bf16* const to = static_cast<bf16*>(out);
  uint16_t* const kept = static_cast<uint16_t*>(pre);
  const cudaError_t e = problem->rows <= kStepRows ? launch_step(problem, to, kept, status, stream)
                                                   : launch_dual<kForward>(problem, to, nullptr, kept, nullptr, status, stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_glu_bwd_get_workspace_size(int64_t rows, int32_t hidden, size_t* bytes) {
  if (!bytes) return KDA_ERR_NULL_POINTER;
  if (rows < 0 || rows >= (int64_t(1) << 31) || hidden < 8 || hidden % 8) return KDA_ERR_INVALID_SHAPE;
  *bytes = kda::bwd_bytes(rows, hidden);
  return KDA_OK;
}

kda_status kda_glu_bwd(const kda_glu_problem* problem, const void* dout, const void* pre, void* dx,
                       void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  using namespace kda;
  kda_status st = check_glu(problem);
  if (st != KDA_OK) return st;
  const kda_glu_problem& q = *problem;
  if (!dw_gate || !dw_up || !workspace || (q.rows > 0 && (!dout || !dx))) return KDA_ERR_NULL_POINTER;
  for (const void* v : {dout, pre, (const void*)dx, (const void*)dw_gate, (const void*)dw_up})
    if (!al_to(v, 16)) return KDA_ERR_MISALIGNED;
  if (!al_to(workspace, 128)) return KDA_ERR_MISALIGNED;
  size_t need = 0;
  st = kda_glu_bwd_get_workspace_size(q.rows, q.hidden, &need);
  if (st != KDA_OK) return st;
  if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
  st = check_device();
  if (st != KDA_OK) return st;
  unsigned* const status = static_cast<unsigned*>(workspace);
  const int64_t M = q.rows, D = q.dim, F = q.hidden;
  cudaError_t e = cudaMemsetAsync(status, 0, M ? kHeader : 4, stream);
  if (M == 0) {  // sums of nothing
    if (e == cudaSuccess) e = cudaMemsetAsync(dw_gate, 0, (size_t)F * D * 2, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(dw_up, 0, (size_t)F * D * 2, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
  }
  unsigned* const counts = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + KDA_STATUS_BYTES);
  bf16* const dg = reinterpret_cast<bf16*>(static_cast<uint8_t*>(workspace) + kHeader);
  bf16* const du = dg + bwd_operand(M, F) / 2;
  float* const parts = reinterpret_cast<float*>(du + bwd_operand(M, F) / 2);
  if (e == cudaSuccess) {
    if (pre) {
      const int64_t blocks = up(M * (F / 8), 256);
      glu_slope_kernel<<<(unsigned)(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0, stream>>>(
          static_cast<const uint16_t*>(pre), static_cast<const bf16*>(dout), dg, du, M, F, q.fn);
      e = cudaGetLastError();
    } else {
      e = launch_dual<kRecompute>(problem, dg, du, nullptr, dout, status, stream);
    }
  }
  GluParams p = {};
  p.stall = q.debug_stall, p.status = status, p.ready = status + 1;
  // dx: both projections' products in one sum
  if (e == cudaSuccess) e = map_of(&p.a[0], dg, M, F, F, kHalf);
  if (e == cudaSuccess) e = map_of(&p.a[1], du, M, F, F, kHalf);
  if (e == cudaSuccess) e = map_of(&p.b[0], q.w_gate, F, D, D, kTileK);
  if (e == cudaSuccess) e = map_of(&p.b[1], q.w_up, F, D, D, kTileK);
  p.M = M, p.N = D, p.k_blocks = (int32_t)up(F, kTileK), p.m_tiles = (int32_t)up(M, kTileM);
  p.n_tiles = (int32_t)up(D, kTileN);
  if (e == cudaSuccess) e = out_map(&p.o[0], dx, M, D, D);
  if (e == cudaSuccess) e = launch<kInput>(p, split_of((int64_t)p.m_tiles * p.n_tiles, 2 * p.k_blocks), parts, counts, stream);
  // The weights' gradients start where dx leaves pairs without work, if it has two turns of tiles at
  // most: 4,097 rows of 1,000 by 2,728 138 us without, 132 with it, of 256 by 1,024 50 and 36.  Behind
  // a longer dx the pairs would come out of step and share less of what L2 holds: 4,097 rows of 4,096 by
  // 12,288 1,524 us without, 1,597 with it.
  p.ahead = (int64_t)p.m_tiles * p.n_tiles <= 2 * kPairs;
  // the gate's rows, then the other's
  if (e == cudaSuccess) e = map_of(&p.a[0], dg, M, F, F, kTileK);
  if (e == cudaSuccess) e = map_of(&p.a[1], du, M, F, F, kTileK);
  if (e == cudaSuccess) e = map_of(&p.b[0], q.x, M, D, q.x_stride, kTileK);
  p.M = F, p.N = D, p.k_blocks = (int32_t)up(M, kTileK), p.m_tiles = (int32_t)(2 * up(F, kTileM));
  if (e == cudaSuccess) e = out_map(&p.o[0], dw_gate, F, D, D);
  if (e == cudaSuccess) e = out_map(&p.o[1], dw_up, F, D, D);
  if (e == cudaSuccess) e = launch<kWeights>(p, split_of((int64_t)p.m_tiles * p.n_tiles, p.k_blocks),
                                               parts + parts_bytes(2 * up(F, kTileK)) / sizeof(float),
                                               counts + kCounters / sizeof(unsigned), stream);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
