// Backward of the expert networks on the 5th-generation tensor cores
// ("Outrageously Large Neural Networks", section 3.4: the experts and the
// gate are trained by plain back-propagation; "Switch Transformer", step 6:
// each expert owns W1 [d, d_ff] and W2 [d_ff, d]). One grouped-GEMM kernel in
// three modes over the rows each expert received in the forward:
//
//   dgrad through W2 (mode 0):  D = dY_rows W2[e]^T           [rows, d_ff]
//       epilogue: dgate partial <D_r, h_r> per 256-column block, and
//       dpre_r = g_r * D_r * [h_r > 0] in bf16 (pad rows written as zero)
//   dgrad through W1 (mode 1):  dX_rows = dpre_rows W1[e]^T   [rows, d]   (fp32)
//   weight gradient  (mode 2):  dW[e] = A_rows^T B_rows       [M, N]      (fp32)
//       dW2: A = h rows, B = g * dY rows;  dW1: A = x rows, B = dpre rows
//   gated dgrad through W2 (mode 3): D as in mode 0; with the kept
//       pre-activations p1, p3 of the row, a = act(p1), h = a * p3:
//       dP1 = g D p3 act'(p1), dP3 = g D a (bf16, padded rows), g h (bf16, packed
//       rows: the weight gradient dW2 = (g h)^T dY's operand, so that only one of
//       its two is rounded) and the dgate partial <D, h>
//   gated dgrad (mode 4): dX_rows = dP1 W1[e]^T + dP3 W3[e]^T, as mode 1 with a
//       reduction that runs over both pairs
//
// The backward's own row buffers (dY, g*dY, dpre, dX) give each expert a
// block of rows padded to a multiple of 64 (at least 64), pad rows zero, at
// the offsets poff[e]. The weight-gradient mode runs its K loop over those
// padded rows: the pad rows of B are zero, so whatever A holds there (the
// next expert's rows, or rows the caller zeroed past the last one) adds
// nothing, and no K tail needs masking.
//
// Operand layouts (bf16, 128-byte swizzle, as the forward kernel):
//   modes 0, 1: A K-major [128 rows x 64 K]; B K-major [256 rows x 64 K]: the
//               weight's own rows (W2[e] is [d_ff, d]: row f holds K = d
//               contiguous values; W1[e] is [d, d_ff]: row i holds d_ff).
//   mode 2:     A MN-major (M contiguous) as two [64 K x 64 M] blocks, B
//               MN-major as four [64 K x 64 N] blocks, a load each; the instruction
//               descriptor's transpose bits select MN-major for both.
// Warp roles, the 4-stage ring, two TMEM accumulators and the bounded waits
// are those of the forward kernel: warp 0 TMA producer, warp 1 TMEM owner and
// MMA issuer, warps 2-5 epilogue.
#include "moe_internal.cuh"
#include "tc_ptx.cuh"
#include "checkpoint.cuh"
#include "gated.cuh"

#include <stdlib.h>

#include <mutex>

namespace moe {
namespace {

constexpr int BM = kTcBM;  // 128 rows (TMEM lanes)
constexpr int BN = 256;    // accumulator columns per tile
constexpr int BK = 64;     // K per stage
constexpr int A_BYTES = BM * BK * 2;  // 16 KB
constexpr int B_BYTES = BK * BN * 2;  // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int TMEM_COLS = 2 * BN;

struct BParams {
  int mode;
  int K;          // modes 0, 1: reduction length
  int N;          // output columns
  int M;          // mode 2: output rows per expert
  int E, n_blocks, m_blocks;
  const int32_t *offset;  // [E+1] the forward's packed row offsets
  const int32_t *poff;    // [E+1] padded row offsets
  const float *row_gate;  // mode 0: [packed rows]
  const __nv_bfloat16 *hbuf;  // mode 0: [packed rows, N]
  const uint8_t *h8, *hscale;  // mode 0: the same in 8 bits [packed rows, N], [.., N / 32]
  void *out;      // mode 0: bf16 [padded rows, N]; mode 1: fp32 [padded rows, N];
                  // mode 2: fp32 (or bf16) [E, M, N]
  float *dgpart;  // mode 0: [padded rows, n_blocks]
  DeviceStatus *st;
  unsigned long long wait_ns;
  uint32_t *sched;  // [2] the CTA-pair kernel's tile counter and done count (zero at launch)
  int dynamic;      // CTA-pair kernel: tiles from the counter (else round robin)
  int tma_out;      // CTA-pair kernel, modes 0 and 1: 32-row groups leave by TMA store
  int snake;        // CTA-pair kernel: 1 = odd waves of tiles run K backwards, 2 = all do
};

// The gated modes' further operands.
template <int MODE>
struct BExtra {};
template <>
struct BExtra<3> {
  const __nv_bfloat16 *pre1, *pre3;  // [packed rows, N]
  __nv_bfloat16 *dP3, *h;            // h: g h
};
template <>
struct BExtra<4> {
  CUtensorMap a, b;  // dP3, W3
};

// Mode 3 has the heaviest epilogue (two operands read, three written, an
// exponential and a reciprocal an element): eight warps instead of four, each
// with two staging tiles of 2 KB, at the price of a stage of the one-CTA kernel's ring.
template <int MODE>
__host__ __device__ constexpr int epi_warps() { return MODE == 3 ? 8 : 4; }
template <int MODE>
__host__ __device__ constexpr int threads_of() { return 64 + 32 * epi_warps<MODE>(); }
template <int MODE>
__host__ __device__ constexpr int stages_of(bool pair) {
  return pair ? 6 : (MODE == 3 ? 3 : 4);
}
constexpr int G_TILE = 32 * 32 / 2;             // a staging tile of bf16, counted in floats
constexpr int G_STG_BYTES = 8 * 2 * G_TILE * 4;  // mode 3

// The CTA-pair kernel's tile ring, as in the forward expert GEMM: tile
// indices from the even CTA's producer to the MMA issuer, both CTAs'
// epilogue warps and the odd CTA's producer (ten arrivals free a slot).
constexpr int kRing = 8;
constexpr int kRingConsumers = 10;

// kind::f16 instruction descriptor: fp32 accumulate, bf16 A and B, M = 128,
// N = 256; bits 15 / 16 select MN-major A / B.
template <int MODE>
__host__ __device__ constexpr uint32_t bwd_idesc() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((MODE == 2 ? 1u : 0u) << 15) |
         ((MODE == 2 ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)(BM >> 4) << 24);
}

template <int MODE>
__device__ __forceinline__ void umma_b(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(bwd_idesc<MODE>()), "r"(acc)
      : "memory");
}

// Tile -> (expert, m block, n block), the expert's first padded row, its
// padded and real row counts, and the number of K blocks.
struct BTile {
  int e, mb, nb, prow0, prows, rows, num_kb;
};

// Weight-gradient tiles of one expert: the blocks of the operand with fewer
// of them run fastest, so the CTAs working at the same time share the larger
// operand's block and the expert's smaller operand stays whole in L2 (dW2:
// 56 blocks of h columns and 16 of dU at the large-expert widths).
__device__ __forceinline__ void wgrad_order(int local, int m_blocks, int n_blocks, int &mb,
                                            int &nb) {
  if (m_blocks <= n_blocks) {
    nb = local / m_blocks;
    mb = local - nb * m_blocks;
  } else {
    mb = local / n_blocks;
    nb = local - mb * n_blocks;
  }
}

template <int MODE>
__device__ __forceinline__ BTile locate(const BParams &p, const int *start, int tile) {
  BTile t;
  if (MODE == 2) {
    const int per = p.m_blocks * p.n_blocks;
    t.e = tile / per;
    const int local = tile - t.e * per;
    wgrad_order(local, p.m_blocks, p.n_blocks, t.mb, t.nb);
  } else {
    int lo = 0, hi = p.E;  // largest e with start[e] <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= tile) lo = mid;
      else hi = mid;
    }
    t.e = lo;
  }
  t.prow0 = p.poff[t.e];
  t.prows = p.poff[t.e + 1] - t.prow0;
  t.rows = p.offset[t.e + 1] - p.offset[t.e];
  if (MODE != 2) {
    const int mt = (t.prows + BM - 1) / BM;
    const int local = tile - start[t.e];
    t.nb = local / mt;
    t.mb = local - t.nb * mt;
    t.num_kb = (MODE == 4 ? 2 : 1) * (p.K / BK);
  } else {
    t.num_kb = t.prows / BK;
  }
  return t;
}

// 32 fp32 sums of a weight gradient, rounded once to bf16.
__device__ __forceinline__ void pack_bf16(const float (&f)[32], uint32_t (&packed)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    packed[j] = *reinterpret_cast<uint32_t *>(&b);
  }
}

// One lane's row m of a finished tile: 32 accumulator columns at a time from
// TMEM (lane_addr: this warp's lanes, this accumulator), stored as the mode
// asks. Warp-collective (every lane loads). Modes 0 and 1 in the CTA-pair
// kernel pass stg (the warp's two staging tiles), tmO (the output [padded
// rows, N]) and cnt: the warp's 32 rows, inside the expert's padded block
// (its size is a multiple of 64), then leave by TMA store, mode 1's pad rows
// included (zero, as dpre's pad rows are).
template <int MODE, bool OB = false>
__device__ __forceinline__ void epilogue_rows(const BParams &p, const BTile &t, int m,
                                              uint32_t lane_addr, float *stg = nullptr,
                                              const CUtensorMap *tmO = nullptr,
                                              uint32_t *cnt = nullptr) {
  const int m0 = m - (int)(threadIdx.x & 31);  // the warp's first row
  const bool tma = MODE != 2 && stg != nullptr && m0 + 32 <= t.prows;
  // Rows this lane writes: mode 0 every padded row of the expert (pad rows
  // as zero), mode 1 the real rows (every padded row through TMA), mode 2 the
  // output rows m < M.
  const bool valid = MODE == 0 ? m < t.prows
                     : MODE != 2 ? (tma || m < t.rows)
                                 : m < p.M;
  const bool real = m < t.rows;
  const size_t pr = (size_t)t.prow0 + m;
  const size_t q = (size_t)p.offset[t.e] + m;
  const float g = (MODE == 0 && valid && real) ? p.row_gate[q] : 0.f;
  float part = 0.f;
  bool bad = false;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    const int n = t.nb * BN + c * 32;
    uint32_t v[32];
    tmem_ld32(lane_addr + (uint32_t)(c * 32), v);  // warp-collective
    if (!valid || n >= p.N) continue;
    if (MODE == 0) {
      float h[32];
      if (real && OB) {
        // e4m3 values of one block of 32 and its scale: exactly hbuf's values.
        const uint4 *hp = reinterpret_cast<const uint4 *>(p.h8 + q * p.N + n);
        const float sc = ckpt_scale(p.hscale[q * (p.N / kCkptBlock) + n / kCkptBlock]);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint4 u = hp[w];
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 lo = ckpt_e4m3x2(uu[j] & 0xffffu), hi = ckpt_e4m3x2(uu[j] >> 16);
            h[16 * w + 4 * j] = lo.x * sc;
            h[16 * w + 4 * j + 1] = lo.y * sc;
            h[16 * w + 4 * j + 2] = hi.x * sc;
            h[16 * w + 4 * j + 3] = hi.y * sc;
          }
        }
      } else if (real) {
        const uint4 *hp = reinterpret_cast<const uint4 *>(p.hbuf + q * p.N + n);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint4 u = hp[w];
          const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162 *>(&uu[j]);
            h[8 * w + 2 * j] = __low2float(b2);
            h[8 * w + 2 * j + 1] = __high2float(b2);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) h[j] = 0.f;
      }
      uint32_t packed[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float d0 = __uint_as_float(v[2 * j]), d1 = __uint_as_float(v[2 * j + 1]);
        part = fmaf(d0, h[2 * j], part);
        part = fmaf(d1, h[2 * j + 1], part);
        const float p0 = h[2 * j] > 0.f ? g * d0 : 0.f;
        const float p1 = h[2 * j + 1] > 0.f ? g * d1 : 0.f;
        bad |= !isfinite(p0) || !isfinite(p1);
        __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
        packed[j] = *reinterpret_cast<uint32_t *>(&b2);
      }
      if (tma) {
        stage_store_bf16(tmO, stg + (*cnt & 1u) * 1024, packed, n, t.prow0 + m0);
        ++*cnt;
      } else {
        uint4 *o =
            reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + pr * p.N + n);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          o[w] = make_uint4(packed[4 * w], packed[4 * w + 1], packed[4 * w + 2],
                            packed[4 * w + 3]);
      }
    } else {
      float f[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        f[j] = __uint_as_float(v[j]);
        bad |= !isfinite(f[j]);
      }
      if (tma) {
        stage_store_f32(tmO, stg + (*cnt & 1u) * 1024, f, n, t.prow0 + m0);
        ++*cnt;
      } else if constexpr (OB) {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                             ((size_t)t.e * p.M + m) * p.N + n);
        uint32_t packed[16];
        pack_bf16(f, packed);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          o[w] = make_uint4(packed[4 * w], packed[4 * w + 1], packed[4 * w + 2],
                            packed[4 * w + 3]);
      } else {
        float *o = MODE != 2
                       ? static_cast<float *>(p.out) + pr * p.N + n
                       : static_cast<float *>(p.out) + ((size_t)t.e * p.M + m) * p.N + n;
#pragma unroll
        for (int w = 0; w < 8; ++w)
          reinterpret_cast<float4 *>(o)[w] =
              make_float4(f[4 * w], f[4 * w + 1], f[4 * w + 2], f[4 * w + 3]);
      }
    }
  }
  if (MODE == 0 && valid) p.dgpart[pr * p.n_blocks + t.nb] = part;
  if (bad) record_error(p.st, MOE_ERR_NONFINITE, (long long)(MODE == 2 ? m : (long long)pr));
}

// Mode 3's epilogue for one warp: its 32 rows and half of the tile's columns
// (half 0 or 1), 32 at a time; pre holds the first 32's p1 and p3, fetched before
// the accumulator was waited for. Global memory is read and written four lanes to a
// row (a lane to a row would touch 32 lines an instruction); p1 and p3 of the
// next 32 columns are fetched while these are worked on. They change to a lane's
// own row through the warp's two staging tiles, where dP1 and dP3 and then h take
// their places on the way back. Warp-collective.
struct GatedPre {
  uint4 v[2][4];  // p1, p3: 8 columns of rows lane / 4 + 8 i
  // Columns n .. n + 31 of the warp's rows from m0 on; zero past the expert's.
  __device__ __forceinline__ void fetch(const BParams &p, const BExtra<3> &ex, const BTile &t,
                                        int m0, int n) {
    const int sub = (threadIdx.x & 31) >> 2, quarter = threadIdx.x & 3;
    const int q0 = p.offset[t.e] + m0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = sub + 8 * i;
      const bool ok = m0 + row < t.rows && n < p.N;
      const size_t at = (size_t)(q0 + row) * p.N + n + quarter * 8;
      v[0][i] = ok ? *reinterpret_cast<const uint4 *>(ex.pre1 + at) : make_uint4(0, 0, 0, 0);
      v[1][i] = ok ? *reinterpret_cast<const uint4 *>(ex.pre3 + at) : make_uint4(0, 0, 0, 0);
    }
  }
};
template <int ACT>
__device__ __forceinline__ void epilogue_gated(const BParams &p, const BExtra<3> &ex,
                                               const BTile &t, int m0, int half,
                                               uint32_t lane_addr, float *stg, GatedPre &pre) {
  const int lane = threadIdx.x & 31;
  const int m = m0 + lane;
  if (m0 >= t.prows) return;  // padded rows come in 64s: all of the warp's or none
  const bool real = m < t.rows;
  const size_t pr = (size_t)t.prow0 + m;
  const int q0 = p.offset[t.e] + m0;  // packed row of the warp's first
  const float g = real ? p.row_gate[q0 + lane] : 0.f;
  float2 part = both(0.f), odd = both(0.f);
  const int sub = lane >> 2, quarter = lane & 3;
  uint4 *const tile = reinterpret_cast<uint4 *>(stg);
  constexpr int kTile = G_TILE / 4;  // in 16-byte pieces
  const auto piece = [&](int i) {  // of row sub + 8 i
    const int row = sub + 8 * i;
    return row * 4 + (quarter ^ ((row >> 1) & 3));
  };
  const int c0 = half * (BN / 64), x = (lane >> 1) & 3;
#pragma unroll 1
  for (int c = c0; c < c0 + BN / 64; ++c) {
    const int n = t.nb * BN + c * 32;
    if (n >= p.N) break;
    uint32_t v[32];
    tmem_ld32(lane_addr + (uint32_t)(c * 32), v);
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) tile[w * kTile + piece(i)] = pre.v[w][i];
    __syncwarp();
    if (c + 1 < c0 + BN / 64) pre.fetch(p, ex, t, m0, n + 32);
    uint4 hidden[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint4 *const at = tile + lane * 4 + (w ^ x);
      const uint4 u1 = at[0], u3 = at[kTile];
      const uint32_t a1[4] = {u1.x, u1.y, u1.z, u1.w}, a3[4] = {u3.x, u3.y, u3.z, u3.w};
      uint32_t o[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p3 = unpack2(a3[j]);
        float2 s;
        const float2 a = gated_act2<ACT, true>(unpack2(a1[j]), &s);
        const float2 D = make_float2(__uint_as_float(v[8 * w + 2 * j]),
                                     __uint_as_float(v[8 * w + 2 * j + 1]));
        const float2 gD = mul2(D, both(g)), h = mul2(a, p3);
        part = fma2(D, h, part);
        const float2 d1 = mul2(gD, mul2(p3, s)), d3 = mul2(gD, a);
        // 0 * d is 0, or a NaN that stays, for any number of places.
        odd = fma2(d1, both(0.f), fma2(d3, both(0.f), odd));
        o[0][j] = pack_bf16x2(d1);
        o[1][j] = pack_bf16x2(d3);
        o[2][j] = pack_bf16x2(mul2(h, both(g)));
      }
      if (!real) o[0][0] = o[0][1] = o[0][2] = o[0][3] = o[1][0] = o[1][1] = o[1][2] = o[1][3] = 0;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        at[q * kTile] = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
      hidden[w] = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = sub + 8 * i;
      const size_t at = (pr - lane + row) * p.N + n + quarter * 8;
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at) = tile[piece(i)];
      *reinterpret_cast<uint4 *>(ex.dP3 + at) = tile[kTile + piece(i)];
    }
    __syncwarp();
#pragma unroll
    for (int w = 0; w < 4; ++w) tile[lane * 4 + (w ^ x)] = hidden[w];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = sub + 8 * i;
      if (m0 + row < t.rows)
        *reinterpret_cast<uint4 *>(ex.h + (size_t)(q0 + row) * p.N + n + quarter * 8) =
            tile[piece(i)];
    }
    __syncwarp();  // read before the next columns are written
  }
  p.dgpart[(pr * p.n_blocks + t.nb) * 2 + half] = real ? part.x + part.y : 0.f;
  if (real && !(odd.x + odd.y == 0.f)) record_error(p.st, MOE_ERR_NONFINITE, (long long)pr);
}

// OB: in mode 2 the weight gradient is written in bf16, in mode 0 the hidden
// rows are read in 8 bits (a checkpoint's). ACT: mode 3's activation.
template <int MODE, bool OB = false, int ACT = 0>
__global__ void __launch_bounds__(threads_of<MODE>(), 1)
k_bwd_tc(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
         const __grid_constant__ BExtra<MODE> ex, const BParams p) {
  constexpr int STAGES = stages_of<MODE>(false);
  pdl_wait();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + STAGES * A_BYTES;
  float *stg_all = reinterpret_cast<float *>(sB + STAGES * B_BYTES);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sB + STAGES * B_BYTES +
                                                (MODE == 3 ? G_STG_BYTES : 0));
  uint64_t *full = bars, *empty = bars + STAGES;
  uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *tile_start = reinterpret_cast<int *>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], epi_warps<MODE>());
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Dgrad modes: tile prefix over experts, ceil(padded rows / BM) * n_blocks each.
  if (MODE != 2 && warp == 2) {
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int t = 0;
      if (e < p.E) t = (p.poff[e + 1] - p.poff[e] + BM - 1) / BM * p.n_blocks;
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < p.E) tile_start[e] = carry + incl - t;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tile_start[p.E] = carry;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total_tiles = MODE == 2 ? p.E * p.m_blocks * p.n_blocks : tile_start[p.E];

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------- producer
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total_tiles; tile += gridDim.x) {
        const BTile t = locate<MODE>(p, tile_start, tile);
        for (int kb = 0; kb < t.num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.st, 31, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_expect_tx(&full[s], STAGE_BYTES);
          if (MODE != 2) {
            const CUtensorMap *ta = &tmA, *tb = &tmB;
            int kx = kb * BK;
            if constexpr (MODE == 4) {
              if (kx >= p.K) {  // the second pair
                ta = &ex.a;
                tb = &ex.b;
                kx -= p.K;
              }
            }
            tma_load_2d(sA + s * A_BYTES, ta, &full[s], kx, t.prow0 + t.mb * BM);
            tma_load_2d(sB + s * B_BYTES, tb, &full[s], kx, t.e * p.N + t.nb * BN);
          } else {
            const int arow = p.offset[t.e] + kb * BK, brow = t.prow0 + kb * BK;
            tma_load_blocks(sA + s * A_BYTES, &tmA, &full[s], arow, t.mb * (BM / 64));
            tma_load_blocks(sB + s * B_BYTES, &tmB, &full[s], brow, t.nb * (BN / 64));
          }
        }
      }
      const uint32_t issued = it;
      for (uint32_t q = issued > (uint32_t)STAGES ? issued - STAGES : 0; q < issued; ++q)
        mbar_drain(&full[q % STAGES], (q / STAGES) & 1u);
    }
    __syncwarp();
    pdl_trigger();
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------- MMA issuer
      uint32_t it = 0;
      int local = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < total_tiles; tile += gridDim.x, ++local) {
        const BTile t = locate<MODE>(p, tile_start, tile);
        const int buf = local & 1;
        const uint32_t use = (uint32_t)(local >> 1);
        if (!mbar_wait(&acc_empty[buf], (use & 1u) ^ 1u, abort_flag, p.st, 32, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t tmem_d = tmem_base + (uint32_t)(buf * BN);
        for (int kb = 0; kb < t.num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!mbar_wait(&full[s], ph, abort_flag, p.st, 33, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * A_BYTES);
          const uint32_t b0 = smem_u32(sB + s * B_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            uint64_t ad, bd;
            if (MODE != 2) {
              ad = sdesc(a0 + kk * 32, 16, 1024);
              bd = sdesc(b0 + kk * 32, 16, 1024);
            } else {
              ad = sdesc(a0 + kk * 2048, BK * 128, 1024);
              bd = sdesc(b0 + kk * 2048, BK * 128, 1024);
            }
            umma_b<MODE>(tmem_d, ad, bd, (kb | kk) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&acc_full[buf]);
      }
      umma_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
    pdl_trigger();
  } else {
    // ----------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    const int r_in_tile = quad * 32 + lane;
    int local = 0;
    for (int tile = blockIdx.x; tile < total_tiles; tile += gridDim.x, ++local) {
      const BTile t = locate<MODE>(p, tile_start, tile);
      const int buf = local & 1;
      const uint32_t use = (uint32_t)(local >> 1);
      [[maybe_unused]] GatedPre pre;
      if constexpr (MODE == 3)
        pre.fetch(p, ex, t, t.mb * BM + quad * 32, t.nb * BN + ((warp - 2) >> 2) * (BN / 2));
      const bool ready = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], use & 1u, abort_flag,
                                                           p.st, 34, p.wait_ns));
      if (!ready) break;
      tc_fence_after();
      const int m = t.mb * BM + r_in_tile;
      const uint32_t lane_addr =
          tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN);
      if constexpr (MODE == 3)
        epilogue_gated<ACT>(p, ex, t, m - lane, (warp - 2) >> 2, lane_addr,
                            stg_all + (warp - 2) * 2 * G_TILE, pre);
      else
        epilogue_rows<MODE, OB>(p, t, m, lane_addr);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
    pdl_trigger();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

// ----------------------------------------------------------------------------- CTA-pair variant
// The same three modes with tcgen05.mma.cta_group::2: a cluster of two CTAs
// on two SMs computes a 256-row x 256-column tile; each CTA loads its own 128
// rows of A and 128 of the tile's 256 B columns (rows of the K-major weight
// in the dgrad modes, 64-column boxes of the MN-major rows in the weight
// gradient), so each SM takes in 32 KB per K step instead of 48 KB. The even
// CTA issues the MMAs; the odd CTA's copies complete on the even CTA's "full"
// barriers, commits arrive on both CTAs' barriers, and both CTAs' epilogues
// arrive on the even CTA's "accumulator empty" barriers (the forward's pair
// kernel, same protocol).
constexpr int P_A_BYTES = BM * BK * 2;          // 16 KB
constexpr int P_B_BYTES = BK * (BN / 2) * 2;    // 16 KB
constexpr int P_STAGE_BYTES = P_A_BYTES + P_B_BYTES;
// Weight-gradient epilogue staging: per epilogue warp two [32 rows x 32
// columns] fp32 tiles (4 KB each) in the 128-byte swizzle.
constexpr int P_STG_TILE = 32 * 32;  // floats
constexpr int P_STG_BYTES = 4 * 2 * P_STG_TILE * 4;

template <int MODE>
__host__ __device__ constexpr uint32_t bwd_idesc_pair() {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((MODE == 2 ? 1u : 0u) << 15) |
         ((MODE == 2 ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)(256 >> 4) << 24);
}

template <int MODE>
__device__ __forceinline__ void umma_b_pair(uint32_t tmem_d, uint64_t a, uint64_t b,
                                            uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
      "l"(a), "l"(b), "r"(bwd_idesc_pair<MODE>()), "r"(acc)
      : "memory");
}

// Pair tiles: dgrad modes over (expert, 256-row block, n block) with
// ceil(padded rows / 256) row blocks per expert; weight gradient over (expert,
// n block, 256-row block of the output) with ceil(M / 256) row blocks.
template <int MODE>
__device__ __forceinline__ BTile locate_pair(const BParams &p, const int *start, int tile) {
  BTile t;
  const int mb2 = (p.M + 2 * BM - 1) / (2 * BM);
  if (MODE == 2) {
    const int per = mb2 * p.n_blocks;
    t.e = tile / per;
    const int local = tile - t.e * per;
    wgrad_order(local, mb2, p.n_blocks, t.mb, t.nb);
  } else {
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= tile) lo = mid;
      else hi = mid;
    }
    t.e = lo;
  }
  t.prow0 = p.poff[t.e];
  t.prows = p.poff[t.e + 1] - t.prow0;
  t.rows = p.offset[t.e + 1] - p.offset[t.e];
  if (MODE != 2) {
    const int mt = (t.prows + 2 * BM - 1) / (2 * BM);
    const int local = tile - start[t.e];
    t.nb = local / mt;
    t.mb = local - t.nb * mt;
    t.num_kb = (MODE == 4 ? 2 : 1) * (p.K / BK);
  } else {
    t.num_kb = t.prows / BK;
  }
  return t;
}

// The weight-gradient epilogue of the CTA-pair kernel: this warp's 32 rows
// m0 .. m0+31 of expert e's dW tile, 32 columns at a time from TMEM into one
// of the warp's two staging tiles, then out by a TMA store into dW viewed as
// [E, M, N] (tmO), which drops rows past M and columns past N. The per-lane
// row stores of the other modes send 32 rows' 16-byte pieces per instruction;
// here each store writes whole 128-byte row segments, and the fp32 output
// (4 bytes per product of a K = rows-per-expert reduction) no longer holds
// the tensor pipe back. cnt counts this warp's staged chunks (buffer parity).
// OB: the tile in bf16 (64-byte rows, 64-byte swizzle), rounded once here.
template <bool OB>
__device__ __forceinline__ void epilogue_wgrad_tma(const BParams &p, const BTile &t, int m0,
                                                   uint32_t lane_addr, float *stg,
                                                   const CUtensorMap *tmO, uint32_t &cnt) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
#pragma unroll 1
  for (int c = 0; c < BN / 32; ++c) {
    const int n = t.nb * BN + c * 32;
    uint32_t v[32];
    tmem_ld32(lane_addr + (uint32_t)(c * 32), v);  // warp-collective
    if (n >= p.N) continue;
    float *buf = stg + (cnt & 1u) * P_STG_TILE;
    if (lane == 0) bulk_wait_read_but1();  // this buffer's previous store has read it
    __syncwarp();
    if constexpr (OB) {
      float f[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        f[j] = __uint_as_float(v[j]);
        bad |= !isfinite(f[j]);
      }
      uint32_t packed[16];
      pack_bf16(f, packed);
      uint4 *row = reinterpret_cast<uint4 *>(buf) + lane * 4;
      const int x = (lane >> 1) & 3;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        row[q ^ x] = make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2],
                                packed[4 * q + 3]);
    } else {
      float4 *row = reinterpret_cast<float4 *>(buf + lane * 32);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float4 f = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                     __uint_as_float(v[4 * q + 2]),
                                     __uint_as_float(v[4 * q + 3]));
        bad |= !isfinite(f.x) || !isfinite(f.y) || !isfinite(f.z) || !isfinite(f.w);
        row[q ^ (lane & 7)] = f;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(tmO, buf, n, m0, t.e);
      bulk_commit();
    }
    ++cnt;
  }
  if (bad && m0 + lane < p.M) record_error(p.st, MOE_ERR_NONFINITE, (long long)(m0 + lane));
}

// tmO: mode 2's output dW as [E, M, N] fp32, box [1, 32, 32], 128-byte
// swizzle; modes 0 and 1: the output [padded rows, N] (bf16 / fp32), box [32,
// 32], when p.tma_out is set.
template <int MODE, bool OB = false, int ACT = 0>
__global__ void __launch_bounds__(threads_of<MODE>(), 1)
k_bwd_tc_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmO, const __grid_constant__ BExtra<MODE> ex,
              const BParams p) {
  constexpr int P_STAGES = stages_of<MODE>(true);
  constexpr int kStgBytes = MODE == 3 ? G_STG_BYTES : P_STG_BYTES;
  pdl_wait();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + P_STAGES * P_A_BYTES;
  float *stg_all = reinterpret_cast<float *>(sB + P_STAGES * P_B_BYTES);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sB + P_STAGES * P_B_BYTES + kStgBytes);
  uint64_t *full = bars, *empty = bars + P_STAGES;
  uint64_t *acc_full = bars + 2 * P_STAGES, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  uint64_t *tfull = drain + 1, *tempty = tfull + kRing;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tempty + kRing);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *ring = reinterpret_cast<volatile int *>(tmem_slot + 2);
  int *tile_start = const_cast<int *>(ring + kRing);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * epi_warps<MODE>());
    }
    for (int r = 0; r < kRing; ++r) {
      mbar_init(&tfull[r], 1);
      mbar_init(&tempty[r], kRingConsumers + 2 * (epi_warps<MODE>() - 4));
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (MODE != 2 && warp == 2) {  // ceil(padded rows / 256) * n_blocks tiles per expert
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int t = 0;
      if (e < p.E) t = (p.poff[e + 1] - p.poff[e] + 2 * BM - 1) / (2 * BM) * p.n_blocks;
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < p.E) tile_start[e] = carry + incl - t;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tile_start[p.E] = carry;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int mb2 = (p.M + 2 * BM - 1) / (2 * BM);
  const int total_tiles = MODE == 2 ? p.E * mb2 * p.n_blocks : tile_start[p.E];

  if (warp == 0) {
    if (lane == 0) {
      // --------------------------------------------------------- producer (both CTAs)
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmA) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&tmB) : "memory");
      // Tiles: each pair's first is its index, every later one taken from the
      // counter by the even CTA's producer (the take issued a few k-blocks
      // before the current tile's last load) and published through the ring.
      uint32_t it = 0;
      bool ok = true;
      long long taken = -1;
      int tile_rr = pair;
      for (int j = 0; ok; ++j) {
        const int slot = j % kRing;
        const uint32_t rph = (uint32_t)(j / kRing) & 1u;
        int tile;
        if (leader) {
          if (j == 0) {
            tile = pair;
          } else if (p.dynamic) {
            if (taken < 0) taken = atomicAdd(p.sched, 1u);
            tile = (int)min(taken + n_pairs, (long long)total_tiles);
            taken = -1;
          } else {
            tile_rr += n_pairs;
            tile = min(tile_rr, total_tiles);
          }
          if (!mbar_wait_cl(&tempty[slot], rph ^ 1u, abort_flag, p.st, 45, p.wait_ns)) {
            ok = false;
            break;
          }
          ring[slot] = tile;
          st_cluster_u32(mapa(smem_u32((const void *)&ring[slot]), 1), (uint32_t)tile);
          mbar_arrive_cluster(smem_u32(&tfull[slot]));
          mbar_arrive_cluster(mapa(smem_u32(&tfull[slot]), 1));
        } else {
          if (!mbar_wait_cl(&tfull[slot], rph, abort_flag, p.st, 46, p.wait_ns)) {
            ok = false;
            break;
          }
          tile = ring[slot];
          mbar_arrive_cluster(mapa(smem_u32(&tempty[slot]), 0));
        }
        if (tile >= total_tiles) break;
        const BTile t = locate_pair<MODE>(p, tile_start, tile);
        const int take_at = t.num_kb > 4 ? t.num_kb - 4 : 0;
        // Odd waves of tiles walk K from the end, starting on the blocks the
        // wave before read last (still in L2); the order is fixed per tile.
        const bool rev = p.snake == 2 || (p.snake == 1 && ((tile / n_pairs) & 1));
        for (int kb = 0; kb < t.num_kb; ++kb, ++it) {
          if (leader && p.dynamic && kb == take_at) taken = atomicAdd(p.sched, 1u);
          const int s = it % P_STAGES;
          const uint32_t ph = (it / P_STAGES) & 1u;
          if (!mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.st, 41, p.wait_ns)) {
            ok = false;
            break;
          }
          const int kx = (rev ? t.num_kb - 1 - kb : kb) * BK;
          const uint32_t full_leader = mapa(smem_u32(&full[s]), 0);
          if (leader) mbar_expect_tx(&full[s], 2 * P_STAGE_BYTES);
          if (MODE != 2) {
            const CUtensorMap *ta = &tmA, *tb = &tmB;
            int kk = kx;
            if constexpr (MODE == 4) {
              if (kx >= p.K) {  // the second pair
                ta = &ex.a;
                tb = &ex.b;
                kk -= p.K;
              }
            }
            tma_load_2d_pair(sA + s * P_A_BYTES, ta, full_leader, kk,
                             t.prow0 + t.mb * 2 * BM + (int)rank * BM);
            tma_load_2d_pair(sB + s * P_B_BYTES, tb, full_leader, kk,
                             t.e * p.N + t.nb * BN + (int)rank * (BN / 2));
          } else {
            const int arow = p.offset[t.e] + kx, brow = t.prow0 + kx;
            const int mcol = t.mb * 2 * BM + (int)rank * BM;
            const int ncol = t.nb * BN + (int)rank * (BN / 2);
            tma_load_blocks_pair(sA + s * P_A_BYTES, &tmA, full_leader, arow, mcol / 64);
            tma_load_blocks_pair(sB + s * P_B_BYTES, &tmB, full_leader, brow, ncol / 64);
          }
        }
      }
      const uint32_t issued = it;
      for (uint32_t q = issued > (uint32_t)P_STAGES ? issued - P_STAGES : 0; q < issued; ++q)
        mbar_drain(&empty[q % P_STAGES], (q / P_STAGES) & 1u);
      if (leader && p.dynamic) {
        // The last pair to finish resets the counter for the next launch.
        __threadfence();
        if (atomicAdd(p.sched + 1, 1u) == (uint32_t)n_pairs - 1) {
          atomicExch(p.sched, 0u);
          atomicExch(p.sched + 1, 0u);
        }
      }
    }
    __syncwarp();
    pdl_trigger();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // --------------------------------------------------------- MMA issuer (even CTA)
      uint32_t it = 0;
      bool ok = true;
      for (int local = 0; ok; ++local) {
        const int slot = local % kRing;
        if (!mbar_wait_cl(&tfull[slot], (uint32_t)(local / kRing) & 1u, abort_flag, p.st, 47,
                          p.wait_ns))
          break;
        const int tile = ring[slot];
        mbar_arrive_cluster(smem_u32(&tempty[slot]));
        if (tile >= total_tiles) break;
        const BTile t = locate_pair<MODE>(p, tile_start, tile);
        const int buf = local & 1;
        const uint32_t use = (uint32_t)(local >> 1);
        if (!mbar_wait(&acc_empty[buf], (use & 1u) ^ 1u, abort_flag, p.st, 42, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t tmem_d = tmem_base + (uint32_t)(buf * BN);
        for (int kb = 0; kb < t.num_kb; ++kb, ++it) {
          const int s = it % P_STAGES;
          const uint32_t ph = (it / P_STAGES) & 1u;
          if (!mbar_wait(&full[s], ph, abort_flag, p.st, 43, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * P_A_BYTES);
          const uint32_t b0 = smem_u32(sB + s * P_B_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            uint64_t ad, bd;
            if (MODE != 2) {
              ad = sdesc(a0 + kk * 32, 16, 1024);
              bd = sdesc(b0 + kk * 32, 16, 1024);
            } else {
              ad = sdesc(a0 + kk * 2048, BK * 128, 1024);
              bd = sdesc(b0 + kk * 2048, BK * 128, 1024);
            }
            umma_b_pair<MODE>(tmem_d, ad, bd, (kb | kk) ? 1u : 0u);
          }
          umma_commit_pair(&empty[s]);
        }
        if (ok) umma_commit_pair(&acc_full[buf]);
      }
      umma_commit_pair(drain, 0x1);
      mbar_drain(drain, 0);
    }
    __syncwarp();
    pdl_trigger();
  } else {
    // ------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    const int r_in_tile = quad * 32 + lane;
    const uint32_t acc_empty_leader0 = mapa(smem_u32(&acc_empty[0]), 0);
    const uint32_t acc_empty_leader1 = mapa(smem_u32(&acc_empty[1]), 0);
    // This warp's two tiles (mode 3: of half the size).
    float *stg = stg_all + (size_t)(warp - 2) * (MODE == 3 ? 2 * G_TILE : 2 * P_STG_TILE);
    uint32_t stg_cnt = 0;
    for (int local = 0;; ++local) {
      const int slot = local % kRing;
      int tile = total_tiles;
      bool got = false;
      if (lane == 0) {
        got = mbar_wait_cl(&tfull[slot], (uint32_t)(local / kRing) & 1u, abort_flag, p.st, 48,
                           p.wait_ns);
        if (got) {
          tile = ring[slot];
          mbar_arrive_cluster(mapa(smem_u32(&tempty[slot]), 0));
        }
      }
      got = __shfl_sync(0xffffffffu, got, 0);
      tile = __shfl_sync(0xffffffffu, tile, 0);
      if (!got || tile >= total_tiles) break;
      const BTile t = locate_pair<MODE>(p, tile_start, tile);
      const int buf = local & 1;
      const uint32_t use = (uint32_t)(local >> 1);
      [[maybe_unused]] GatedPre pre;
      if constexpr (MODE == 3)
        pre.fetch(p, ex, t, t.mb * 2 * BM + (int)rank * BM + quad * 32,
                  t.nb * BN + ((warp - 2) >> 2) * (BN / 2));
      const bool ready = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], use & 1u, abort_flag,
                                                           p.st, 44, p.wait_ns));
      if (!ready) break;
      tc_fence_after();
      const int m = t.mb * 2 * BM + (int)rank * BM + r_in_tile;
      const uint32_t lane_addr =
          tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * BN);
      if constexpr (MODE == 2)
        epilogue_wgrad_tma<OB>(p, t, m - lane, lane_addr, stg, &tmO, stg_cnt);
      else if constexpr (MODE == 3)
        epilogue_gated<ACT>(p, ex, t, m - lane, (warp - 2) >> 2, lane_addr, stg, pre);
      else
        epilogue_rows<MODE, OB>(p, t, m, lane_addr, p.tma_out ? stg : nullptr, &tmO, &stg_cnt);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(buf ? acc_empty_leader1 : acc_empty_leader0);
    }
    if (lane == 0) bulk_wait_all();  // this warp's TMA stores are complete
    pdl_trigger();
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(TMEM_COLS)
                 : "memory");
  }
}

template <int MODE>
constexpr size_t bwd_smem_bytes_pair(int E) {
  constexpr int st = stages_of<MODE>(true);
  return 1024 + (size_t)st * P_STAGE_BYTES + (MODE == 3 ? G_STG_BYTES : P_STG_BYTES) +
         (2 * st + 5 + 2 * kRing) * 8 + 8 + (size_t)kRing * 4 + (size_t)(E + 1) * 4;
}

template <int MODE>
constexpr size_t bwd_smem_bytes(int E) {
  constexpr int st = stages_of<MODE>(false);
  return 1024 + (size_t)st * STAGE_BYTES + (MODE == 3 ? G_STG_BYTES : 0) + (2 * st + 5) * 8 + 8 +
         (size_t)(E + 1) * 4;
}

cudaLaunchAttribute cluster2_attr() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = 2;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// Clusters of two the pair kernel of this mode can keep resident (0 if none),
// for the shared-memory size of this E; looked up once per (mode, size).
template <int MODE>
int pair_clusters_bwd(size_t smem) {
  constexpr int kSlots = 8;
  static std::mutex mu;
  static size_t keys[kSlots];
  static int vals[kSlots];
  static int used = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (keys[i] == smem) return vals[i];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sm_count() / 2));
  cfg.blockDim = dim3(threads_of<MODE>());
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1] = {cluster2_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_smem(k_bwd_tc_pair<MODE>) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k_bwd_tc_pair<MODE>, &cfg) != cudaSuccess) {
    n = 0;
    cudaGetLastError();
  }
  if (used < kSlots) {
    keys[used] = smem;
    vals[used] = n;
    ++used;
  }
  return n;
}

template <int MODE, bool OB = false, int ACT = 0>
cudaError_t launch_mode_pair(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &o,
                             const BParams &p, int clusters, cudaStream_t s,
                             const BExtra<MODE> &ex = {}) {
  const size_t smem = bwd_smem_bytes_pair<MODE>(p.E);
  cudaError_t err = allow_smem(k_bwd_tc_pair<MODE, OB, ACT>);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(threads_of<MODE>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {cluster2_attr(), {}};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled(kPdlGemm) ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_bwd_tc_pair<MODE, OB, ACT>, a, b, o, ex, p);
}

template <int MODE, bool OB = false, int ACT = 0>
cudaError_t launch_mode(const CUtensorMap &a, const CUtensorMap &b, const BParams &p,
                        cudaStream_t s, const BExtra<MODE> &ex = {}) {
  const size_t smem = bwd_smem_bytes<MODE>(p.E);
  cudaError_t err = allow_smem(k_bwd_tc<MODE, OB, ACT>);
  if (err != cudaSuccess) return err;
  launch_pdl_c(kPdlGemm, k_bwd_tc<MODE, OB, ACT>, sm_count(), threads_of<MODE>(), smem, s, a, b, ex,
               p);
  return cudaGetLastError();
}

// 3-D tensor [E, M, N], fp32 (N % 4 == 0) or bf16 (N % 8 == 0): the weight
// gradient, box [1, 32 rows, 32 columns] in the 128-byte (bf16: 64-byte)
// swizzle, for the CTA-pair kernel's TMA stores (rows past M and columns past
// N of a box are not written).
bool make_out_map3(CUtensorMap *m, void *base, int E, int M, int N, bool bf16) {
  auto fn = encode_fn();
  if (!fn || N % (bf16 ? 8 : 4) != 0) return false;
  const cuuint64_t eb = bf16 ? 2 : 4;
  cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)M, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)N * eb, (cuuint64_t)M * N * eb};
  cuuint32_t box[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base,
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            bf16 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


}  // namespace

bool bwd_tc_supported(const moe_config &c) {
  return c.act_dtype == MOE_BF16 && c.d % 64 == 0 && c.d_ff % 64 == 0 &&
         bwd_smem_bytes<0>(c.E) <= 227 * 1024 && encode_fn() != nullptr;
}

// MOE_BWD_TC_VARIANT=single or =pair forces one kernel (read at each call);
// otherwise the CTA pair runs where its reduction is long (K >= 1024; for the
// weight gradient, the rows per expert, bounded by the capacity) and it has
// at least pair_waves (four, unless the caller measured otherwise) waves of 256 x
// 256 tiles.
static int bwd_variant() {
  const char *v = getenv("MOE_BWD_TC_VARIANT");
  if (!v || !*v) return 0;
  return v[0] == 's' ? 1 : (v[0] == 'p' ? 2 : 0);
}

template <int MODE>
static int pick_pair(const BwdGemm &g, long long k_len, long long tiles) {
  const int force = bwd_variant();
  if (force == 1 || bwd_smem_bytes_pair<MODE>(g.E) > 227 * 1024) return 0;
  const int clusters = pair_clusters_bwd<MODE>(bwd_smem_bytes_pair<MODE>(g.E));
  if (clusters <= 0) return 0;
  if (force == 2) return clusters;
  return (k_len >= 1024 && tiles >= (long long)g.pair_waves * clusters) ? clusters : 0;
}

cudaError_t launch_bwd_gemm(const BwdGemm &g, DeviceStatus *st, cudaStream_t s) {
  CUtensorMap ta, tb;
  BParams p{};
  p.mode = g.mode;
  p.K = g.K;
  p.N = g.N;
  p.M = g.M;
  p.E = g.E;
  p.n_blocks = (g.N + BN - 1) / BN;
  p.m_blocks = (g.M + BM - 1) / BM;
  p.offset = g.offset;
  p.poff = g.poff;
  p.row_gate = g.row_gate;
  p.hbuf = static_cast<const __nv_bfloat16 *>(g.hbuf);
  p.h8 = g.h8;
  p.hscale = g.hscale;
  p.out = g.out;
  p.dgpart = g.dgpart;
  p.st = st;
  p.wait_ns = wait_limit_ns();
  p.sched = &st->gemm_next;  // gemm_next, gemm_done: adjacent words
  {
    const char *v = getenv("MOE_FFN_SCHED");  // =static: round robin (for comparisons)
    p.dynamic = v && v[0] == 's' ? 0 : 1;
    // =0: every tile's K forward, =all: every tile's backwards (comparisons, tests)
    const char *sv = getenv("MOE_FFN_SNAKE");
    p.snake = !sv || !*sv ? 1 : (sv[0] == '0' ? 0 : (sv[0] == 'a' ? 2 : 1));
  }
  const long long nb = (g.N + BN - 1) / BN;
  if (g.mode == 2) {
    // A: the forward's packed rows [a_rows, M]; B: padded rows [b_rows, N].
    CUtensorMap to;
    int cl = pick_pair<2>(g, g.k_len, (long long)g.E * ((g.M + 255) / 256) * nb);
    if ((uintptr_t)g.out % 16 != 0 || !make_out_map3(&to, g.out, g.E, g.M, g.N, g.out_bf16)) cl = 0;
    if (!make_blocks_map(&ta, g.A, (uint64_t)g.a_rows, (uint64_t)g.M, 64, BM / 64) ||
        !make_blocks_map(&tb, g.B, (uint64_t)g.b_rows, (uint64_t)g.N, 64, cl > 0 ? 2 : 4))
      return cudaErrorInvalidValue;
    if (cl > 0)
      return g.out_bf16 ? launch_mode_pair<2, true>(ta, tb, to, p, cl, s)
                        : launch_mode_pair<2>(ta, tb, to, p, cl, s);
    return g.out_bf16 ? launch_mode<2, true>(ta, tb, p, s) : launch_mode<2>(ta, tb, p, s);
  }
  // A: padded rows [a_rows, K]; B: the weight as [E*N rows, K] (the pair
  // kernel loads half of a tile's 256 B rows per CTA).
  const long long tiles = (g.a_rows + 255) / 256 * nb;
  const int cl = g.mode == 0   ? pick_pair<0>(g, g.K, tiles)
                 : g.mode == 1 ? pick_pair<1>(g, g.K, tiles)
                 : g.mode == 3 ? pick_pair<3>(g, g.K, tiles)
                               : pick_pair<4>(g, 2ll * g.K, tiles);
  const uint64_t rows = (uint64_t)g.a_rows, wrows = (uint64_t)g.E * g.N;
  const uint32_t box_b = cl > 0 ? BN / 2 : BN;
  if (!make_map(&ta, g.A, rows, (uint64_t)g.K, BM) ||
      !make_map(&tb, g.B, wrows, (uint64_t)g.K, box_b))
    return cudaErrorInvalidValue;
  CUtensorMap to = ta;  // unused unless p.tma_out
  if (g.mode == 3) {
    BExtra<3> ex{};
    ex.pre1 = static_cast<const __nv_bfloat16 *>(g.pre1);
    ex.pre3 = static_cast<const __nv_bfloat16 *>(g.pre3);
    ex.dP3 = static_cast<__nv_bfloat16 *>(g.out3);
    ex.h = static_cast<__nv_bfloat16 *>(g.h);
    return gated_dispatch(g.activation, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      return cl > 0 ? launch_mode_pair<3, false, ACT>(ta, tb, to, p, cl, s, ex)
                    : launch_mode<3, false, ACT>(ta, tb, p, s, ex);
    });
  }
  BExtra<4> ex4{};
  if (g.mode == 4 && (!make_map(&ex4.a, g.A3, rows, (uint64_t)g.K, BM) ||
                      !make_map(&ex4.b, g.B3, wrows, (uint64_t)g.K, box_b)))
    return cudaErrorInvalidValue;
  if (cl > 0) {
    p.tma_out = make_rows_map(&to, g.out, rows, (uint64_t)g.N, g.mode != 0) ? 1 : 0;
    if (g.mode == 4) return launch_mode_pair<4>(ta, tb, to, p, cl, s, ex4);
    if (g.mode == 0 && g.h8) return launch_mode_pair<0, true>(ta, tb, to, p, cl, s);
    return g.mode == 0 ? launch_mode_pair<0>(ta, tb, to, p, cl, s)
                       : launch_mode_pair<1>(ta, tb, to, p, cl, s);
  }
  if (g.mode == 4) return launch_mode<4>(ta, tb, p, s, ex4);
  if (g.mode == 0 && g.h8) return launch_mode<0, true>(ta, tb, p, s);
  return g.mode == 0 ? launch_mode<0>(ta, tb, p, s) : launch_mode<1>(ta, tb, p, s);
}

}  // namespace moe
