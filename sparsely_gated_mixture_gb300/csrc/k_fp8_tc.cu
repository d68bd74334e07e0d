// The gated experts' products in 8 bits on the 5th-generation tensor cores:
//   layer 1: p1 = x W1 + b1, p3 = x W3 + b3, h = act(p1) * p3, rounded to bf16
//            and put in 8 bits with a scale for each 128 columns
//   layer 2: z = gate * (h W2 + b2)
// tcgen05.mma kind::mxf8f6f4 takes e4m3 operands and applies a power-of-two
// scale to each row and 32 values of K as it multiplies: a byte of a TMEM word
// for each row, which of the four is in the instruction. The four MMAs of a block
// of 128 take the same byte, so a word serves four blocks of K. Operands are K-major, 128 bytes
// of K a stage, as the bf16 kernels' 64 values; so are the tiles, 128 rows (a
// CTA) or 256 (a pair of CTAs) by 256 columns, in layer 1 128 of W1 and the
// same 128 of W3: one accumulator holds p1 and p3 of the same places, and a
// thread all 128 of its row's hidden values that share a scale.
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM owner, 2 scales, 4-7 epilogue.
// The scale warp has a ring of its own, a slot for four K blocks, in the form
// that tcgen05.cp takes to TMEM: 16 bytes for a lane's rows l, l + 32, l + 64, l
// + 96. It reads the next four blocks' bytes before it waits for a slot.
//
// TMEM: two accumulators of 256 columns and 2 x 12 columns of scales are more
// than its 512, so the accumulators lie at columns 0 and 224. The epilogue takes
// the 32 columns that they share first and reports them (ovl), and the MMAs of
// the next tile wait for that alone beside their own accumulator.
#include "gated.cuh"
#include "tc_ptx.cuh"

#include <stdlib.h>

#include <mutex>

namespace moe {
namespace {

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int kThreads = 256;
constexpr int A_BYTES = BM * BK;           // 16 KB
constexpr int S_BYTES = 512 + 1024;        // scales of 128 rows and 256 columns
constexpr int TMEM_COLS = 512, ACC1 = 224, SF_COL = 480;
constexpr int SF_SLOTS = 4;                // of four K blocks' scales each
constexpr int STG_TILE = 32 * 32 / 2;      // floats: [32 x 32] bf16 or [32 x 16] fp32
template <int CG>
__host__ __device__ constexpr int stages_of() { return CG == 2 ? 6 : 4; }
template <int CG>
__host__ __device__ constexpr int b_bytes() { return BN / CG * BK; }
constexpr int STG_BYTES = 4 * 2 * STG_TILE * 4;

struct Params {
  int K, N, E, KB, NB, n_blocks, max_rows;  // KB, NB: scale blocks of K and of a weight's N
  const int32_t *offset;
  const float *row_gate;
  const uint32_t *sa;          // [KB / 4][max_rows]: bytes of four K blocks
  const uint8_t *sb, *sb3;     // [E][NB][KB]
  const __nv_bfloat16 *bias, *bias3;
  uint8_t *h8, *sh;            // layer 1: [max_rows][128 NB], [NB / 4][max_rows][4]
  void *z;                     // layer 2: [max_rows][N] fp32 or bf16
  int z_bf16, tma_out;
  DeviceStatus *st;
  unsigned long long wait_ns;
};

// kind::mxf8f6f4: e4m3 both, both K-major, fp32 accumulate, scales UE8M0 (bit
// 23), byte `id` of the scales' words (bits 4 and 29).
__device__ __forceinline__ uint32_t idesc_of(int cg, uint32_t id) {
  return ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(BM * cg >> 4) << 24) | id << 4 |
         id << 29;
}

template <int CG>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t sfa, uint32_t sfb,
                                     uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes, one after the other) to four TMEM
// columns, the same in each quarter of the lanes.
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t smem) {
  // No swizzle; 8 rows are 128 bytes, and so is the way to the next 8.
  const uint64_t d = (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 |
                     (uint64_t)1 << 46;
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

template <int CG>
__device__ __forceinline__ void commit8(uint64_t *bar) {
  if constexpr (CG == 2) umma_commit_pair(bar);
  else umma_commit(bar);
}

// Loads into this CTA; the bytes count on `bar` (a pair's: the even CTA's).
template <int CG>
__device__ __forceinline__ void load_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                          int y) {
  if constexpr (CG == 2) tma_load_2d_pair(dst, map, mapa(smem_u32(bar), 0), x, y);
  else tma_load_2d(dst, map, bar, x, y);
}
template <int CG>
__device__ __forceinline__ void load_weight(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                            int y, int z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)map), "r"(mapa(smem_u32(bar), 0)), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Two values of a bias of any width; zero past it.
__device__ __forceinline__ float2 bias2(const __nv_bfloat16 *b, int e, int n, int N) {
  const __nv_bfloat16 *at = b + (size_t)e * N + n;
  return make_float2(n < N ? __bfloat162float(at[0]) : 0.f,
                     n + 1 < N ? __bfloat162float(at[1]) : 0.f);
}

struct Tile {
  int e, mb, nb, row0, rows;
};

// tmA: rows [max_rows, 128 KB], box [128, 128]; tmB, tmB3: weights [E, N, 128
// KB], box [1, 128, 128] (layer 2: tmB3 is tmB); tmO: z [max_rows, N], box [32, 32]
// (fp32: [32, 16]).
template <int LAYER, int ACT, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_fp8_tc(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
         const __grid_constant__ CUtensorMap tmB3, const __grid_constant__ CUtensorMap tmO,
         const Params p) {
  pdl_wait();
  constexpr int STAGES = stages_of<CG>(), B_BYTES = b_bytes<CG>();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = sA + STAGES * A_BYTES;
  float *stg_all = reinterpret_cast<float *>(sB + STAGES * B_BYTES);
  uint8_t *sS = reinterpret_cast<uint8_t *>(stg_all) + STG_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sS + SF_SLOTS * S_BYTES);
  uint64_t *full = bars, *empty = full + STAGES;
  uint64_t *acc_full = empty + STAGES, *acc_empty = acc_full + 2, *ovl = acc_empty + 2;
  uint64_t *sf_full = ovl + 2, *sf_empty = sf_full + SF_SLOTS, *drain = sf_empty + SF_SLOTS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *tile_start = reinterpret_cast<int *>(tmem_slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const bool leader = rank == 0;
  const int unit = (int)blockIdx.x / CG, n_units = (int)gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < SF_SLOTS; ++s) {
      mbar_init(&sf_full[s], CG);  // each CTA's scale warp
      mbar_init(&sf_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4 * CG);
      mbar_init(&ovl[b], 4 * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {  // ceil(rows / (128 CG)) * n_blocks tiles an expert
    int carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int t = 0;
      if (e < p.E)
        t = (p.offset[e + 1] - p.offset[e] + CG * BM - 1) / (CG * BM) * p.n_blocks;
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
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(TMEM_COLS)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = tile_start[p.E];
  const auto locate = [&](int tile) {
    int lo = 0, hi = p.E;  // largest e with tile_start[e] <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= tile) lo = mid;
      else hi = mid;
    }
    Tile t;
    t.e = lo;
    t.row0 = p.offset[lo];
    t.rows = p.offset[lo + 1] - t.row0;
    const int mt = (t.rows + CG * BM - 1) / (CG * BM), local = tile - tile_start[lo];
    t.nb = local / mt;
    t.mb = local - t.nb * mt;
    return t;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------- producer (both CTAs)
      uint32_t it = 0;
      bool ok = true;
      for (int tile = unit; ok && tile < total; tile += n_units) {
        const Tile t = locate(tile);
        const int arow = t.row0 + (t.mb * CG + (int)rank) * BM;
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&empty[s], ((it / STAGES) & 1u) ^ 1u, abort_flag, p.st, 121, p.wait_ns)) {
            ok = false;
            break;
          }
          if (leader) mbar_expect_tx(&full[s], CG * (A_BYTES + B_BYTES));
          load_rows<CG>(sA + s * A_BYTES, &tmA, &full[s], kb * BK, arow);
#pragma unroll
          for (int q = 0; q < 2 / CG; ++q) {
            const int half = CG == 2 ? (int)rank : q;  // of the tile's 256 columns
            load_weight<CG>(sB + s * B_BYTES + q * (128 * BK), LAYER == 1 && half ? &tmB3 : &tmB,
                            &full[s], kb * BK,
                            LAYER == 1 ? t.nb * 128 : t.nb * BN + half * 128, t.e);
          }
        }
      }
      // Copies in flight land first. The odd CTA's count on the even one's barriers:
      // they have landed once their MMAs are done.
      const uint32_t issued = it;
      for (uint32_t q = issued > (uint32_t)STAGES ? issued - STAGES : 0; q < issued; ++q)
        mbar_drain(leader ? &full[q % STAGES] : &empty[q % STAGES], (q / STAGES) & 1u);
    }
    __syncwarp();
    pdl_trigger();
  } else if (warp == 2) {
    // --------------------------------------------------------------- scales (both CTAs)
    // Lane l < 8 reads column block l / 4's byte of K block l % 4 of a group.
    const int half = (lane >> 2) & 1;
    int tile = unit, k0 = 0;  // the next group to read
    Tile t{};
    uint32_t a[4], b = 0;
    const auto read = [&] {
      if (k0 == 0) t = locate(tile);
      const int arow = t.row0 + (t.mb * CG + (int)rank) * BM;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = arow + lane + 32 * j;
        a[j] = row < p.max_rows ? p.sa[(size_t)(k0 >> 2) * p.max_rows + row] : 0x7f7f7f7fu;
      }
      const int nb = LAYER == 1 ? t.nb : min(2 * t.nb + half, p.NB - 1), kb = k0 + (lane & 3);
      const uint8_t *sb = (LAYER == 1 && half ? p.sb3 : p.sb) + ((size_t)t.e * p.NB + nb) * p.KB;
      b = lane < 8 && kb < p.KB ? (uint32_t)sb[kb] << 8 * (lane & 3) : 0u;
      k0 += 4;
      if (k0 >= p.KB) {
        k0 = 0;
        tile += n_units;
      }
    };
    bool more = tile < total;
    if (more) read();
    for (uint32_t g = 0; more; ++g) {
      const uint4 av = make_uint4(a[0], a[1], a[2], a[3]);
      uint32_t w = b | __shfl_xor_sync(0xffffffffu, b, 1);
      w |= __shfl_xor_sync(0xffffffffu, w, 2);
      const uint32_t b0 = __shfl_sync(0xffffffffu, w, 0), b1 = __shfl_sync(0xffffffffu, w, 4);
      more = tile < total;
      if (more) read();  // the next group's, in flight over the wait
      const int s = g % SF_SLOTS;
      if (!__all_sync(0xffffffffu, mbar_wait(&sf_empty[s], ((g / SF_SLOTS) & 1u) ^ 1u, abort_flag,
                                             p.st, 122, p.wait_ns)))
        break;
      uint4 *out = reinterpret_cast<uint4 *>(sS + s * S_BYTES) + lane;
      out[0] = av;
      out[32] = make_uint4(b0, b0, b0, b0);
      out[64] = make_uint4(b1, b1, b1, b1);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(mapa(smem_u32(&sf_full[s]), 0));
        else mbar_arrive(&sf_full[s]);
      }
    }
    pdl_trigger();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------- MMA issuer
      uint32_t it = 0, g = 0;  // K blocks, groups of four
      int local = 0;
      bool ok = true;
      for (int tile = unit; ok && tile < total; tile += n_units, ++local) {
        const int buf = local & 1, prev = local - 1;
        if (!mbar_wait(&acc_empty[buf], ((local >> 1) & 1u) ^ 1u, abort_flag, p.st, 123,
                       p.wait_ns))
          break;
        if (local > 0 && !mbar_wait(&ovl[prev & 1], (prev >> 1) & 1u, abort_flag, p.st, 124,
                                    p.wait_ns))
          break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(buf ? ACC1 : 0);
        uint32_t sf = 0;
        for (int kb = 0; kb < p.KB; ++kb, ++it) {
          if ((kb & 3) == 0) {
            const int q = g % SF_SLOTS;
            const uint32_t ph = (g / SF_SLOTS) & 1u;
            if (!(CG == 2 ? mbar_wait_cl(&sf_full[q], ph, abort_flag, p.st, 127, p.wait_ns)
                          : mbar_wait(&sf_full[q], ph, abort_flag, p.st, 127, p.wait_ns))) {
              ok = false;
              break;
            }
            tc_fence_after();
            // Copies and MMAs run in order, so this slot's last readers are done.
            sf = tmem + SF_COL + (g & 1u) * 16;
            const uint32_t ss = smem_u32(sS + q * S_BYTES);
            copy_scales<CG>(sf, ss);
            copy_scales<CG>(sf + 4, ss + 512);
            copy_scales<CG>(sf + 8, ss + 1024);
            commit8<CG>(&sf_empty[q]);
            ++g;
          }
          const int s = it % STAGES;
          if (!mbar_wait(&full[s], (it / STAGES) & 1u, abort_flag, p.st, 125, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * A_BYTES), b0 = smem_u32(sB + s * B_BYTES);
          const uint32_t idesc = idesc_of(CG, (uint32_t)kb & 3u);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mma8<CG>(d, sdesc(a0 + kk * 32, 16, 1024), sdesc(b0 + kk * 32, 16, 1024), sf, sf + 4,
                     idesc, (kb | kk) ? 1u : 0u);
          commit8<CG>(&empty[s]);
        }
        if (ok) commit8<CG>(&acc_full[buf]);
      }
      if constexpr (CG == 2) umma_commit_pair(drain, 0x1);
      else umma_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncwarp();
    pdl_trigger();
  } else if (warp >= 4) {
    // --------------------------------------------------------------- epilogue (both CTAs)
    const int quad = warp & 3;
    float *stg = stg_all + quad * 2 * STG_TILE;
    uint32_t stg_cnt = 0;
    const auto arrive = [&](uint64_t *bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_remote(mapa(smem_u32(bar), 0));
        else mbar_arrive(bar);
      }
    };
    int local = 0;
    for (int tile = unit; tile < total; tile += n_units, ++local) {
      const Tile t = locate(tile);
      const int buf = local & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], (local >> 1) & 1u, abort_flag, p.st,
                                             126, p.wait_ns)))
        break;
      tc_fence_after();
      const int m0 = (t.mb * CG + (int)rank) * BM + quad * 32, m = m0 + lane;
      const bool valid = m < t.rows;
      const size_t r = (size_t)t.row0 + m;
      const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf ? ACC1 : 0);
      // The shared columns first: the last ones of accumulator 0, the first of 1.
      if constexpr (LAYER == 1) {
        uint32_t h[4][16];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = buf ? i : 3 - i, n = t.nb * 128 + c * 32;
          uint32_t v1[32], v3[32];
          tmem_ld32(acc + c * 32, v1);
          tmem_ld32(acc + 128 + c * 32, v3);
          if (i == 0) arrive(&ovl[buf]);
          if (i == 3) arrive(&acc_empty[buf]);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 p1 = make_float2(__uint_as_float(v1[2 * j]), __uint_as_float(v1[2 * j + 1]));
            float2 p3 = make_float2(__uint_as_float(v3[2 * j]), __uint_as_float(v3[2 * j + 1]));
            if (p.bias) p1 = add2(p1, bias2(p.bias, t.e, n + 2 * j, p.N));
            if (p.bias3) p3 = add2(p3, bias2(p.bias3, t.e, n + 2 * j, p.N));
            h[i][j] = pack_bf16x2(mul2(gated_act2<ACT, false>(p1, nullptr), p3));
            const float2 f = unpack2(h[i][j]);
            top = max_nan(top, max_nan(fabsf(f.x), fabsf(f.y)));
          }
        }
        if (valid) {
          const uint32_t byte = fp8_scale_byte(top);
          const float inv = fp8_inverse(byte);
          p.sh[((size_t)(t.nb >> 2) * p.max_rows + r) * 4 + (t.nb & 3)] = (uint8_t)byte;
          uint4 *out = reinterpret_cast<uint4 *>(p.h8 + (r * p.NB + t.nb) * 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = buf ? i : 3 - i;
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 lo = mul2(unpack2(h[i][2 * j]), both(inv));
              const float2 hi = mul2(unpack2(h[i][2 * j + 1]), both(inv));
              w[j] = fp8_pack2(lo.x, lo.y) | fp8_pack2(hi.x, hi.y) << 16;
            }
            out[2 * c] = make_uint4(w[0], w[1], w[2], w[3]);
            out[2 * c + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      } else {
        const float g = valid ? p.row_gate[r] : 0.f;
        const bool tma = p.tma_out && m0 + 32 <= t.rows;
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const int c = buf ? i : 7 - i, n = t.nb * BN + c * 32;
          uint32_t v[32];
          tmem_ld32(acc + c * 32, v);
          if (i == 0) arrive(&ovl[buf]);
          if (i == 7) arrive(&acc_empty[buf]);
          if (!valid || n >= p.N) continue;
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            f[j] = __uint_as_float(v[j]);
            if (p.bias && n + j < p.N) f[j] += __bfloat162float(p.bias[(size_t)t.e * p.N + n + j]);
            f[j] *= g;
            bad |= n + j < p.N && !isfinite(f[j]);
          }
          uint32_t packed[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
            packed[j] = *reinterpret_cast<uint32_t *>(&b);
          }
          if (tma) {
            float *to = stg + (stg_cnt++ & 1u) * STG_TILE;
            if (p.z_bf16) {
              stage_store_bf16(&tmO, to, packed, n, t.row0 + m0);
            } else {
              stage_store_f32x16(&tmO, to, f, n, t.row0 + m0);
              to = stg + (stg_cnt++ & 1u) * STG_TILE;
              stage_store_f32x16(&tmO, to, f + 16, n + 16, t.row0 + m0);
            }
          } else if (p.z_bf16) {  // N is a multiple of 8
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.z) + r * p.N + n);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + 8 * q < p.N)
                o[q] = make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2],
                                  packed[4 * q + 3]);
          } else {
            float *o = static_cast<float *>(p.z) + r * p.N + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (n + j < p.N) o[j] = f[j];
          }
        }
        if (bad) record_error(p.st, MOE_ERR_NONFINITE, (long long)r);
      }
    }
    if (lane == 0) bulk_wait_all();
    pdl_trigger();
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TMEM_COLS)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TMEM_COLS)
                   : "memory");
  }
}

template <int CG>
constexpr size_t smem_bytes(int E) {
  return 1024 + (size_t)stages_of<CG>() * (A_BYTES + b_bytes<CG>()) + SF_SLOTS * S_BYTES +
         STG_BYTES + (2 * stages_of<CG>() + 2 * SF_SLOTS + 7) * 8 + 8 + (size_t)(E + 1) * 4;
}
static_assert(smem_bytes<1>(1024) <= 227 * 1024 && smem_bytes<2>(1024) <= 227 * 1024, "");

// Rows [rows, cols] of bytes (cols a multiple of 128), box [128, 128].
bool map_rows8(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
  cuuint32_t box[2] = {BK, BM}, one[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weights [E, N, cols] of bytes, box [1, 128, 128]; rows past N read as zero.
bool map_weight8(CUtensorMap *m, const void *base, uint64_t E, uint64_t N, uint64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, N, E}, strides[2] = {cols, cols * N};
  cuuint32_t box[3] = {BK, 128, 1}, one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int LAYER, int ACT, int CG>
cudaError_t run(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &b3,
                const CUtensorMap &o, const Params &p, int units, cudaStream_t s) {
  const size_t smem = smem_bytes<CG>(p.E);
  const cudaError_t err = allow_smem(k_fp8_tc<LAYER, ACT, CG>);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CG * units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled(kPdlGemm) ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_tc<LAYER, ACT, CG>, a, b, b3, o, p);
}

// Pairs of CTAs that can be resident at once (0 if none); E <= 1024 all take the
// same shared memory to within 4 KB, so the largest stands for all.
int pair_units() {
  static std::mutex mu;
  static int known = -1;
  std::lock_guard<std::mutex> lock(mu);
  if (known >= 0) return known;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sm_count() / 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<2>(1024);
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (allow_smem(k_fp8_tc<2, 0, 2>) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k_fp8_tc<2, 0, 2>, &cfg) != cudaSuccess) {
    n = 0;
    cudaGetLastError();
  }
  known = n;
  return n;
}

// MOE_FFN_TC_VARIANT=single or =pair forces one form (read at each call).
int forced() {
  const char *v = getenv("MOE_FFN_TC_VARIANT");
  if (!v || !*v) return 0;
  return v[0] == 's' ? 1 : (v[0] == 'p' ? 2 : 0);
}

}  // namespace

bool fp8_tc_supported() { return encode_fn() != nullptr; }

cudaError_t launch_fp8_tc(const Fp8Layer &q, cudaStream_t s) {
  const int K = q.layer == 1 ? q.c.d : q.c.d_ff, N = q.layer == 1 ? q.c.d_ff : q.c.d;
  Params p{};
  p.K = K;
  p.N = N;
  p.E = q.c.E;
  p.KB = (int)fp8_blocks(K);
  p.NB = (int)fp8_blocks(N);
  p.n_blocks = q.layer == 1 ? p.NB : (N + BN - 1) / BN;
  p.max_rows = q.max_rows;
  p.offset = q.offset;
  p.row_gate = q.row_gate;
  p.sa = reinterpret_cast<const uint32_t *>(q.sa);
  p.sb = q.sb;
  p.sb3 = q.layer == 1 ? q.sb3 : q.sb;
  p.bias = static_cast<const __nv_bfloat16 *>(q.bias);
  p.bias3 = static_cast<const __nv_bfloat16 *>(q.bias3);
  p.h8 = q.h8;
  p.sh = q.sh;
  p.z = q.z;
  p.z_bf16 = q.z_bf16 ? 1 : 0;
  p.st = q.st;
  p.wait_ns = wait_limit_ns();
  const uint64_t cols = (uint64_t)p.KB * BK;
  CUtensorMap ta, tb, tb3, to;
  if (!map_rows8(&ta, q.a8, (uint64_t)q.max_rows, cols) ||
      !map_weight8(&tb, q.W, (uint64_t)p.E, (uint64_t)N, cols) ||
      !map_weight8(&tb3, q.layer == 1 ? q.W3 : q.W, (uint64_t)p.E, (uint64_t)N, cols))
    return cudaErrorInvalidValue;
  to = ta;  // unused unless p.tma_out
  if (q.layer == 2)
    p.tma_out = q.z_bf16 ? make_rows_map(&to, q.z, (uint64_t)q.max_rows, (uint64_t)N, false)
                         : make_rows_map16(&to, q.z, (uint64_t)q.max_rows, (uint64_t)N);
  // The CTA pairs where the bf16 layers take theirs. Here they gain nothing: a stage
  // holds twice the K (8192 tokens, top-2 of 8 experts, one CTA and pairs forced: d =
  // d_ff = 1024 119 and 123 us, 1536 190 and 192, 2048 247 and 251, 4096 684 and 690;
  // 4096 x 14336 2049 and 2071).
  const long long tiles = (q.max_rows / 256) * (long long)p.n_blocks;
  const int pairs = forced() == 1 ? 0 : pair_units();
  const bool pair = pairs > 0 && (forced() == 2 || (K >= 2048 && tiles >= 4ll * pairs));
  if (q.layer == 2)
    return pair ? run<2, 0, 2>(ta, tb, tb3, to, p, pairs, s)
                : run<2, 0, 1>(ta, tb, tb3, to, p, sm_count(), s);
  return gated_dispatch(q.activation, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    return pair ? run<1, ACT, 2>(ta, tb, tb3, to, p, pairs, s)
                : run<1, ACT, 1>(ta, tb, tb3, to, p, sm_count(), s);
  });
}

}  // namespace moe
