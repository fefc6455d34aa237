// Product of MXFP4 activations and MXFP4 weights on the block-scaled 4-bit tensor cores.
#include <algorithm>

#include "qe_internal.h"
#include "qe_ptx.cuh"
#include "qe_quant.cuh"

namespace qe {
namespace {

constexpr int kMxStageK = 256;  // channels per pipeline stage: 128 bytes of codes, one swizzle row
constexpr int kSplitThreads = 192;

struct MxArgs {
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  int T, N, K, KT;  // KT = ceil(K / 128) scale tiles along K
  void* Y;
  int y_bf16;
  int* err;
};

template <int BN>
struct SplitCfg {
  static constexpr int kNB = (BN + 127) / 128;  // scale tiles across the token tile
  static constexpr int kA = 16384, kB = BN * 128, kSA = 1024, kSB = 1024 * kNB;
  static constexpr int kStage = kA + kB + kSA + kSB;
  static constexpr int kStages = BN <= 16 ? 5 : BN <= 64 ? 4 : BN <= 128 ? 3 : 4;
  static constexpr int kSfCols = 8 + 8 * kNB;   // tensor memory columns of a stage's scales
  static constexpr int kTmemUsed = BN + 2 * kSfCols;
  static constexpr int kTmemCols = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 256;
  static_assert(kStage % 1024 == 0, "stages keep the swizzle's alignment");
  static_assert(BN * 128 * 4 <= kStages * kStage, "the partial tile reuses the stages");
};

// Y tile of 128 output channels (MMA rows) x BN tokens (MMA columns), the K range split over the cluster's
// CTAs, whose fp32 partial tiles are then added in rank order through distributed shared memory.
// Weights stream once through each CTA's ring of TMA stages, so few tokens are bound by HBM; clusters make
// enough CTAs to keep all SMs streaming when there are few tiles.
template <int BN>
__global__ void __launch_bounds__(kSplitThreads) k_mx4_split(const __grid_constant__ CUtensorMap tm_w,
                                                             const __grid_constant__ CUtensorMap tm_x, const MxArgs a,
                                                             int splits) {
  using C = SplitCfg<BN>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * C::kStage);
  uint64_t* empty = full + NS;
  uint64_t* accf = empty + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n_tile = blockIdx.x / splits, n0 = n_tile * 128, t0 = blockIdx.y * BN;
  const int KS = (a.K + kMxStageK - 1) / kMxStageK;
  const int s0 = static_cast<int>(static_cast<int64_t>(KS) * rank / splits);
  const int nk = static_cast<int>(static_cast<int64_t>(KS) * (rank + 1) / splits) - s0;
  const int ncols = min(BN, a.T - t0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(accf, 1);
    mbar_fence_init();
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool acc_ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      for (; it < nk; ++it) {
        const int s = it % NS, ks = s0 + it;
        if (!mbar_wait(&empty[s], ((it / NS) & 1) ^ 1, a.err, DEVERR_WAIT_PRODUCER)) break;
        uint8_t* st = smem + s * C::kStage;
        const uint32_t sf = kMxTileBytes * min(2, a.KT - 2 * ks);
        const size_t rb = t0 / 128;
        const bool two = C::kNB == 2 && t0 + 128 < a.T;
        mbar_arrive_expect_tx(&full[s], C::kA + C::kB + sf * (two ? 3 : 2));
        tma_load_2d(st, &tm_w, ks * 128, n0, &full[s]);
        tma_load_2d(st + C::kA, &tm_x, ks * 128, t0, &full[s]);
        bulk_load(st + C::kA + C::kB, a.w_scales + (static_cast<size_t>(n_tile) * a.KT + 2 * ks) * kMxTileBytes, sf,
                  &full[s]);
        bulk_load(st + C::kA + C::kB + C::kSA, a.x_scales + (rb * a.KT + 2 * ks) * kMxTileBytes, sf, &full[s]);
        if (two)
          bulk_load(st + C::kA + C::kB + C::kSA + 1024, a.x_scales + ((rb + 1) * a.KT + 2 * ks) * kMxTileBytes, sf,
                    &full[s]);
      }
      drain_ring(full, NS, it);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t id = idesc_mxf4(128, BN);
    const bool leader = elect_one();
    for (int it = 0; it < nk; ++it) {
      const int s = it % NS, ks = s0 + it;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / NS) & 1, a.err, DEVERR_WAIT_MMA))) break;
      tc_fence_after();
      if (leader) {
        const uint32_t at = smem_u32(smem + s * C::kStage);
        const uint32_t sfa = tmem + BN + (it & 1) * C::kSfCols, sfb = sfa + 8;
        const int tiles = min(2, a.KT - 2 * ks);
        const uint32_t sa = at + C::kA + C::kB, sb = sa + C::kSA;
        for (int k = 0; k < tiles; ++k) {
          tmem_cp_32x128b(sfa + 4 * k, smem_desc_rows16(sa + k * kMxTileBytes));
#pragma unroll
          for (int b = 0; b < C::kNB; ++b)
            tmem_cp_32x128b(sfb + (k * C::kNB + b) * 4, smem_desc_rows16(sb + b * 1024 + k * kMxTileBytes));
        }
        const uint64_t da = smem_desc_sw128(at), db = smem_desc_sw128(at + C::kA);
        const int mmas = min(4, (a.K - ks * kMxStageK + 63) / 64);
        for (int m = 0; m < mmas; ++m) {
          const uint32_t sel = static_cast<uint32_t>(m & 1) * 2;
          mma_mxf4(tmem, da + 2 * m, db + 2 * m, id | (sel << 29) | (sel << 4), sfa + 4 * (m >> 1),
                   sfb + 4 * C::kNB * (m >> 1), (it | m) != 0);
        }
        tc_commit(&empty[s]);
        if (it == nk - 1) tc_commit(accf);
      }
      __syncwarp();
    }
  } else {
    acc_ok = mbar_wait(accf, 0, a.err, DEVERR_WAIT_EPILOGUE);
    acc_ok = __all_sync(0xffffffffu, acc_ok);
    tc_fence_after();
    const int q = warp & 3;
    const int o = 32 * q + lane;
    float* part = reinterpret_cast<float*>(smem);
    if (acc_ok) {
      for (int c0 = 0; c0 < ncols; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(32 * q) << 16) + c0, v);
        tmem_wait_ld();
        reg_fence(v);
        if (splits > 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + o] = __uint_as_float(v[j]);
        } else if (n0 + o < a.N) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (c0 + j < ncols) {
              const size_t y = static_cast<size_t>(t0 + c0 + j) * a.N + n0 + o;
              if (a.y_bf16) static_cast<uint16_t*>(a.Y)[y] = f32_to_bf16_bits(__uint_as_float(v[j]));
              else static_cast<float*>(a.Y)[y] = __uint_as_float(v[j]);
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  if (splits > 1) {
    cluster_sync_all();
    const uint32_t part = smem_u32(smem);
    const int total = ncols * 128;
    const int i1 = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / splits);
    for (int i = static_cast<int>(static_cast<int64_t>(total) * rank / splits) + threadIdx.x; i < i1; i += kSplitThreads) {
      float v = 0.0f;
      for (int r = 0; r < splits; ++r) v += ld_cluster_f32(mapa(part + i * 4, r));
      const int n = n0 + (i & 127);
      if (n < a.N) {
        const size_t y = static_cast<size_t>(t0 + (i >> 7)) * a.N + n;
        if (a.y_bf16) static_cast<uint16_t*>(a.Y)[y] = f32_to_bf16_bits(v);
        else static_cast<float*>(a.Y)[y] = v;
      }
    }
    cluster_sync_all();  // no CTA leaves while another may still read its partial tile
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// ------------------------------------------------------------------ many tokens
// Y tile of 256 tokens x 256 output channels per pair of CTAs (cta_group::2: each CTA holds 128 token rows, half of
// the weight rows and a 128 x 256 accumulator), persistent over the tiles. A tile reads 512 rows for 256 x 256
// outputs, half of what the two CTAs would read as 128 x 256 tiles of their own: at the 4-bit rate the
// shared memory fill is what limits smaller tiles.
struct PairCfg {
  static constexpr int kEpiWarps = 8;  // two for each 32 token rows, alternate chunks of 32 columns
  static constexpr int kA = 16384, kB = 16384, kSA = 1024, kSB = 2048;
  static constexpr int kStage = kA + kB + kSA + kSB;
  static constexpr int kStages = 5;
  // Tensor memory: two accumulators of 256 columns that share the columns [192, 256), and two sets of scales.
  // The epilogue drains the shared columns first, so the next tile's MMAs start after a quarter of it.
  static constexpr int kAcc1 = 192, kSf = 448, kSfCols = 24;
  // An epilogue warp's staging buffer: a 32 x 32 block of Y, swizzled for its TMA store (two of them in bf16), or
  // padded rows of fp32 where Y's rows allow no TMA store.
  static constexpr int kPad = 33;
  static constexpr int kOut = 5120;
  static constexpr int kTrans = kEpiWarps * kOut;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + kTrans + 256;
  static_assert(kStage % 1024 == 0 && kSf + 2 * kSfCols <= 512 && 32 * kPad * 4 <= kOut, "layout");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};
constexpr int kPairThreads = 64 + 32 * PairCfg::kEpiWarps;

struct PairArgs {
  int T, N, K, KT;
  int m_tiles, n_tiles, group;  // group: token tiles walked together, so that their activations stay in L2
  void* Y;
  int y_bf16, tma;              // tma: Y's rows are multiples of 16 bytes
  int* err;
};

__device__ __forceinline__ void pair_tile(const PairArgs& a, int tile, int& mt, int& nt) {
  const int per = a.group * a.n_tiles, g = tile / per, r = tile - g * per;
  const int rows = min(a.group, a.m_tiles - g * a.group);
  mt = g * a.group + r % rows;
  nt = r / rows;
}

// Stores a warp's 32 rows x 32 columns of Y from its registers (v: this lane's row). `turn` counts the warp's
// TMA stores: a staging half is written again once the store before last (bf16) or the last (fp32) has
// read it.
__device__ __forceinline__ void pair_store(const PairArgs& a, const CUtensorMap* tm_y, const uint32_t (&v)[32], int row0,
                                           int col, int lane, uint8_t* out, int& turn) {
  if (a.tma) {
    if (col >= a.N || row0 >= a.T) return;
    if (a.y_bf16) {
      // rows of 64 bytes, 16-byte pieces permuted by bits 7-8 of their offset (64-byte swizzle)
      uint8_t* half = out + (turn & 1) * 2048;
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h =
              __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(half + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tm_y, half, col, row0);
        bulk_commit();
      }
    } else {
      // rows of 128 bytes, pieces permuted by bits 7-9 (128-byte swizzle)
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(out + lane * 128 + (i ^ (lane & 7)) * 16) =
            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tm_y, out, col, row0);
        bulk_commit();
      }
    }
    ++turn;
  } else if (col < a.N) {
    // through shared memory, a row per store
    float* tw = reinterpret_cast<float*>(out);
#pragma unroll
    for (int i = 0; i < 32; ++i) tw[lane * PairCfg::kPad + i] = __uint_as_float(v[i]);
    __syncwarp();
    const int rows = min(32, a.T - row0);
    for (int r = 0; r < rows; ++r) {
      const float f = tw[r * PairCfg::kPad + lane];
      if (col + lane < a.N) {
        const size_t y = static_cast<size_t>(row0 + r) * a.N + col + lane;
        if (a.y_bf16) static_cast<uint16_t*>(a.Y)[y] = f32_to_bf16_bits(f);
        else static_cast<float*>(a.Y)[y] = f;
      }
    }
    __syncwarp();
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
    k_mx4_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
               const __grid_constant__ CUtensorMap tm_y, const PairArgs a) {
  using C = PairCfg;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + NS * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * C::kStage + C::kTrans);
  uint64_t* empty = full + NS;
  uint64_t* accf = empty + NS;   // [2] a tile's MMAs are done
  uint64_t* freed = accf + 2;    // the shared columns of a tile are drained (even CTA's, from both CTAs)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(freed + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int KS = (a.K + kMxStageK - 1) / kMxStageK;
  const int tiles = a.m_tiles * a.n_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&accf[0], 1);
    mbar_init(&accf[1], 1);
    mbar_init(freed, 2 * C::kEpiWarps);
    mbar_fence_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_xs);
    prefetch_tmap(&tm_ws);
    prefetch_tmap(&tm_y);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are ready before either's loads or arrivals reach them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int mt, nt;
        pair_tile(a, tile, mt, nt);
        const int m0 = mt * 256 + cta * 128, n0 = nt * 256 + cta * 128;
        for (int ks = 0; ks < KS; ++ks, ++it) {
          const int s = it % NS;
          if (!mbar_wait(&empty[s], ((it / NS) & 1) ^ 1, a.err, DEVERR_WAIT_PRODUCER)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::kStage;
          // the even CTA's barrier counts both CTAs' bytes
          if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
          const uint32_t bar = mapa(smem_u32(&full[s]), 0);
          tma_load_2d_pair(st, &tm_x, ks * 128, m0, bar);
          tma_load_2d_pair(st + C::kA, &tm_w, ks * 128, n0, bar);
          tma_load_2d_pair(st + C::kA + C::kB, &tm_xs, ks * 256, mt * 2 + cta, bar);
          tma_load_2d_pair(st + C::kA + C::kB + C::kSA, &tm_ws, ks * 256, nt * 2, bar);
        }
      }
      if (cta == 0) drain_ring(full, NS, it);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (cta == 0) {
      constexpr uint32_t id = idesc_mxf4(256, 256);
      const bool leader = elect_one();
      int it = 0, n = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs, ++n) {
        if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(freed, (n - 1) & 1, a.err, DEVERR_WAIT_MMA))) break;
        tc_fence_after();
        const uint32_t acc = tmem + ((n & 1) ? C::kAcc1 : 0);
        for (int ks = 0; ks < KS; ++ks, ++it) {
          const int s = it % NS;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / NS) & 1, a.err, DEVERR_WAIT_MMA))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            const uint32_t at = smem_u32(smem + s * C::kStage);
            const uint32_t sfa = tmem + C::kSf + (it & 1) * C::kSfCols, sfb = sfa + 8;
            const uint32_t sa = at + C::kA + C::kB, sb = sa + C::kSA;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              tmem_cp_32x128b_pair(sfa + 4 * k, smem_desc_rows16(sa + k * kMxTileBytes));
#pragma unroll
              for (int b = 0; b < 2; ++b)
                tmem_cp_32x128b_pair(sfb + (2 * k + b) * 4, smem_desc_rows16(sb + b * 1024 + k * kMxTileBytes));
            }
            const uint64_t da = smem_desc_sw128(at), db = smem_desc_sw128(at + C::kA);
            const int mmas = min(4, (a.K - ks * kMxStageK + 63) / 64);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t sel = static_cast<uint32_t>(m & 1) * 2;
              if (m < mmas)
                mma_mxf4_pair(acc, da + 2 * m, db + 2 * m, id | (sel << 29) | (sel << 4), sfa + 4 * (m >> 1),
                              sfb + 8 * (m >> 1), (ks | m) != 0);
            }
            tc_commit_pair(&empty[s]);
            if (ks == KS - 1) tc_commit_pair(&accf[n & 1]);
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* out = staging + (warp - 2) * C::kOut;
    int turn = 0;
    const uint32_t freed0 = mapa(smem_u32(freed), 0);
    int n = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++n) {
      int mt, nt;
      pair_tile(a, tile, mt, nt);
      if (!__all_sync(0xffffffffu, mbar_wait(&accf[n & 1], (n >> 1) & 1, a.err, DEVERR_WAIT_EPILOGUE))) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((n & 1) ? C::kAcc1 : 0) + (static_cast<uint32_t>(32 * q) << 16);
      const int row0 = mt * 256 + cta * 128 + 32 * q, n0 = nt * 256;
      // chunks of 32 columns, the shared ones first: 6, 7, 0 .. 5 of the first accumulator, 0 .. 7 of the second
      const int first = ((n & 1) ? 0 : 6) + half;
#pragma unroll 1
      for (int j = 0; j < 8; j += 2) {
        const int c = ((first + j) & 7) * 32;
        uint32_t v[32];
        tmem_ld32(acc + c, v);
        tmem_wait_ld();
        reg_fence(v);
        if (j == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(freed0);
        }
        pair_store(a, &tm_y, v, row0, n0 + c, lane, out, turn);
      }
    }
    if (lane == 0) bulk_wait_all();
    tc_fence_before();
  }
  __syncthreads();
  cluster_sync_all();  // neither CTA frees memory that the other's instructions may still use
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int BN>
cudaError_t launch_split_t(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const MxArgs& a, const Mx4Plan& p,
                           cudaStream_t st) {
  using C = SplitCfg<BN>;
  cudaError_t e = cudaFuncSetAttribute(k_mx4_split<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_tiles * p.splits), static_cast<unsigned>(p.t_tiles));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_mx4_split<BN>, tm_w, tm_x, a, p.splits);
}

}  // namespace

Mx4Plan plan_mx4(int T, int N, int K) {
  Mx4Plan p{};
  int sms = decode_grid_sms();
  if (sms == 0) sms = 148;
  p.pair = T > 256;
  if (p.pair) {
    p.bn = 256;
    p.n_tiles = static_cast<int>(ceil_div(N, 256));
    p.t_tiles = static_cast<int>(ceil_div(T, 256));
    p.splits = 1;
    p.ctas = static_cast<int>(2 * std::min<int64_t>(sms / 2, static_cast<int64_t>(p.n_tiles) * p.t_tiles));
    return p;
  }
  p.bn = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  p.n_tiles = static_cast<int>(ceil_div(N, 128));
  p.t_tiles = static_cast<int>(ceil_div(T, p.bn));
  // as many CTAs as two per SM (one at 256 tokens) hold, in clusters of at most eight along K
  const int slots = p.bn == 256 ? sms : 2 * sms;
  const int64_t tiles = static_cast<int64_t>(p.n_tiles) * p.t_tiles;
  const int stages = static_cast<int>(ceil_div(K, kMxStageK));
  p.splits = 1;
  while (p.splits < 8 && tiles * p.splits * 2 <= slots && p.splits * 2 <= stages) p.splits *= 2;
  p.ctas = static_cast<int>(tiles * p.splits);
  return p;
}

cudaError_t launch_mx4_pair(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const CUtensorMap& tm_ws,
                            const CUtensorMap& tm_xs, const CUtensorMap* tm_y, const Mx4Plan& p, int T, int N, int K,
                            void* Y, bool y_bf16, int* err, cudaStream_t st) {
  using C = PairCfg;
  cudaError_t e = cudaFuncSetAttribute(k_mx4_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  PairArgs a{};
  a.T = T;
  a.N = N;
  a.K = K;
  a.KT = static_cast<int>(ceil_div(K, kMxTileCols));
  a.m_tiles = p.t_tiles;
  a.n_tiles = p.n_tiles;
  a.group = std::min(p.t_tiles, 8);
  a.Y = Y;
  a.y_bf16 = y_bf16;
  a.tma = tm_y != nullptr;
  a.err = err;
  k_mx4_pair<<<p.ctas, kPairThreads, C::kSmem, st>>>(tm_x, tm_w, tm_xs, tm_ws, tm_y ? *tm_y : tm_x, a);
  return cudaGetLastError();
}

cudaError_t launch_mx4_product(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const Mx4Plan& p, const uint8_t* w_scales,
                               const uint8_t* x_scales, int T, int N, int K, void* Y, bool y_bf16, int* err,
                               cudaStream_t st) {
  MxArgs a{};
  a.w_scales = w_scales;
  a.x_scales = x_scales;
  a.T = T;
  a.N = N;
  a.K = K;
  a.KT = static_cast<int>(ceil_div(K, kMxTileCols));
  a.Y = Y;
  a.y_bf16 = y_bf16;
  a.err = err;
  switch (p.bn) {
    case 16: return launch_split_t<16>(tm_w, tm_x, a, p, st);
    case 32: return launch_split_t<32>(tm_w, tm_x, a, p, st);
    case 64: return launch_split_t<64>(tm_w, tm_x, a, p, st);
    case 128: return launch_split_t<128>(tm_w, tm_x, a, p, st);
    default: return launch_split_t<256>(tm_w, tm_x, a, p, st);
  }
}

}  // namespace qe
