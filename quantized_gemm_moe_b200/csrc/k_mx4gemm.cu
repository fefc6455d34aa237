// Product of MXFP4 activations and MXFP4 weights on the block-scaled 4-bit tensor cores:
//   Y[t][o] = sum_k x[t][k] w[o][k],  x = 2^Ex[t][k/32] * E2M1,  w = 2^Ew[o][k/32] * E2M1
// tcgen05.mma kind::mxf4 multiplies 64 channels of both operands with their scales and adds in fp32, so nothing is
// unpacked: codes go from HBM to shared memory by TMA, their scale bytes on to tensor memory by tcgen05.cp.
// Two kernels: few tokens stream the weights (HBM bound), many fill the tensor cores.
#include <algorithm>
#include <atomic>

#include "qe_internal.h"
#include "qe_launch.cuh"
#include "qe_ptx.cuh"
#include "qe_quant.cuh"

namespace qe {
namespace {

constexpr int kMxStageK = 256;  // channels per pipeline stage: 128 bytes of codes, one swizzle row

// Y[t][n .. n+4) = v, as far as the row of N channels reaches.
__device__ __forceinline__ void store4(void* Y, int y_bf16, int N, int t, int n, const float4& v) {
  const size_t y = static_cast<size_t>(t) * N + n;
  if ((N & 3) == 0) {
    if (n < N) {
      if (y_bf16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Y) + y) = make_uint2(bf16x2_word(v.x, v.y), bf16x2_word(v.z, v.w));
      else *reinterpret_cast<float4*>(static_cast<float*>(Y) + y) = v;
    }
  } else {
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j < N) {
        if (y_bf16) static_cast<uint16_t*>(Y)[y + j] = f32_to_bf16_bits(f[j]);
        else static_cast<float*>(Y)[y + j] = f[j];
      }
    }
  }
}

// ------------------------------------------------------------------ few tokens
struct SplitArgs {
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  int T, N, K, KT;      // KT = ceil(K / 128) scale tiles along K
  int bn, splits;       // MMA columns: T rounded up to 16, at most 128; CTAs along K
  int stages, tmem_cols;
  int w_early;          // the weights were written before the previous kernel began
  void* Y;
  int y_bf16;
  int* err;
};
constexpr int kSplitThreads = 192;
constexpr int kSplitA = 16384, kSplitSA = 1024;

constexpr int kSplitSfCols = 16;  // tensor memory columns of a stage's scales
__host__ __device__ constexpr int split_stage_bytes(int bn) { return kSplitA + bn * 128 + 2 * kSplitSA; }
// Two CTAs share an SM's 228 KB.
constexpr int split_stages(int bn) { return 114176 / split_stage_bytes(bn); }

// v = the sum in rank order of four floats at `at` in each of S CTAs' partial tiles, for U addresses at once (eight
// 16-byte loads of distributed shared memory in flight: one at a time, their latency was half of a short call).
template <int S, int U>
__device__ __forceinline__ void sum_parts(const uint32_t (&from)[S], const uint32_t (&at)[U], float4 (&v)[U]) {
  float4 p[U][S];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int r = 0; r < S; ++r) p[u][r] = ld_cluster_f32x4(from[r] + at[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    v[u] = p[u][0];
#pragma unroll
    for (int r = 1; r < S; ++r) {
      v[u].x += p[u][r].x;
      v[u].y += p[u][r].y;
      v[u].z += p[u][r].z;
      v[u].w += p[u][r].w;
    }
  }
}

// Adds the cluster's partial tiles, four channels of a token at a time, and writes this CTA's share of them.
template <int S>
__device__ __forceinline__ void split_reduce(const SplitArgs& a, uint32_t part, int rank, int n0) {
  constexpr int U = 8 / S;
  uint32_t from[S];
#pragma unroll
  for (int r = 0; r < S; ++r) from[r] = S > 1 ? mapa(part, r) : part;
  const int total = a.T * 32;
  const int i0 = static_cast<int>(static_cast<int64_t>(total) * rank / S), i1 = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / S);
  for (int i = i0 + threadIdx.x; i < i1; i += kSplitThreads * U) {
    uint32_t at[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = 16 * min(i + u * kSplitThreads, i1 - 1);
    sum_parts<S, U>(from, at, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = i + u * kSplitThreads;
      if (j < i1) store4(a.Y, a.y_bf16, a.N, j >> 5, n0 + (j & 31) * 4, v[u]);
    }
  }
}

// At most 128 tokens. Y tile of 128 output channels (MMA rows) x all tokens (MMA columns), the K range split over
// the cluster's CTAs, whose fp32 partial tiles are then added in rank order through distributed shared memory.
// Weights stream once through each CTA's ring of TMA stages, so few tokens are bound by HBM; clusters make
// enough CTAs to keep all SMs streaming when there are few tiles. 16 x 29568 -> 8192: 24.9 us, 5.2 TB/s, of which
// about 4.5 us are set-up, the first loads and the sum.
__global__ void __launch_bounds__(kSplitThreads) k_mx4_split(const __grid_constant__ CUtensorMap tm_w,
                                                             const __grid_constant__ CUtensorMap tm_x,
                                                             const SplitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NS = a.stages, kB = a.bn * 128, stage = split_stage_bytes(a.bn);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NS * stage);
  uint64_t* empty = full + NS;
  uint64_t* accf = empty + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n_tile = blockIdx.x / a.splits, n0 = n_tile * 128;
  const int KS = (a.K + kMxStageK - 1) / kMxStageK;
  const int s0 = static_cast<int>(static_cast<int64_t>(KS) * rank / a.splits);
  const int nk = static_cast<int>(static_cast<int64_t>(KS) * (rank + 1) / a.splits) - s0;

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
    tmem_alloc(tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      auto load_w = [&](int it) {
        const int s = it % NS, ks = s0 + it;
        uint8_t* st = smem + s * stage;
        const uint32_t sf = kMxTileBytes * min(2, a.KT - 2 * ks);
        mbar_arrive_expect_tx(&full[s], kSplitA + kB + 2 * sf);
        tma_load_2d(st, &tm_w, ks * 128, n0, &full[s]);
        bulk_load(st + kSplitA + kB, a.w_scales + (static_cast<size_t>(n_tile) * a.KT + 2 * ks) * kMxTileBytes, sf, &full[s]);
      };
      auto load_x = [&](int it) {
        const int s = it % NS, ks = s0 + it;
        uint8_t* st = smem + s * stage;
        const uint32_t sf = kMxTileBytes * min(2, a.KT - 2 * ks);
        tma_load_2d(st + kSplitA, &tm_x, ks * 128, 0, &full[s]);
        bulk_load(st + kSplitA + kB + kSplitSA, a.x_scales + static_cast<size_t>(2 * ks) * kMxTileBytes, sf, &full[s]);
      };
      const int ahead = min(nk, NS);
      if (!a.w_early) grid_dep_wait();
      for (int it = 0; it < ahead; ++it) load_w(it);
      if (a.w_early) grid_dep_wait();
      for (int it = 0; it < ahead; ++it) load_x(it);
      int it = ahead;
      for (; it < nk; ++it) {
        if (!mbar_wait(&empty[it % NS], ((it / NS) & 1) ^ 1, a.err, DEVERR_WAIT_PRODUCER)) break;
        load_w(it);
        load_x(it);
      }
      drain_ring(full, NS, it);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t id = idesc_mxf4(128, a.bn);
    const bool leader = elect_one();
    for (int it = 0; it < nk; ++it) {
      const int s = it % NS, ks = s0 + it;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / NS) & 1, a.err, DEVERR_WAIT_MMA))) break;
      tc_fence_after();
      if (leader) {
        const uint32_t at = smem_u32(smem + s * stage);
        const uint32_t sfa = tmem + a.bn + (it & 1) * kSplitSfCols, sfb = sfa + 8;
        const int tiles = min(2, a.KT - 2 * ks);
        const uint32_t sa = at + kSplitA + kB, sb = sa + kSplitSA;
        for (int k = 0; k < tiles; ++k) {
          tmem_cp_32x128b(sfa + 4 * k, smem_desc_rows16(sa + k * kMxTileBytes));
          tmem_cp_32x128b(sfb + 4 * k, smem_desc_rows16(sb + k * kMxTileBytes));
        }
        const uint64_t da = smem_desc_sw128(at), db = smem_desc_sw128(at + kSplitA);
        const int mmas = min(4, (a.K - ks * kMxStageK + 63) / 64);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t sel = static_cast<uint32_t>(m & 1) * 2;
          if (m < mmas)
            mma_mxf4(tmem, da + 2 * m, db + 2 * m, id | (sel << 29) | (sel << 4), sfa + 4 * (m >> 1),
                     sfb + 4 * (m >> 1), (it | m) != 0);
        }
        tc_commit(&empty[s]);
        if (it == nk - 1) tc_commit(accf);
      }
      __syncwarp();
    }
  } else {
    // the partial tile [token][channel], over the stages: all of them have been read
    const int o = 32 * (warp & 3) + lane;
    float* part = reinterpret_cast<float*>(smem);
    if (__all_sync(0xffffffffu, mbar_wait(accf, 0, a.err, DEVERR_WAIT_EPILOGUE))) {
      tc_fence_after();
      for (int c0 = 0; c0 < a.T; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c0, v);
        tmem_wait_ld();
        reg_fence(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + o] = __uint_as_float(v[j]);
      }
    }
    tc_fence_before();
  }
  if (a.splits > 1) cluster_sync_all();
  else __syncthreads();
  const uint32_t part = smem_u32(smem);
  switch (a.splits) {
    case 1: split_reduce<1>(a, part, rank, n0); break;
    case 2: split_reduce<2>(a, part, rank, n0); break;
    case 4: split_reduce<4>(a, part, rank, n0); break;
    default: split_reduce<8>(a, part, rank, n0); break;
  }
  if (a.splits > 1) cluster_sync_all();  // no CTA leaves while another may still read its partial tile
  else __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, a.tmem_cols);
}

// ------------------------------------------------------------------ many tokens
// Y tile of 256 tokens x 256 output channels per pair of CTAs (cta_group::2: each CTA holds 128 token rows, half of
// the weight rows and a 128 x 256 accumulator), persistent over the tiles. 8192 x 8192 -> 29568: 637 us (624 to
// 652 from one GPU to another), 6.2 PFLOP/s or 0.93 of four times the measured bf16 rate (733 to 773 us back to back, under
// the power cap; 1407 us with 128 x 256 tiles of single CTAs). A stage of 256 channels takes 0.29 us while one pair works
// and 0.37 us on average in that product, where a pair runs 1632 (296 tiles on 74 pairs: 0.33 us between K = 1536 and
// 4608, 0.39 to 0.41 beyond). Reading the activations from L2 once for a whole row of tiles left the time as it was, so
// L2 is not what makes the difference. About 6 us of a call are set-up, the first loads and the last tile's stores.
struct PairCfg {
  static constexpr int kEpiWarps = 8;  // two for each 32 token rows, alternate chunks of 32 columns
  static constexpr int kA = 16384, kB = 16384, kSA = 1024, kSB = 2048;
  static constexpr int kStage = kA + kB + kSA + kSB;
  // Six stages: 8192 x 1536 -> 8960 52.8 us with five and 49.3 with six, 8192 x 8192 -> 29568 640 and 624.
  static constexpr int kStages = 6;
  // Tensor memory: two accumulators of 256 columns that share the columns [192, 256), and two sets of scales.
  // The epilogue drains the shared columns first, so the next tile's MMAs start after a quarter of it.
  static constexpr int kAcc1 = 192, kSf = 448, kSfCols = 24;
  // An epilogue warp's staging buffer: 32 rows of 64 bytes of Y.
  static constexpr int kOut = 2048;
  static constexpr int kStaging = kStages * kStage, kBars = kStaging + kEpiWarps * kOut;
  // No room to round the base up: dynamic shared memory begins on a multiple of 1024 bytes (the kernel checks).
  static constexpr size_t kSmem = kBars + 256;
  static_assert(kStage % 1024 == 0 && kSf + 2 * kSfCols <= 512, "layout");
  static_assert(kSmem <= 227 * 1024 && kEpiWarps * 16384 <= kStages * kStage, "shared memory");
};
constexpr int kPairThreads = 64 + 32 * PairCfg::kEpiWarps;

struct PairArgs {
  int T, N, K;
  int m_tiles, n_tiles, group;  // group: token tiles walked together, so that their activations stay in L2
  void* Y;
  int y_bf16, tma;              // tma: Y's rows are multiples of 16 bytes
  int w_early;                  // the weights were written before the previous kernel began
  int* err;
};

__device__ __forceinline__ void pair_tile(const PairArgs& a, int tile, int& mt, int& nt) {
  const int per = a.group * a.n_tiles, g = tile / per, r = tile - g * per;
  const int rows = min(a.group, a.m_tiles - g * a.group);
  mt = g * a.group + r % rows;
  nt = r / rows;
}

// Stores 32 rows of 64 bytes of Y by TMA: v is this lane's row (two bf16 or one fp32 to a word). 16-byte pieces are
// permuted by bits 7-8 of their offset (64-byte swizzle).
__device__ __forceinline__ void pair_store_tma(const CUtensorMap* tm_y, const uint32_t (&v)[16], int row0, int col, int lane,
                                               uint8_t* out, bool fresh) {
  if (!fresh) {
    if (lane == 0) bulk_wait_read<0>();  // the store before has read the buffer
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(out + lane * 64 + (i ^ ((lane >> 1) & 3)) * 16) =
        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm_y, out, col, row0);
    bulk_commit();
  }
}
// Where rows of N elements allow no TMA store: through the same buffer, a row to a store instruction (several rows of
// less are slower), or four rows of bf16 where they keep 8-byte words aligned. Words are permuted within their row so
// that neither the lanes' rows nor a row's words meet on a bank. (2048 x 1536 -> 8960: 16.4 us, 8964 19.0, 8961 24.0.)
__device__ __forceinline__ void pair_store_bf16(const PairArgs& a, const uint32_t (&v)[16], int row0, int col, int lane,
                                                uint32_t* tw) {
  const int rows = min(32, a.T - row0), left = a.N - col;  // elements up to the row's end
  uint16_t* y = static_cast<uint16_t*>(a.Y) + static_cast<size_t>(row0) * a.N + col;
#pragma unroll
  for (int w = 0; w < 16; ++w) tw[lane * 16 + (w ^ (lane >> 1))] = v[w];
  __syncwarp();
  if ((a.N & 3) == 0) {
    const int w = 2 * (lane & 7);
    if (2 * w < left) {
#pragma unroll 4
      for (int r = lane >> 3; r < rows; r += 4)
        *reinterpret_cast<uint2*>(y + static_cast<size_t>(r) * a.N + 2 * w) =
            make_uint2(tw[r * 16 + (w ^ (r >> 1))], tw[r * 16 + ((w + 1) ^ (r >> 1))]);
    }
  } else if (lane < left) {
#pragma unroll 4
    for (int r = 0; r < rows; ++r)
      y[static_cast<size_t>(r) * a.N + lane] = static_cast<uint16_t>(tw[r * 16 + ((lane >> 1) ^ (r >> 1))] >> (16 * (lane & 1)));
  }
  __syncwarp();
}
__device__ __forceinline__ void pair_store_f32(const PairArgs& a, const uint32_t (&v)[32], int row0, int col, int lane,
                                               uint32_t* tw) {
#pragma unroll 1
  for (int h = 0; h < 2; ++h, row0 += 16) {  // 16 rows fill the buffer
    if (lane >> 4 == h) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(tw + (lane & 15) * 32 + (i ^ (lane & 7)) * 4) =
            make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
    __syncwarp();
    const int rows = min(16, a.T - row0);
    uint32_t* y = static_cast<uint32_t*>(a.Y) + static_cast<size_t>(row0) * a.N + col;
    if (lane < a.N - col) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r) y[static_cast<size_t>(r) * a.N + lane] = tw[r * 32 + (lane ^ ((r & 7) * 4))];
    }
    __syncwarp();
  }
}
// 32 rows x 32 columns of Y from a warp's accumulator registers. fresh: `out` is 4 KB that no store reads.
__device__ __forceinline__ void pair_store(const PairArgs& a, const CUtensorMap* tm_y, const uint32_t (&v)[32], int row0,
                                           int col, int lane, uint8_t* out, bool fresh) {
  if (col >= a.N || row0 >= a.T) return;
  uint32_t w[16];
  if (a.y_bf16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2_word(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    if (a.tma) pair_store_tma(tm_y, w, row0, col, lane, out, fresh);
    else pair_store_bf16(a, w, row0, col, lane, reinterpret_cast<uint32_t*>(out));
  } else if (a.tma) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = v[16 * h + i];
      if (col + 16 * h < a.N) pair_store_tma(tm_y, w, row0, col + 16 * h, lane, fresh ? out + 2048 * h : out, fresh);
    }
  } else {
    pair_store_f32(a, v, row0, col, lane, reinterpret_cast<uint32_t*>(out));
  }
}

// Adds the K slices' partial tiles (fp32 rows of 256 columns, 16-byte pieces permuted by the row) and stores this
// slice's share of the CTA's 128 rows.
template <int S>
__device__ __forceinline__ void pair_reduce(const PairArgs& a, uint32_t part, int cta, int slice, int m0, int n0) {
  constexpr int U = 8 / S, total = 128 / S * 64;
  uint32_t from[S];
#pragma unroll
  for (int r = 0; r < S; ++r) from[r] = mapa(part, cta + 2 * r);
  for (int i = threadIdx.x; i < total; i += kPairThreads * U) {
    uint32_t at[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(i + u * kPairThreads, total - 1), row = 128 / S * slice + (j >> 6);
      at[u] = static_cast<uint32_t>(row * 1024 + (((j & 63) ^ (row & 7)) * 16));
    }
    sum_parts<S, U>(from, at, v);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = i + u * kPairThreads, row = m0 + 128 / S * slice + (j >> 6);
      if (j < total && row < a.T) store4(a.Y, a.y_bf16, a.N, row, n0 + 4 * (j & 63), v[u]);
    }
  }
}

// S > 1: a cluster of S pairs takes one tile, a slice of K each, and adds the slices' partial tiles through
// distributed shared memory: few tiles with a long K then use more SMs.
template <int S>
__global__ void __launch_bounds__(kPairThreads)
    k_mx4_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_xs, const __grid_constant__ CUtensorMap tm_ws,
               const __grid_constant__ CUtensorMap tm_y, const PairArgs a) {
  using C = PairCfg;
  constexpr int NS = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_1k[];
  uint8_t* smem = smem_1k;
  if ((smem_u32(smem) & 1023u) != 0) {  // the same in every CTA: all of them leave
    record_error(a.err, DEVERR_SMEM_BASE);
    return;
  }
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* empty = full + NS;
  uint64_t* accf = empty + NS;   // [2] a tile's MMAs are done
  uint64_t* freed = accf + 2;    // the shared columns of a tile are drained (even CTA's, from both CTAs)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(freed + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const int cta = crank & 1, lead = crank & ~1, slice = crank >> 1;
  const int pair = blockIdx.x / (2 * S), pairs = gridDim.x / (2 * S);
  const int KS_all = (a.K + kMxStageK - 1) / kMxStageK;
  const int ks0 = static_cast<int>(static_cast<int64_t>(KS_all) * slice / S);
  const int KS = static_cast<int>(static_cast<int64_t>(KS_all) * (slice + 1) / S) - ks0;
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
      // stage it of tile (mt, nt); the even CTA's barrier counts both CTAs' bytes
      auto load_w = [&](int it, int ks, int nt) {
        const int s = it % NS;
        uint8_t* st = smem + s * C::kStage;
        if (cta == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
        const uint32_t bar = mapa(smem_u32(&full[s]), lead);
        ks += ks0;
        tma_load_2d_pair(st + C::kA, &tm_w, ks * 128, nt * 256 + cta * 128, bar);
        tma_load_2d_pair(st + C::kA + C::kB + C::kSA, &tm_ws, ks * 256, nt * 2, bar);
      };
      auto load_x = [&](int it, int ks, int mt) {
        const int s = it % NS;
        uint8_t* st = smem + s * C::kStage;
        const uint32_t bar = mapa(smem_u32(&full[s]), lead);
        ks += ks0;
        tma_load_2d_pair(st, &tm_x, ks * 128, mt * 256 + cta * 128, bar);
        tma_load_2d_pair(st + C::kA + C::kB, &tm_xs, ks * 256, mt * 2 + cta, bar);
      };
      int it = 0, ahead = min(KS, NS);
      bool ok = true;
      if (!a.w_early) grid_dep_wait();
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int mt, nt;
        pair_tile(a, tile, mt, nt);
        int ks = 0;
        if (it == 0) {  // the first stages are free, and their weights need no wait
          for (ks = 0; ks < ahead; ++ks) load_w(ks, ks, nt);
          if (a.w_early) grid_dep_wait();
          for (ks = 0; ks < ahead; ++ks) load_x(ks, ks, mt);
          it = ahead;
        }
        for (; ks < KS; ++ks, ++it) {
          if (!mbar_wait(&empty[it % NS], ((it / NS) & 1) ^ 1, a.err, DEVERR_WAIT_PRODUCER)) {
            ok = false;
            break;
          }
          load_w(it, ks, nt);
          load_x(it, ks, mt);
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
            const int mmas = min(4, (a.K - (ks0 + ks) * kMxStageK + 63) / 64);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint32_t sel = static_cast<uint32_t>(m & 1) * 2;
              if (m < mmas)
                mma_mxf4_pair(acc, da + 2 * m, db + 2 * m, id | (sel << 29) | (sel << 4), sfa + 4 * (m >> 1),
                              sfb + 8 * (m >> 1), (ks | m) != 0);
            }
            tc_commit_pair(&empty[s], lead);
            if (ks == KS - 1) tc_commit_pair(&accf[n & 1], lead);
          }
          __syncwarp();
        }
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    if constexpr (S > 1) {
      // this slice's partial tile, over the stages: all of them have been read
      if (__all_sync(0xffffffffu, mbar_wait(&accf[0], 0, a.err, DEVERR_WAIT_EPILOGUE))) {
        tc_fence_after();
        uint8_t* row = smem + (32 * q + lane) * 1024;
#pragma unroll 1
        for (int c = half * 128; c < half * 128 + 128; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(32 * q) << 16) + c, v);
          tmem_wait_ld();
          reg_fence(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(row + ((c / 4 + i) ^ (lane & 7)) * 16) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    }
    uint8_t* out = smem + C::kStaging + (warp - 2) * C::kOut;
    const uint32_t freed0 = mapa(smem_u32(freed), lead);
    int n = 0;
    for (int tile = pair; S == 1 && tile < tiles; tile += pairs, ++n) {
      int mt, nt;
      pair_tile(a, tile, mt, nt);
      if (!__all_sync(0xffffffffu, mbar_wait(&accf[n & 1], (n >> 1) & 1, a.err, DEVERR_WAIT_EPILOGUE))) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((n & 1) ? C::kAcc1 : 0) + (static_cast<uint32_t>(32 * q) << 16);
      const int row0 = mt * 256 + cta * 128 + 32 * q, n0 = nt * 256;
      // fp32 takes twice the stores; after the last tile the stages are free, each store has a block of its own there, and
      // none waits for the one before (130 x 4096 -> 6144: 12.2 and 11.7 us; bf16 gains nothing)
      const bool last = !a.y_bf16 && tile + pairs >= tiles;
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
        pair_store(a, &tm_y, v, row0, n0 + c, lane, last ? smem + (warp - 2) * 16384 + j * 2048 : out, last);
      }
    }
    if (lane == 0) bulk_wait_read<0>();  // the writes themselves end with the grid
    tc_fence_before();
  }
  __syncthreads();
  if constexpr (S > 1) {
    cluster_sync_all();
    int mt, nt;
    pair_tile(a, pair, mt, nt);
    pair_reduce<S>(a, smem_u32(smem), cta, slice, mt * 256 + cta * 128, nt * 256);
  }
  cluster_sync_all();  // no CTA frees memory that the others' instructions may still use
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

}  // namespace

namespace {

// Clusters of 2 * S CTAs of k_mx4_pair<S> that the current device holds at once (looked up once per device).
template <int S>
int resident_clusters() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * S);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = PairCfg::kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(k_mx4_pair<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(PairCfg::kSmem)) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k_mx4_pair<S>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 0;
    }
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

// Up to 128 tokens a tile's MMAs have as many columns as there are tokens, and the split kernel streams weights
// through all SMs; above, 256 x 256 tiles load less for each product (130 x 4096 -> 6144, bf16: 10.7 us, and 11.5 with
// 144-column tiles; 256 x 8192 -> 8192: 15.6 and 17.8; both with five stages. With six 10.6 and 14.2).
Mx4Plan plan_mx4(int T, int N, int K) {
  Mx4Plan p{};
  int sms = decode_grid_sms();
  if (sms == 0) sms = 148;
  const int stages = static_cast<int>(ceil_div(K, kMxStageK));
  p.splits = 1;
  p.pair = T > 128;
  if (p.pair) {
    p.n_tiles = static_cast<int>(ceil_div(N, 256));
    p.t_tiles = static_cast<int>(ceil_div(T, 256));
    const int64_t tiles = static_cast<int64_t>(p.n_tiles) * p.t_tiles;
    // K slices where the tiles leave SMs idle and a slice's saving (0.29 us a stage) exceeds the 2 to 3 us that the
    // larger cluster and its sum cost: 512 x 8192 -> 1024: 15.0, 12.8 and 11.5 us with 1, 2 and 4 slices;
    // 512 x 4096 -> 4096: 10.9 and 11.7 with 1 and 2
    if (stages >= 20) {
      if (tiles <= resident_clusters<4>()) p.splits = 4;
      else if (tiles <= resident_clusters<2>()) p.splits = 2;
    }
    p.ctas = static_cast<int>(p.splits > 1 ? 2 * p.splits * tiles : 2 * std::min<int64_t>(sms / 2, tiles));
    return p;
  }
  p.n_tiles = static_cast<int>(ceil_div(N, 128));
  p.t_tiles = 1;
  // as many CTAs as two per SM hold, in clusters of at most eight along K, with three stages each at least
  // (128 x 1536 -> 8960: 8.5, 7.9 and 10.5 us with 1, 2 and 4; 1 x 8192 -> 1024: 17.6, 11.1, 7.5 and 5.6 with 1, 2, 4 and 8)
  while (p.splits < 8 && static_cast<int64_t>(p.n_tiles) * p.splits <= sms && stages >= 6 * p.splits) p.splits *= 2;
  p.ctas = p.n_tiles * p.splits;
  return p;
}

cudaError_t launch_mx4_pair(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const CUtensorMap& tm_ws,
                            const CUtensorMap& tm_xs, const CUtensorMap* tm_y, const Mx4Plan& p, int T, int N, int K,
                            void* Y, bool y_bf16, bool w_early, int* err, cudaStream_t st) {
  using C = PairCfg;
  auto k = p.splits == 1 ? k_mx4_pair<1> : p.splits == 2 ? k_mx4_pair<2> : k_mx4_pair<4>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  PairArgs a{};
  a.T = T;
  a.N = N;
  a.K = K;
  a.m_tiles = p.t_tiles;
  a.n_tiles = p.n_tiles;
  // Token tiles walked together while a tile of weights is in use: as many as keep their activations within 36 MB
  // of L2, in equal groups, so that the weights are read from HBM once for each group (8192 x 8192 -> 29568, sustained, with
  // five stages: 776 us in groups of 8, 743 in one of 32; 8192 x 29568 -> 8192: 766 in groups of 8, 825 in one of 32).
  const int most = static_cast<int>(std::max<int64_t>(1, (int64_t(36) << 20) / (int64_t(256) * K * 17 / 32)));
  a.group = static_cast<int>(ceil_div(p.t_tiles, ceil_div(p.t_tiles, most)));
  a.Y = Y;
  a.y_bf16 = y_bf16;
  a.tma = tm_y != nullptr;
  a.w_early = w_early;
  a.err = err;
  return launch_dependent(k, dim3(static_cast<unsigned>(p.ctas)), kPairThreads, C::kSmem, 2 * p.splits, st, tm_x, tm_w, tm_xs,
                          tm_ws, tm_y ? *tm_y : tm_x, a);
}

cudaError_t launch_mx4_split(const CUtensorMap& tm_w, const CUtensorMap& tm_x, const Mx4Plan& p, const uint8_t* w_scales,
                             const uint8_t* x_scales, int T, int N, int K, void* Y, bool y_bf16, bool w_early, int* err,
                             cudaStream_t st) {
  SplitArgs a{};
  a.w_scales = w_scales;
  a.x_scales = x_scales;
  a.T = T;
  a.N = N;
  a.K = K;
  a.KT = static_cast<int>(ceil_div(K, kMxTileCols));
  a.bn = static_cast<int>(round_up(T, 16));
  a.splits = p.splits;
  a.stages = split_stages(a.bn);
  const int cols = a.bn + 2 * kSplitSfCols;
  a.tmem_cols = cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
  a.w_early = w_early;
  a.Y = Y;
  a.y_bf16 = y_bf16;
  a.err = err;
  const size_t smem = 1024 + size_t(a.stages) * split_stage_bytes(a.bn) + 256;
  cudaError_t e = cudaFuncSetAttribute(k_mx4_split, cudaFuncAttributeMaxDynamicSharedMemorySize, 114 * 1024);
  if (e != cudaSuccess) return e;
  return launch_dependent(k_mx4_split, dim3(static_cast<unsigned>(p.ctas)), kSplitThreads, smem, p.splits, st, tm_w, tm_x, a);
}

}  // namespace qe
