// y = x . w^T with both operands in microscaled 4-bit floating point, on the
// block-scaled tcgen05 tensor cores (kind::mxf4 / kind::mxf4nvf4): the
// products of e2m1 codes are scaled by their blocks' scales inside the MMA
// and accumulated in fp32 tensor memory; nothing is dequantized.
//
//   y[m, n] = xrow[m] wrow[n] sum_b sx[m, b] sw[n, b] sum_{k in b} cx[m, k] cw[n, k]
//
// (the row scales only for nv; applied to the fp32 sum, then one rounding to
// bf16).
//
// The weight is always the A operand and the tokens the B operand: up to 128
// tokens a CTA takes 128 output channels x NB = 16 ... 128 token columns, so
// a decode step streams the weight once through tiles of 16 columns; above,
// two CTAs work on 256 channels x 256 or 384 tokens (pair kernel, below).  A
// stage is 256 channels: 128-byte rows of codes (TMA, 128-byte swizzle) and 2
// (mx) or 4 (nv) scale tiles of 512 bytes per 128 rows, copied to shared
// memory in one piece and to TMEM by tcgen05.cp, which the tensor pipe runs in
// order with the MMAs.  A K tail of 128 channels issues half the stage's MMAs.
//
// Warp roles: 0 TMA producer, 1 TMEM allocation and MMA issue, 2..5
// epilogue.  K may be split over a thread-block cluster of up to 8 CTAs (few
// tiles); the fp32 partial tiles are added through distributed shared memory
// in rank order, so a launch configuration always gives the same bits.
//
// Every mbarrier wait is bounded; see w4_common.cuh.  Two kinds of waits are
// not: CTA and cluster barriers, which every thread reaches, also after a wait
// that gave up (no role returns early); and the allocation of tensor memory,
// which waits for CTAs on the same SM to free theirs.  Those never wait for
// this kernel: dependents are let start only once a CTA holds its own.
#include <cooperative_groups.h>
#include <cudaTypedefs.h>

#include "fp4.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace cg = cooperative_groups;

namespace {

constexpr int kFp4Threads = 192;
constexpr int kRows = 128;       // output channels of a tile
constexpr int kStageK = 256;     // channels of a stage
constexpr int kMaxSplit = 8;
constexpr unsigned kKernelIdFp4 = 8;

template <int FMT, int NB>
struct Fp4Tile {
  static_assert(NB <= 128, "one scale tile across the tokens");
  static constexpr int kWords = fp4_stage_words(FMT);
  static constexpr uint32_t kABytes = kRows * kStageK / 2;
  static constexpr uint32_t kBBytes = NB * kStageK / 2;
  static constexpr uint32_t kSfaBytes = kWords * 512;
  static constexpr uint32_t kSfbBytes = kWords * 512;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr int kMinSplitKb = NB <= 32 ? 6 : NB == 64 ? 4 : 2;
  static constexpr int kStages = static_cast<int>(109u * 1024u / kStageBytes);  // two CTAs per SM
  // TMEM: NB accumulator columns, then the scale columns of two stages.
  static constexpr uint32_t kSfCols = 4 * kWords * 2;
  static constexpr uint32_t kUsed = NB + 2 * kSfCols;
  static constexpr uint32_t kTmemCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  static_assert(kUsed <= 256, "two CTAs' TMEM fits an SM");
  static constexpr uint32_t bars = kStages * kStageBytes;
  static constexpr uint32_t misc = bars + (2 * kStages + 2) * 8;
  static constexpr size_t bytes = misc + 16 + 1024;  // + alignment
};

struct Fp4Args {
  const uint8_t* wscales;
  const uint8_t* xscales;
  const float* wrow;
  const float* xrow;
  __nv_bfloat16* y;
  int M, N, K;
  int m_tiles;
  int tiles;  // pair kernel: all tiles
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 32 rows of 16 bytes (unswizzled 8-row core matrices, 128 bytes apart) to
// 32 TMEM lanes x 4 columns, repeated in all four lane quarters.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t smem) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 32;  // SBO
  d |= static_cast<uint64_t>(1u) << 46;         // descriptor version
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Instruction descriptor of the block-scaled kinds: e2m1 operands, K-major,
// M x N, scale ids within a TMEM scale word.
template <int FMT>
__device__ __forceinline__ constexpr uint32_t idesc_fp4(int N, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4)       // B scale id
         | (1u << 7) | (1u << 10)                  // A, B: e2m1
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | ((FMT == kFp4Mx ? 1u : 0u) << 23)       // scales: ue8m0, else ue4m3
         | (static_cast<uint32_t>(kRows >> 7) << 27)  // M / 128
         | (static_cast<uint32_t>(sf_id) << 29);   // A scale id
}

template <int FMT>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == kFp4Mx)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

template <int FMT, int NB>
__global__ void __launch_bounds__(kFp4Threads)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                    const Fp4Args a, int static_w, unsigned* err) {
  using T = Fp4Tile<FMT, NB>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  auto stage = [&](int s) { return base + static_cast<uint32_t>(s) * T::kStageBytes; };
  auto full = [&](int s) { return base + T::bars + 8u * s; };
  auto empty = [&](int s) { return base + T::bars + 8u * (S + s); };
  const uint32_t acc_full = base + T::bars + 8u * (2 * S);
  const uint32_t done_bar = acc_full + 8u;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + T::misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + T::misc + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int ks, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tile = static_cast<int>(blockIdx.x) / ks;
  const int tile_m = tile % a.m_tiles;  // token tiles of one weight tile run together
  const int tile_n = tile / a.m_tiles;
  const int n0 = tile_n * kRows;
  const int m0 = tile_m * NB;
  const int all_kb = (a.K + kStageK - 1) / kStageK;
  const int kb_begin = static_cast<int>(static_cast<int64_t>(rank) * all_kb / ks);
  const int num_kb = static_cast<int>(static_cast<int64_t>(rank + 1) * all_kb / ks) - kb_begin;
  // 512-byte scale tiles of one 128-row tile.
  const int words = a.K / (4 * fp4_block(FMT));

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), T::kTmemCols);  // no limit: see above
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The next kernel may be scheduled from here on: not before this CTA holds
  // its TMEM, or a dependent that allocated first would wait for this kernel
  // while this CTA waits for its TMEM.
  if (threadIdx.x == 0) pdl_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA --
    // The whole warp walks the stages and one elected lane issues: the
    // operands of TMA and tcgen05 instructions stay warp-uniform.
    const bool one = elect_one();
    auto scale_bytes = [&](int kb) {  // of a row tile: fewer in a K tail
      const int left = words - (kb_begin + kb) * T::kWords;
      return static_cast<uint32_t>(left < T::kWords ? left : T::kWords) * 512u;
    };
    auto load_w = [&](int st, int kb) {
      const uint32_t w = scale_bytes(kb);
      mbar_arrive_expect_tx(full(st), T::kABytes + T::kBBytes + 2 * w);
      tma_load_2d(stage(st), &tw, (kb_begin + kb) * (kStageK / 2), n0, full(st));
      bulk_load(stage(st) + T::kABytes + T::kBBytes,
                a.wscales + (static_cast<int64_t>(tile_n) * words +
                             static_cast<int64_t>(kb_begin + kb) * T::kWords) * 512,
                w, full(st));
    };
    auto load_x = [&](int st, int kb) {
      const uint32_t w = scale_bytes(kb);
      tma_load_2d(stage(st) + T::kABytes, &tx, (kb_begin + kb) * (kStageK / 2), m0, full(st));
      bulk_load(stage(st) + T::kABytes + T::kBBytes + T::kSfaBytes,
                a.xscales + (static_cast<int64_t>(m0 / 128) * words +
                             static_cast<int64_t>(kb_begin + kb) * T::kWords) * 512,
                w, full(st));
    };
    const int first = num_kb < S ? num_kb : S;
    if (!static_w) pdl_wait();
    for (int kb = 0; kb < first; ++kb) {
      if (one) {
        load_w(kb, kb);
        if (!static_w) load_x(kb, kb);
      }
    }
    if (static_w) {
      pdl_wait();
      for (int kb = 0; kb < first; ++kb)
        if (one) load_x(kb, kb);
    }
    int st = 0;
    uint32_t ph = 1;  // phase of stage st that is being filled
    int kb = first;
    for (; kb < num_kb; ++kb) {
      if (!mbar_wait(empty(st), ph ^ 1u, abort_flag, err, kKernelIdFp4)) break;
      if (one) {
        load_w(st, kb);
        load_x(st, kb);
      }
      if (++st == S) st = 0, ph ^= 1u;
    }
    if (*abort_flag && one) {
      // Drain this CTA's own loads before leaving.
      for (int k = kb - S; k < kb; ++k) {
        if (k < 0) continue;
        volatile int dummy = 0;
        mbar_wait(full(k % S), (k / S) & 1u, &dummy, err, kKernelIdFp4, kWaitLimitNs / 4);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA --
    const bool one = elect_one();
    bool issued = false;
    int st = 0;
    uint32_t ph = 0;
    // The loads wait for the preceding kernel, however long it runs: the limit
    // of the waits below starts after it.
    pdl_wait();
    for (int kb = 0; kb < num_kb; ++kb) {
      if (!mbar_wait(full(st), ph, abort_flag, err, kKernelIdFp4)) break;
      tc_fence_after();
      const bool whole = a.K - (kb_begin + kb) * kStageK >= kStageK;  // else a tail of 128 channels
      const uint32_t sfa = tmem + NB + (kb & 1) * T::kSfCols;
      const uint32_t sfb = sfa + 4 * T::kWords;
      const uint32_t sf_smem = stage(st) + T::kABytes + T::kBBytes;
      const uint64_t da = sdesc_k_sw128(stage(st));
      const uint64_t db = sdesc_k_sw128(stage(st) + T::kABytes);
      if (one) {
#pragma unroll
        for (int w = 0; w < T::kWords; ++w) {
          if (w < T::kWords / 2 || whole) {
            tmem_cp_scales(sfa + 4 * w, sf_smem + 512 * w);
            tmem_cp_scales(sfb + 4 * w, sf_smem + T::kSfaBytes + 512 * w);
          }
        }
#pragma unroll
        for (int kk = 0; kk < kStageK / 64; ++kk) {
          // 64 channels are 32 bytes (+2 in the address field); an mx scale
          // word holds two such steps, an nv word one.
          const int w = FMT == kFp4Mx ? kk / 2 : kk;
          const int id = FMT == kFp4Mx ? (kk & 1) * 2 : 0;
          if (kk < kStageK / 128 || whole)
            umma_fp4<FMT>(tmem, da + 2ull * kk, db + 2ull * kk, idesc_fp4<FMT>(NB, id), sfa + 4 * w,
                          sfb + 4 * w, (kb | kk) != 0);
        }
        umma_commit(empty(st));
      }
      issued = true;
      if (++st == S) st = 0, ph ^= 1u;
    }
    if (one) {
      if (!*abort_flag) {
        umma_commit(acc_full);
      } else if (issued) {
        umma_commit(done_bar);  // in-flight MMAs end before TMEM is freed
        volatile int dummy = 0;
        mbar_wait(done_bar, 0, &dummy, err, kKernelIdFp4, kWaitLimitNs / 4);
      }
    }
  } else {
    // ------------------------------------------------------- epilogue --
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const int n = n0 + 32 * q + lane;
    pdl_wait();
    const float wr = (a.wrow && n < a.N) ? __ldg(a.wrow + n) : 1.f;
    const bool ok = mbar_wait(acc_full, 0, abort_flag, err, kKernelIdFp4);
    tc_fence_after();
    if (ok) {
      const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
      if (ks > 1) {
        // fp32 partial tile [token][channel] into the idle stage buffers.
        float* part = reinterpret_cast<float*>(base_ptr);
#pragma unroll 1
        for (int c = 0; c < NB; c += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(lane_addr + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            part[(c + i) * kRows + 32 * q + lane] = __uint_as_float(r[i]);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < NB; c += 16) {
          if (m0 + c >= a.M) break;
          uint32_t r[16];
          tmem_ld_32x32b_x16(lane_addr + c, r);
          tmem_ld_wait();
          if (n < a.N) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int m = m0 + c + i;
              if (m < a.M) {
                const float xr = a.xrow ? __ldg(a.xrow + m) : 1.f;
                a.y[static_cast<int64_t>(m) * a.N + n] =
                    __float2bfloat16_rn(__uint_as_float(r[i]) * wr * xr);
              }
            }
          }
        }
      }
    }
  }

  if (ks > 1) {
    // Every thread of every CTA of the cluster passes both barriers, also
    // after a timeout, so none is left waiting (they have no limit of their own).
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // all partial tiles written
    if (warp >= 2 && !*abort_flag) {
      // CTA `rank` adds its share of the tile (pieces of 4 channels of a
      // token) over the cluster in rank order.
      const int live = a.M - m0 < NB ? a.M - m0 : NB;
      const int total = live * (kRows / 4);
      const int e1 = static_cast<int>(static_cast<int64_t>(rank + 1) * total / ks);
      float* part = reinterpret_cast<float*>(base_ptr);
      for (int e = static_cast<int>(static_cast<int64_t>(rank) * total / ks) + threadIdx.x - 64;
           e < e1; e += kFp4Threads - 64) {
        const int off = 4 * e;
        float4 t[kMaxSplit];
#pragma unroll
        for (int p = 0; p < kMaxSplit; ++p)
          if (p < ks) t[p] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, p) + off);
        float v[4] = {t[0].x, t[0].y, t[0].z, t[0].w};
#pragma unroll
        for (int p = 1; p < kMaxSplit; ++p)
          if (p < ks) {
            v[0] += t[p].x;
            v[1] += t[p].y;
            v[2] += t[p].z;
            v[3] += t[p].w;
          }
        const int m = m0 + off / kRows, n = n0 + off % kRows;
        const float xr = a.xrow ? __ldg(a.xrow + m) : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (a.wrow && n + i < a.N) v[i] *= __ldg(a.wrow + n + i);
        __nv_bfloat16* dst = a.y + static_cast<int64_t>(m) * a.N + n;
        if (n + 4 <= a.N && (a.N & 3) == 0) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0] * xr, v[1] * xr);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(v[2] * xr, v[3] * xr);
          *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                      *reinterpret_cast<const uint32_t*>(&hi));
        } else {
          for (int i = 0; i < 4; ++i)
            if (n + i < a.N) dst[i] = __float2bfloat16_rn(v[i] * xr);
        }
      }
    }
    cluster.sync();  // peers keep their partials until every reader is done
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, T::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Pair kernel (more than 128 tokens): a cluster of two CTAs computes a tile
// of 256 output channels x NB tokens with cta_group::2 MMAs.  Each CTA holds
// its 128 channels' codes and half of the tokens' codes, so a token tile is
// fetched once for 256 channels.
//
// What bounds a large product is the traffic from L2 into shared memory: the
// tensor pipe takes 256 channels of a 128 x 256 tile in 512 cycles, in which
// a CTA working alone has to fetch 54 KB (nv).  Per multiply-add a pair
// fetches 0.70 (NB = 256) or 0.59 (NB = 384) of that.  NB = 384 is two MMAs
// of 192 columns; with the scale columns of two stages it fills TMEM (384 +
// 2 x 64 of 512 columns).
//
// Persistent: one pair per two SMs walks the tiles; the loads of the next
// tile run under the epilogue of the last, and its MMAs under the stores (the
// accumulators are single: they are handed back once they are in registers).
//
// Both CTAs' loads complete on the first CTA's barrier of the stage, whose
// MMA warp issues for both (all loads are tensor-map loads, which may signal
// the peer's barrier; scale tiles are rows of 256 words).  MMA completion is
// committed to both CTAs' barriers.
//
// Issue order and uniformity matter as much as bandwidth: with the MMA loop
// under `lane == 0` every tcgen05 operand went through a vector register and
// one pair alone took 1.16 us per stage (NB = 384, nv); with the warp walking
// the loop and an elected lane issuing 0.62 us; with the loads signalling the
// first CTA's barrier themselves, where a relaying thread of each CTA had
// passed "stage full" on, 0.45 us (NB = 256: 0.30).  With every pair at work a
// stage takes 0.57 (0.39) us: 8192 x 5120 x 17408 runs at 5.4 ... 5.9 PFLOP/s in
// short bursts, and at 4.7 once the power limit has brought the SM clock down to
// 1.2 GHz.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 64 + 256;

template <int FMT, int NB>
struct PairTile {
  static constexpr int kParts = NB > 256 ? 2 : 1;          // MMAs side by side
  static constexpr int kPartN = NB / kParts;               // their columns
  static constexpr int kSfTiles = NB / 128;                // scale tiles across the tokens
  static constexpr int kWords = fp4_stage_words(FMT);
  static constexpr uint32_t kABytes = kRows * kStageK / 2;
  static constexpr uint32_t kPartBytes = kPartN / 2 * kStageK / 2;  // one CTA's half of a part
  static constexpr uint32_t kBBytes = kParts * kPartBytes;
  static constexpr uint32_t kSfaBytes = kWords * 512;
  static constexpr uint32_t kSfbBytes = kSfTiles * kWords * 512;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr int kStages = static_cast<int>(222u * 1024u / kStageBytes);
  static constexpr uint32_t kSfCols = 4 * kWords * (1 + kSfTiles);
  static_assert(NB + 2 * kSfCols <= 512, "accumulators and two stages of scales fit TMEM");
  static constexpr uint32_t bars = kStages * kStageBytes;
  static constexpr uint32_t misc = bars + (2 * kStages + 3) * 8;
  static constexpr uint32_t xrow = (misc + 16 + 15) & ~15u;  // NB token scales
  static constexpr size_t bytes = xrow + NB * 4 + 1024;
};

__device__ __forceinline__ void pair_cp_scales(uint32_t taddr, uint32_t smem) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

template <int FMT>
__device__ __forceinline__ void pair_umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == kFp4Mx)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
        "[%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Arrives on the barrier at this offset in both CTAs when the MMAs issued so
// far have completed.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Arrives on the barrier at this offset in CTA 0 of the pair.
__device__ __forceinline__ void arrive_at_first(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(bar)
      : "memory");
}

// 2-D tiled load into this CTA's shared memory, completion counted on the
// barrier at this offset in CTA 0 of the pair (`bar`: its cluster address).
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}

// mbar_wait whose success also makes the peer CTA's writes visible.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity,
                                                  volatile int* abort, unsigned* err) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (it == 0) t0 = globaltimer();
    if ((it & 63u) == 63u) {
      if (*abort) return false;
      if (globaltimer() - t0 > kWaitLimitNs) {
        *abort = 1;
        record_error(err, kErrWaitTimeout, kKernelIdFp4);
        return false;
      }
    }
  }
}

template <int FMT, int NB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
    fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tw,
                         const __grid_constant__ CUtensorMap tx,
                         const __grid_constant__ CUtensorMap tws,
                         const __grid_constant__ CUtensorMap txs, const Fp4Args a, int static_w,
                         unsigned* err) {
  using T = PairTile<FMT, NB>;
  constexpr int S = T::kStages;
  extern __shared__ uint8_t smem_raw[];
  // The dynamic shared memory starts at the same address in both CTAs, so
  // offsets (descriptors, barriers) agree between them.
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  auto stage = [&](int s) { return base + static_cast<uint32_t>(s) * T::kStageBytes; };
  auto full = [&](int s) { return base + T::bars + 8u * s; };
  auto empty = [&](int s) { return base + T::bars + 8u * (S + s); };
  const uint32_t acc_full = base + T::bars + 8u * (2 * S);
  const uint32_t acc_empty = acc_full + 8u;
  const uint32_t done_bar = acc_full + 16u;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + T::misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + T::misc + 8);
  float* xrow_s = reinterpret_cast<float*>(base_ptr + T::xrow);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int pairs = static_cast<int>(gridDim.x >> 1);
  const int my_tiles = a.tiles > pair ? (a.tiles - pair + pairs - 1) / pairs : 0;
  const int num_kb = (a.K + kStageK - 1) / kStageK;
  // Tile i of this pair; the token tiles of one weight tile run together.
  auto tile_n0 = [&](int i) {
    return ((pair + i * pairs) / a.m_tiles) * 2 * kRows + static_cast<int>(rank) * kRows;
  };
  auto tile_m0 = [&](int i) { return ((pair + i * pairs) % a.m_tiles) * NB; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * 8);  // the epilogue warps of both CTAs
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
    tma_prefetch_desc(&tws);
    tma_prefetch_desc(&txs);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cg::cluster_group cluster = cg::this_cluster();
  // Barriers of both CTAs are initialized.  Neither the allocation above nor the
  // three cluster barriers have a limit: a cluster's CTAs start together, and
  // all their threads reach each of them.
  cluster.sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0) pdl_launch_dependents();  // holds its TMEM, as above

  if (warp == 0) {
    // ------------------------------------------------------------ TMA --
    const bool one = elect_one();
    const uint32_t full0 = in_first(full(0));
    // Boxes that reach over the end of a tensor (K tail, last row tiles) are
    // filled with zeros and count in full.
    auto load_w = [&](int st, int n0, int kb) {
      if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * T::kStageBytes);
      pair_load_2d(stage(st), &tw, kb * (kStageK / 2), n0, full0 + 8u * st);
      pair_load_2d(stage(st) + T::kABytes + T::kBBytes, &tws, kb * 256, n0 / 128, full0 + 8u * st);
    };
    auto load_x = [&](int st, int m0, int kb) {
#pragma unroll
      for (int p = 0; p < T::kParts; ++p)
        pair_load_2d(stage(st) + T::kABytes + p * T::kPartBytes, &tx, kb * (kStageK / 2),
                     m0 + p * T::kPartN + static_cast<int>(rank) * (T::kPartN / 2),
                     full0 + 8u * st);
      pair_load_2d(stage(st) + T::kABytes + T::kBBytes + T::kSfaBytes, &txs, kb * 256, m0 / 128,
                   full0 + 8u * st);
    };
    // The weight's first stages may be fetched before the preceding kernel
    // ends if the caller says that it does not write them.
    int ahead = 0;
    if (static_w && my_tiles > 0)
      for (; ahead < S && ahead < num_kb; ++ahead)
        if (one) load_w(ahead, tile_n0(0), ahead);
    pdl_wait();
    int st = 0, filled = 0;  // next stage; stages begun, counted up to S
    uint32_t ph = 0;         // phase of stage st that is being filled
    for (int i = 0; i < my_tiles && !*abort_flag; ++i) {
      const int n0 = tile_n0(i), m0 = tile_m0(i);
      for (int kb = 0; kb < num_kb; ++kb) {
        if (filled == S) {
          if (!mbar_wait_cluster(empty(st), ph ^ 1u, abort_flag, err)) break;
        } else {
          ++filled;
        }
        if (one) {
          if (i > 0 || kb >= ahead) load_w(st, n0, kb);
          load_x(st, m0, kb);
        }
        if (++st == S) st = 0, ph ^= 1u;
      }
    }
    if (*abort_flag && one && rank == 0) {
      // Drain both CTAs' loads: of each stage, the fill begun last.  A fill
      // that the peer did not begin cannot complete; it is waited for up to
      // the limit.
      for (int k = 0; k < (ahead > filled ? ahead : filled); ++k) {
        volatile int dummy = 0;
        mbar_wait(full(k), k < st ? ph : ph ^ (filled == S ? 1u : 0u), &dummy, err, kKernelIdFp4,
                  kWaitLimitNs / 4);
      }
    }
  } else if (warp == 1) {
    // The whole warp walks the stages and one elected lane issues: the
    // operands of the tcgen05 instructions stay warp-uniform.
    const bool one = elect_one();
    if (rank == 0) {
      // ------------------------------------------------------------ MMA --
      bool issued = false;
      int st = 0;
      uint32_t ph = 0, buf = 0;
      pdl_wait();  // as above: no limit runs while the preceding kernel does
      for (int i = 0; i < my_tiles && !*abort_flag; ++i) {
        // Both CTAs have read the last tile's accumulators.
        if (i > 0 && !mbar_wait_cluster(acc_empty, (i - 1) & 1u, abort_flag, err)) break;
        tc_fence_after();
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_cluster(full(st), ph, abort_flag, err)) break;
          tc_fence_after();
          const uint32_t sfa = tmem + NB + buf * T::kSfCols;
          const uint32_t sfb = sfa + 4 * T::kWords;
          const uint32_t sf_smem = stage(st) + T::kABytes + T::kBBytes;
          const uint64_t da = sdesc_k_sw128(stage(st));
          const uint64_t db = sdesc_k_sw128(stage(st) + T::kABytes);
          const bool whole = a.K - kb * kStageK >= kStageK;  // else a tail of 128 channels
          if (one) {
#pragma unroll
            for (int w = 0; w < T::kWords; ++w) {
              if (w < T::kWords / 2 || whole) {
                pair_cp_scales(sfa + 4 * w, sf_smem + 512 * w);
#pragma unroll
                for (int c = 0; c < T::kSfTiles; ++c)
                  pair_cp_scales(sfb + 4 * (w * T::kSfTiles + c),
                                 sf_smem + T::kSfaBytes + 512 * (c * T::kWords + w));
              }
            }
#pragma unroll
            for (int kk = 0; kk < kStageK / 64; ++kk) {
              const int w = FMT == kFp4Mx ? kk / 2 : kk;
              const int id = FMT == kFp4Mx ? (kk & 1) * 2 : 0;
              // M = 256 here: one more in the descriptor's M / 128 field.
              const uint32_t idesc = idesc_fp4<FMT>(T::kPartN, id) + (1u << 27);
              if (kk < kStageK / 128 || whole) {
#pragma unroll
                for (int p = 0; p < T::kParts; ++p)
                  pair_umma<FMT>(tmem + p * T::kPartN, da + 2ull * kk,
                                 db + static_cast<uint64_t>(p * (T::kPartBytes >> 4)) + 2ull * kk,
                                 idesc, sfa + 4 * w,
                                 sfb + 4 * w * T::kSfTiles + p * (T::kPartN / 32), (kb | kk) != 0);
              }
            }
            pair_commit(empty(st));
          }
          issued = true;
          buf ^= 1u;
          if (++st == S) st = 0, ph ^= 1u;
        }
        if (one && !*abort_flag) pair_commit(acc_full);
      }
      if (*abort_flag && issued && one) {
        pair_commit(done_bar);  // in-flight MMAs end before TMEM is freed
        volatile int dummy = 0;
        mbar_wait(done_bar, 0, &dummy, err, kKernelIdFp4, kWaitLimitNs / 4);
      }
    }
  } else {
    // ------------------------------------------------------- epilogue --
    const int q = warp & 3;             // TMEM lane quarter of this warp
    const int half = (warp - 2) >> 2;   // columns [half * NB / 2, + NB / 2)
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    pdl_wait();
    for (int i = 0; i < my_tiles; ++i) {
      const int n = tile_n0(i) + 32 * q + lane, m0 = tile_m0(i);
      const float wr = (a.wrow && n < a.N) ? __ldg(a.wrow + n) : 1.f;
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the last tile's scales are read
      for (int c = threadIdx.x - 64; c < NB; c += 256)
        xrow_s[c] = a.xrow && m0 + c < a.M ? __ldg(a.xrow + m0 + c) : 1.f;
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the eight epilogue warps
      const bool ok = mbar_wait_cluster(acc_full, i & 1u, abort_flag, err);
      tc_fence_after();
      if (ok) {
        const int c0 = half * (NB / 2);
        const int live = a.M - m0 - c0;  // columns that are tokens
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.y) + static_cast<int64_t>(m0 + c0) * a.N + n;
        // Columns c0 + 32 j + 0 ... 31, rounded, two per word.
        auto fetch = [&](int j, uint32_t offset, uint32_t* v) {
          uint32_t r[2][16];
          __syncwarp();
          tmem_ld_32x32b_x16(lane_addr + c0 + 32 * j + offset, r[0]);
          tmem_ld_32x32b_x16(lane_addr + c0 + 32 * j + 16 + offset, r[1]);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 xr = *reinterpret_cast<const float2*>(xrow_s + c0 + 32 * j + 2 * x);
            const __nv_bfloat162 y = __floats2bfloat162_rn(
                __uint_as_float(r[x >> 3][2 * x & 15]) * wr * xr.x,
                __uint_as_float(r[x >> 3][(2 * x & 15) + 1]) * wr * xr.y);
            v[x] = *reinterpret_cast<const uint32_t*>(&y);
          }
        };
        auto store = [&](int j, const uint32_t* v) {
          if (n >= a.N) return;
          if (32 * j + 32 <= live) {
#pragma unroll
            for (int x = 0; x < 32; ++x, dst += a.N)
              *dst = static_cast<uint16_t>(v[x / 2] >> (16 * (x & 1)));
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x, dst += a.N)
              if (32 * j + x < live) *dst = static_cast<uint16_t>(v[x / 2] >> (16 * (x & 1)));
          }
        };
        if (i + 1 == my_tiles) {
#pragma unroll 1
          for (int j = 0; j < NB / 64 && 32 * j < live; ++j) {
            uint32_t v[16];
            fetch(j, 0, v);
            store(j, v);
          }
        } else {
          // All columns go to registers first and the accumulators are handed
          // back before any of them is stored: the next tile's MMAs run under
          // the stores (1999 x 11008 x 4096: 40.5 -> 38.2 us).
          uint32_t held[NB / 64][16];
          // 0, in a way that makes each read of 32 columns depend on the last
          // one's results: read ahead, they would spill.
          const uint32_t zero = static_cast<uint32_t>(a.M >> 31);
          uint32_t order = 0;
#pragma unroll
          for (int j = 0; j < NB / 64; ++j) {
            fetch(j, order & zero, held[j]);
#pragma unroll
            for (int x = 0; x < 16; ++x) order |= held[j][x];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at_first(acc_empty);
#pragma unroll
          for (int j = 0; j < NB / 64; ++j)
            if (32 * j < live) store(j, held[j]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster.sync();  // neither CTA's memory is in use by the other any more
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
  cluster.sync();  // both are there until both have freed their TMEM
}

PFN_cuTensorMapEncodeTiled encode_fn() {
  static PFN_cuTensorMapEncodeTiled fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !p)
      return nullptr;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled>(p);
  }
  return fn;
}

// Codes [rows, K / 2]: boxes of one stage's 128 bytes by box_rows.
CUresult encode_codes(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int box_rows) {
  const PFN_cuTensorMapEncodeTiled fn = encode_fn();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {kStageK / 2, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Scale tiles [row tiles, K words of 512 bytes]: boxes of one stage's tiles
// (1024 or 2048 bytes, as 256 elements of 4 or 8) by box_tiles row tiles.
CUresult encode_scales(CUtensorMap* map, const void* base, int64_t rows, int64_t K, int fmt,
                       int box_tiles) {
  const PFN_cuTensorMapEncodeTiled fn = encode_fn();
  if (!fn) return CUDA_ERROR_NOT_FOUND;
  const cuuint64_t elem = fmt == kFp4Mx ? 4 : 8;
  const cuuint64_t bytes = static_cast<cuuint64_t>(K / (4 * fp4_block(fmt))) * 512;
  const cuuint64_t dims[2] = {bytes / elem, static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t box[2] = {256, static_cast<cuuint32_t>(box_tiles)};
  const cuuint32_t es[2] = {1, 1};
  return fn(map, fmt == kFp4Mx ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT64, 2,
            const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <auto kern, size_t kBytes>
cudaError_t opt_in_smem() {
  static unsigned long long done = 0;  // bit d: device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kBytes));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELEASE);
  }
  return cudaSuccess;
}

// CTAs that split K: enough to fill the GPU (clusters of odd sizes do not pack
// to the last slot, so 264 of 296 at two per SM), each keeping at least
// `min_kb` stages, under which the ring is latency-bound anyway and the join
// of the partial tiles (0.5 us for 16 tokens, several for 128) is lost time.
// Measured at one token: 5120 x 17408 19.5 us unsplit, 13.9 / 12.4 / 12.0 by
// 2 / 4 / 6; 6144 x 2048 5.4 unsplit, 6.0 / 6.3 by 2 / 4; 17408 x 5120 11.8
// unsplit, 12.4 by 2.  At 128 tokens 2048 x 2048: 12.5 unsplit, 8.4 by 4.
int k_split(int64_t tiles, int num_kb, int min_kb, int num_sms) {
  const int64_t fit = static_cast<int64_t>(num_sms) * 264 / 148 / tiles;
  int ks = num_kb / min_kb;
  if (ks > fit) ks = static_cast<int>(fit);
  return ks < 1 ? 1 : ks > kMaxSplit ? kMaxSplit : ks;
}

template <int FMT, int NB>
cudaError_t launch(const uint8_t* xcodes, const uint8_t* wcodes, Fp4Args a, int static_w,
                   cudaStream_t stream, int num_sms, unsigned* err) {
  using T = Fp4Tile<FMT, NB>;
  constexpr auto kern = fp4_gemm_kernel<FMT, NB>;
  CUtensorMap tw, tx;
  if (encode_codes(&tw, wcodes, a.N, a.K, kRows) != CUDA_SUCCESS ||
      encode_codes(&tx, xcodes, a.M, a.K, NB) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem<kern, T::bytes>();
  if (e != cudaSuccess) return e;
  a.m_tiles = (a.M + NB - 1) / NB;
  const int64_t tiles = static_cast<int64_t>((a.N + kRows - 1) / kRows) * a.m_tiles;
  const int num_kb = (a.K + kStageK - 1) / kStageK;
  const int ks = k_split(tiles, num_kb, T::kMinSplitKb, num_sms);
  static_assert(NB * kRows * 4 <= T::kStages * T::kStageBytes, "a partial tile fits the stages");
  if (tiles * ks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * ks), 1, 1);
  cfg.blockDim = dim3(kFp4Threads, 1, 1);
  cfg.dynamicSmemBytes = T::bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, a, static_w, err);
}

template <int FMT, int NB>
cudaError_t launch_pair(const uint8_t* xcodes, const uint8_t* wcodes, Fp4Args a, int static_w,
                        cudaStream_t stream, int num_sms, unsigned* err) {
  using T = PairTile<FMT, NB>;
  constexpr auto kern = fp4_gemm_pair_kernel<FMT, NB>;
  CUtensorMap tw, tx, tws, txs;
  if (encode_codes(&tw, wcodes, a.N, a.K, kRows) != CUDA_SUCCESS ||
      encode_codes(&tx, xcodes, a.M, a.K, T::kPartN / 2) != CUDA_SUCCESS ||
      encode_scales(&tws, a.wscales, a.N, a.K, FMT, 1) != CUDA_SUCCESS ||
      encode_scales(&txs, a.xscales, a.M, a.K, FMT, T::kSfTiles) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem<kern, T::bytes>();
  if (e != cudaSuccess) return e;
  a.m_tiles = (a.M + NB - 1) / NB;
  const int64_t tiles = static_cast<int64_t>((a.N + 2 * kRows - 1) / (2 * kRows)) * a.m_tiles;
  const int64_t pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  if (tiles > 0x7FFFFFFF - pairs) return cudaErrorInvalidValue;
  a.tiles = static_cast<int>(tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = T::bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tw, tx, tws, txs, a, static_w, err);
}

// Above 128 tokens: the pair kernel with 256 or 384 token columns, or, where
// that leaves most SMs idle over a long K, the single-CTA kernel with 128
// columns and K split over a cluster.  Time model in microseconds, fitted to
// launches of 200 ... 8192 tokens on 148 SMs (within 12 %): waves x (stages x
// per-stage cost + epilogue), plus the join of a split's partial tiles.
// 5120 x 17408 at 200 tokens: pair 25.0, split 19.9; 11008 x 4096 at 200:
// 10.7, 19.3; 8192 tokens x 5120 x 17408: 256 columns 263, 384 columns 249;
// 1999 x 11008 x 4096: 40, 47.
int large_shape(int M, int N, int num_kb, int num_sms) {
  auto waves = [](int64_t tiles, int64_t slots) {
    return static_cast<double>((tiles + slots - 1) / slots);
  };
  const int64_t pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  const int64_t wide = (N + 255) / 256;
  const double p256 = waves(wide * ((M + 255) / 256), pairs) * (0.39 * num_kb + 2.0);
  const double p384 = waves(wide * ((M + 383) / 384), pairs) * (0.57 * num_kb + 3.0);
  const int64_t tiles = static_cast<int64_t>((N + 127) / 128) * ((M + 127) / 128);
  const int64_t slots = 2 * static_cast<int64_t>(num_sms);
  const int ks = k_split(tiles, num_kb, 2, num_sms);
  const double split =
      waves(tiles * ks, slots) * (0.4 * ((num_kb + ks - 1) / ks) + 2.0) + (ks > 1 ? 5.0 : 0.0);
  if (split < p256 && split < p384) return 128;
  return p384 < p256 ? 384 : 256;
}

template <int FMT>
cudaError_t launch_fmt(const uint8_t* xcodes, const uint8_t* wcodes, const Fp4Args& a,
                       int static_w, cudaStream_t s, int sms, unsigned* err) {
  if (a.M <= 16) return launch<FMT, 16>(xcodes, wcodes, a, static_w, s, sms, err);
  if (a.M <= 32) return launch<FMT, 32>(xcodes, wcodes, a, static_w, s, sms, err);
  if (a.M <= 64) return launch<FMT, 64>(xcodes, wcodes, a, static_w, s, sms, err);
  const int shape =
      a.M <= 128 ? 128 : large_shape(a.M, a.N, (a.K + kStageK - 1) / kStageK, sms);
  if (shape == 128) return launch<FMT, 128>(xcodes, wcodes, a, static_w, s, sms, err);
  if (shape == 256) return launch_pair<FMT, 256>(xcodes, wcodes, a, static_w, s, sms, err);
  return launch_pair<FMT, 384>(xcodes, wcodes, a, static_w, s, sms, err);
}

}  // namespace

cudaError_t launch_fp4_linear(const uint8_t* xcodes, const uint8_t* xscales, const float* xrow,
                              int M, const uint8_t* wcodes, const uint8_t* wscales,
                              const float* wrow, int N, int K, int fmt, void* y, bool static_w,
                              cudaStream_t stream, int num_sms, unsigned* err) {
  Fp4Args a;
  a.wscales = wscales;
  a.xscales = xscales;
  a.wrow = wrow;
  a.xrow = xrow;
  a.y = static_cast<__nv_bfloat16*>(y);
  a.M = M;
  a.N = N;
  a.K = K;
  a.m_tiles = 1;
  a.tiles = 0;
  return fmt == kFp4Mx ? launch_fmt<kFp4Mx>(xcodes, wcodes, a, static_w, stream, num_sms, err)
                       : launch_fmt<kFp4Nv>(xcodes, wcodes, a, static_w, stream, num_sms, err);
}

}  // namespace w4
