// Causal attention over the 8-bit paged cache (layout: kv8.cuh), rows kernel:
// decode and short runs of new tokens.
//
//   o_i = sum_j p_ij v_j,  p_i = softmax over j <= len - n + i of
//   scale * q_i . k_j,  k_j = ks[page j] * code,  v_j = vs[page j] * code
//
// Rows: the query heads that share a kv head and the new tokens of a
// sequence are the rows of one problem (row = token * group + head of the
// group), taken 16 at a time as the M of mma.m16n8k16.  The cache is read
// once per 16 rows, so for single tokens the kernel is bound by HBM.
//
// Work split: a thread-block cluster of `ks` CTAs owns one (sequence, kv
// head, 16 rows); its warps take tiles of 64 tokens in turn.  Each warp runs
// its own online softmax; the partial results are joined in a fixed order,
// first over a CTA's warps and then, through distributed shared memory, over
// the cluster: no workspace, and the same bits on every run.
//
// A warp streams its tiles through its own ring of shared memory: each lane
// copies (cp.async, 16 bytes) exactly the bytes of its own operand
// fragments and reads only those back, so the ring needs no barrier.
//   keys:   the columns of score tile j (8 tokens) are the tokens
//           16 (c / 2) + 2 j + c % 2, and k-step s of a lane quad covers
//           channels 64 (s / 4) + 16 t + 4 (s % 4) + 0..3 (the queries are
//           loaded in that order), so a lane's fragments are 16 contiguous
//           bytes of a key row;
//   values: with that order of columns the probabilities that a lane holds
//           after the score product are its A fragments for the tokens
//           16 t .. 16 t + 15, so its value fragments are 16 contiguous bytes
//           of a value row.
// Each lane's 16 score columns lie in one page whatever the page size (>= 16),
// so a key scale and a value scale per lane and tile suffice.
//
// Numerics: codes are exact in fp16.  Each query row is scaled by a power of
// two that brings its largest magnitude into [128, 256) (exact for channels
// within 2^21 of it) and the scores, in fp32, are scaled back with the key
// scale.  Probabilities are weighted by value scale / largest value scale so
// far and rounded to fp16 with a shift of 2^14 (the largest is 2^14, full
// precision down to 2^-28 of it); sums and outputs are fp32.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "kv8.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kTileTokens = 64;
constexpr int kSlots = 3;  // ring slots per warp, alternately key and value tiles
constexpr float kShift = 14.f;  // probabilities are kept times 2^14
constexpr unsigned kKernelIdAttn = 32;

template <int D>
struct AttnSmem {
  static constexpr int kSlotBytes = kTileTokens * D;
  static constexpr int kRing = kWarps * kSlots * kSlotBytes;
  // Joined partial of the CTA (read by the cluster's peers), apart from the
  // ring: rows of D floats, then maxima and sums.
  static constexpr int part = kRing;
  static constexpr int ml = part + 16 * D * 4;
  static constexpr int bytes = ml + 2 * 16 * 4;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four codes -> two packed pairs of fp16 values.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kKvInt8) {
    // 1024 + (code + 128) has the biased code in its low byte.
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

struct AttnArgs {
  Kv8Cache c;
  Kv8Batch bt;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t ldq;
  int q_heads, group, row_tiles;
  float scale_log2;  // softmax scale * log2(e)
};

template <int FMT, int D>
__global__ void __launch_bounds__(kAttnThreads, 2)
    kv8_attention_rows_kernel(const AttnArgs a, unsigned* err) {
  using SM = AttnSmem<D>;
  constexpr int kSteps = D / 16;       // k-steps of the score product
  constexpr int kChunks = D / 64;      // 16-byte pieces of a key row per lane
  constexpr int kDTiles = D / 8;       // 8-channel tiles of the output
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int ks, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int prob = static_cast<int>(blockIdx.x) / ks;
  const int rt = prob % a.row_tiles;
  const int bh = prob / a.row_tiles;
  const int h = bh % a.c.heads, b = bh / a.c.heads;
  pdl_wait();
  pdl_launch_dependents();
  const Kv8Seq s = kv8_sequence(a.bt, b, a.c.log_page);
  if (s.bad && threadIdx.x == 0 && h == 0 && rt == 0 && rank == 0)
    record_error(err, kErrBadIndex, kKernelIdAttn);
  const int n_rows = s.n * a.group;
  const int r0 = rt * 16;
  if (r0 >= n_rows) return;  // the whole cluster
  const int live_rows = n_rows - r0 < 16 ? n_rows - r0 : 16;

  // Rows g and g + 8 of this lane: the last position each sees.
  int limit[2];
  uint32_t qa[kSteps][4];
  float q_back[2];  // undoes the query scaling, times the softmax scale
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = r0 + g + 8 * i;
    const bool live = r < n_rows;
    const int tok = live ? r / a.group : 0;
    limit[i] = live ? s.len - s.n + tok : -1;
    const __nv_bfloat16* qr = a.q + static_cast<int64_t>(s.row0 + tok) * a.ldq +
                              (h * a.group + (live ? r % a.group : 0)) * D;
    uint32_t raw[kSteps][2];
    uint32_t big = 0;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(
                                 qr + 64 * (st / 4) + 16 * t + 4 * (st % 4)))
                           : make_uint2(0, 0);
      raw[st][0] = v.x;
      raw[st][1] = v.y;
      const uint32_t m = __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu);
      big = __vmaxu2(big, m);
    }
    big = max(big & 0xFFFFu, big >> 16);
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // Largest magnitude in [2^e, 2^(e+1)); scaled by 2^(7 - e).
    const int e = static_cast<int>(big >> 7) - 127;
    const float up = __int_as_float((min(7 - e, 126) + 127) << 23);
    q_back[i] = __int_as_float((max(e - 7, -126) + 127) << 23) * a.scale_log2;
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const __half2 x = __floats2half2_rn(__uint_as_float(raw[st][w] << 16) * up,
                                            __uint_as_float(raw[st][w] & 0xFFFF0000u) * up);
        qa[st][2 * w + i] = *reinterpret_cast<const uint32_t*>(&x);
      }
  }

  // Tiles of this CTA: the cluster's tiles in contiguous shares.
  const int last_tok = (r0 + live_rows - 1) / a.group;  // the tile's last new token
  const int keys = s.len - s.n + last_tok + 1;          // <= 0: nothing is seen
  const int first_limit = s.len - s.n + r0 / a.group;
  const int tiles = keys > 0 ? (keys + kTileTokens - 1) / kTileTokens : 0;
  const int t_begin = static_cast<int>(static_cast<int64_t>(rank) * tiles / ks);
  const int t_end = static_cast<int>(static_cast<int64_t>(rank + 1) * tiles / ks);
  const int my_tiles = t_end - t_begin > warp ? (t_end - t_begin - warp + kWarps - 1) / kWarps : 0;

  const int32_t* table = a.bt.table + static_cast<int64_t>(b) * a.bt.max_pages;
  const int page_mask = (1 << a.c.log_page) - 1;
  const uint32_t ring = smem_u32(smem) + warp * (kSlots * SM::kSlotBytes) + lane * 16;
  bool bad_page = false;
  // The page that holds 16-token granule `gr` of tile i, -1 if none does.
  auto page_of = [&](int i, int gr) {
    const int tok = (t_begin + warp + i * kWarps) * kTileTokens + 16 * gr;
    if (i >= my_tiles || tok >= keys) return -1;
    const int p = __ldg(table + (tok >> a.c.log_page));
    if (p < 0 || p >= a.c.num_pages) {
      bad_page = true;
      return -1;
    }
    return p;
  };
  // Unit u: keys (even) or values (odd) of tile u / 2 into slot u % kSlots.
  auto issue = [&](int u) {
    const int i = u >> 1;
    if (i < my_tiles) {
      const uint32_t dst = ring + (u % kSlots) * SM::kSlotBytes;
      const int tok0 = (t_begin + warp + i * kWarps) * kTileTokens;
      const int gr = (u & 1) ? t : g >> 1;
      const int page = page_of(i, gr);
      const int in_page = (tok0 + 16 * gr) & page_mask;
      const int64_t head = (static_cast<int64_t>(page < 0 ? 0 : page) * a.c.heads + h)
                           << a.c.log_page;
      if (u & 1) {
        const uint8_t* src = a.c.v + head * D + in_page + (static_cast<int64_t>(g) << a.c.log_page);
#pragma unroll
        for (int j = 0; j < kDTiles; ++j)
          cp_async16(dst + j * 512, src + (static_cast<int64_t>(8 * j) << a.c.log_page), page >= 0);
      } else {
        const uint8_t* src = a.c.k + (head + in_page + (g & 1)) * D + 16 * t;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            cp_async16(dst + (j * kChunks + c) * 512, src + 2 * j * D + 64 * c, page >= 0);
      }
    }
    cp_commit();
  };

  float o[kDTiles][4];
#pragma unroll
  for (int j = 0; j < kDTiles; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float v_ref = 0.f;  // largest value scale so far: o is in its units

#pragma unroll
  for (int u = 0; u < kSlots; ++u) issue(u);
  auto scales_of = [&](int i, float& sk, float& sv) {
    const int p = page_of(i, t);
    const int64_t at = static_cast<int64_t>(p < 0 ? 0 : p) * a.c.heads + h;
    sk = p < 0 ? 0.f : __ldg(a.c.ks + at);
    sv = p < 0 ? 0.f : __ldg(a.c.vs + at);
  };
  float sk_next, sv_next;
  scales_of(0, sk_next, sv_next);

  for (int i = 0; i < my_tiles; ++i) {
    const int tok0 = (t_begin + warp + i * kWarps) * kTileTokens;
    const float sk = sk_next, sv = sv_next;
    scales_of(i + 1, sk_next, sv_next);
    // ---- scores ----
    cp_wait<kSlots - 1>();
    float sc[8][4];
    {
      const uint32_t src = ring + ((2 * i) % kSlots) * SM::kSlotBytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[j][x] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint4 w = lds128(src + (j * kChunks + c) * 512);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t b0, b1;
            codes_to_f16<FMT>(ww[x], b0, b1);
            mma_f16(sc[j], qa[4 * c + x], b0, b1);
          }
        }
      }
    }
    issue(2 * i + kSlots);
    // ---- online softmax ----
    const float f[2] = {q_back[0] * sk, q_back[1] * sk};
    const bool all_seen = tok0 + kTileTokens - 1 <= first_limit && live_rows == 16;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = sc[j][x] * f[x >> 1];
        // Columns of this lane: tokens 16 t + 2 j + 0, 1.  A masked column
        // may hold anything, so it is replaced, not added to.
        if (!all_seen && tok0 + 16 * t + 2 * j + (x & 1) > limit[x >> 1]) v = -INFINITY;
        sc[j][x] = v;
        top[x >> 1] = fmaxf(top[x >> 1], v);
      }
    float keep[2];
    float v_new = fmaxf(v_ref, quad_max(sv));
    const float v_old = v_new > 0.f ? v_ref / v_new : 0.f;
    const float v_rel = v_new > 0.f ? sv / v_new : 0.f;
    v_ref = v_new;
    float base[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float mn = fmaxf(m[r], quad_max(top[r]));
      const float at = mn == -INFINITY ? 0.f : mn;
      keep[r] = exp2f(m[r] - at);
      m[r] = mn;
      base[r] = at - kShift;
      l[r] *= keep[r];
      keep[r] *= v_old;
    }
    uint32_t pa[4][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float p0 = exp2f(sc[j][2 * r] - base[r]), p1 = exp2f(sc[j][2 * r + 1] - base[r]);
        l[r] += p0 + p1;
        const __half2 p = __floats2half2_rn(p0 * v_rel, p1 * v_rel);
        pa[j >> 1][2 * (j & 1) + r] = *reinterpret_cast<const uint32_t*>(&p);
      }
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[j][x] *= keep[x >> 1];
    // ---- outputs ----
    cp_wait<kSlots - 1>();
    {
      const uint32_t src = ring + ((2 * i + 1) % kSlots) * SM::kSlotBytes;
      // Bytes behind the last key may hold anything, NaN codes included.
      const int held = keys - tok0 - 16 * t;  // tokens of this lane's 16 that count
      const bool ragged = tok0 + kTileTokens > keys;
#pragma unroll
      for (int j = 0; j < kDTiles; ++j) {
        const uint4 w = lds128(src + j * 512);
        uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (ragged) {
            const int nb = held - 4 * x;  // bytes of this word that count
            ww[x] &= nb >= 4 ? 0xFFFFFFFFu : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
          }
          uint32_t b0, b1;
          codes_to_f16<FMT>(ww[x], b0, b1);
          mma_f16(o[j], pa[x], b0, b1);
        }
      }
    }
    issue(2 * i + 1 + kSlots);
  }
  cp_wait<0>();
  if (bad_page) record_error(err, kErrBadIndex, kKernelIdAttn);

  // ---- join the warps of the CTA ----
  l[0] = quad_sum(l[0]);
  l[1] = quad_sum(l[1]);
  __syncthreads();  // every ring is idle
  float* wo = reinterpret_cast<float*>(smem) + warp * (16 * D);  // [row][channel]
  float* wm = reinterpret_cast<float*>(smem) + kWarps * 16 * D;  // [warp][16] maxima, then sums
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (t == 0) {
      wm[warp * 16 + g + 8 * r] = m[r];
      wm[(kWarps + warp) * 16 + g + 8 * r] = l[r];
    }
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
      *reinterpret_cast<float2*>(wo + (g + 8 * r) * D + 8 * j + 2 * t) =
          make_float2(o[j][2 * r] * v_ref, o[j][2 * r + 1] * v_ref);
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem + SM::part);
  float* part_ml = reinterpret_cast<float*>(smem + SM::ml);
  const float* all_o = reinterpret_cast<const float*>(smem);
  auto store = [&](int row, int d, float4 v) {
    const int r = r0 + row;
    __nv_bfloat16* dst = a.out +
                         (static_cast<int64_t>(s.row0 + r / a.group) * a.q_heads + h * a.group +
                          r % a.group) * D + d;
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                                *reinterpret_cast<const uint32_t*>(&y));
  };
  for (int e = threadIdx.x; e < live_rows * (D / 4); e += kAttnThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wm[w * 16 + row]);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(wm[w * 16 + row] - at);
      sum += f * wm[(kWarps + w) * 16 + row];
      const float4 x = *reinterpret_cast<const float4*>(all_o + (w * 16 + row) * D + d);
      v.x += f * x.x;
      v.y += f * x.y;
      v.z += f * x.z;
      v.w += f * x.w;
    }
    if (ks == 1) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      store(row, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    } else {
      *reinterpret_cast<float4*>(part + row * D + d) = v;
      if (d == 0) {
        part_ml[row] = mx;
        part_ml[16 + row] = sum;
      }
    }
  }
  if (ks == 1) return;

  // ---- join the CTAs of the cluster, each a share of the rows' channels ----
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int total = live_rows * (D / 4);
  const int e1 = (rank + 1) * total / ks;
  for (int e = rank * total / ks + threadIdx.x; e < e1; e += kAttnThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float mx = -INFINITY;
    for (int p = 0; p < ks; ++p) mx = fmaxf(mx, cluster.map_shared_rank(part_ml, p)[row]);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < ks; ++p) {
      const float* ml = cluster.map_shared_rank(part_ml, p);
      const float f = exp2f(ml[row] - at);
      sum += f * ml[16 + row];
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, p) + row * D + d);
      v.x += f * x.x;
      v.y += f * x.y;
      v.z += f * x.z;
      v.w += f * x.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    store(row, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
  }
  cluster.sync();  // peers keep their partials until every reader is done
}

template <int FMT, int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream, int num_sms, unsigned* err) {
  using SM = AttnSmem<D>;
  constexpr auto kern = kv8_attention_rows_kernel<FMT, D>;
  static unsigned long long done = 0;  // bit d: device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELEASE);
  }
  const int64_t probs = static_cast<int64_t>(a.bt.batch) * a.c.heads * a.row_tiles;
  // A problem's tiles are split over a cluster while the CTAs still fit the
  // GPU at once; the table's width bounds the lengths.
  const int64_t tiles = ((static_cast<int64_t>(a.bt.max_pages) << a.c.log_page) + kTileTokens - 1) /
                        kTileTokens;
  int ks = 1;
  while (ks < 8 && ks * 2 * kWarps <= tiles && probs * ks * 2 <= 2 * num_sms) ks *= 2;
  if (probs * ks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(probs * ks), 1, 1);
  cfg.blockDim = dim3(kAttnThreads, 1, 1);
  cfg.dynamicSmemBytes = SM::bytes;
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
  return cudaLaunchKernelEx(&cfg, kern, a, err);
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8Cache& c, const Kv8Batch& bt, const void* q, int64_t ldq,
                                 int q_heads, int D, int fmt, float scale, void* out,
                                 cudaStream_t stream, int num_sms, unsigned* err) {
  AttnArgs a;
  a.c = c;
  a.bt = bt;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ldq = ldq;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.row_tiles = static_cast<int>((static_cast<int64_t>(bt.max_new) * a.group + 15) / 16);
  a.scale_log2 = scale * 1.4426950408889634f;
  if (fmt == kKvInt8)
    return D == 64 ? launch_rows<kKvInt8, 64>(a, stream, num_sms, err)
                   : launch_rows<kKvInt8, 128>(a, stream, num_sms, err);
  return D == 64 ? launch_rows<kKvE4m3, 64>(a, stream, num_sms, err)
                 : launch_rows<kKvE4m3, 128>(a, stream, num_sms, err);
}

}  // namespace w4
