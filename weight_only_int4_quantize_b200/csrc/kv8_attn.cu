// Causal attention over the 8-bit paged cache (layout: kv8.cuh), rows kernel:
// decode and short runs of new tokens.
//
//   o_i = sum_j p_ij v_j,  p_i = softmax over j <= len - n + i of
//   scale * q_i . k_j,  k_j = ks[page j] * code,  v_j = vs[page j] * code
//
// Rows: the query heads that share a kv head and the new tokens of a
// sequence are the rows of one problem (row = token * group + head of the
// group), taken 8 or 16 at a time (NT = 1, 2) as the N of mma.m16n8k16: the
// products are S^T = K Q^T and O^T = V^T P^T, so the cache is the A operand
// and no multiply is spent on rows that a small group does not have.
//
// Work split: a thread-block cluster of `ks` CTAs owns one (sequence, kv
// head, row tile); its warps take tiles of 64 tokens in turn.  Each warp runs
// its own online softmax; the partial results are joined in a fixed order,
// first over a CTA's warps and then, through distributed shared memory, over
// the cluster: no workspace, and the same bits on every run.
//
// A warp streams its tiles through its own ring of shared memory: each lane
// (g = lane / 4, t = lane % 4) copies (cp.async, 16 bytes) exactly the bytes
// of its own operand fragments and reads only those back, so the ring needs
// no barrier.
//   keys:   row r of score tile i (16 tokens) is token 16 (r / 2) + 4 i + r % 2
//           of the 64, rows r >= 8 token 16 (r / 2 - 4) + 4 i + 2 + r % 2, and
//           k-step s covers channels 64 (s / 4) + 16 t + 4 (s % 4) + 0..3 of
//           lane quad t (the queries are loaded in that order), so a lane's
//           fragments are 16 contiguous bytes of key rows;
//   values: the probabilities of score tile i, transposed 8 x 8 at a time
//           (movmatrix), are the B fragments of k-step i; with that order of
//           rows a lane's value fragments are the tokens 16 t .. 16 t + 15,
//           16 contiguous bytes of a value row.
// A lane's score rows all lie in the 16 tokens of granule g / 2, so in one
// page whatever the page size (>= 16): a key scale and a value scale per lane
// and tile suffice.
//
// Numerics: codes are exact in fp16.  Each query row is scaled by a power of
// two that brings its largest magnitude into [128, 256) (exact for channels
// within 2^21 of it) and the scores, in fp32, are scaled back with the key
// scale.  Probabilities are weighted by value scale / largest value scale so
// far and rounded to fp16 with a shift of 2^14 (the largest is 2^14, full
// precision down to 2^-28 of it); sums and outputs are fp32.
#include <cooperative_groups.h>

#include <type_traits>

#include "kv8.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace cg = cooperative_groups;

namespace {

constexpr int kTileTokens = 64;
constexpr float kShift = 14.f;  // probabilities are kept times 2^14
constexpr unsigned kKernelIdAttn = 32;
constexpr int kMaxSplit = 16;  // CTAs per cluster

// A launch's shape: 8 NT rows, W warps per CTA.  16 rows need some 210
// registers, so two CTAs of four warps share an SM, with three ring slots
// (alternately key and value tiles) per warp; 8 rows need 150, so three CTAs
// do, or one of twelve warps where few long problems leave one CTA per SM (a
// warp alone on its scheduler waits for its own instructions), with two slots.
template <int D, int NT, int W>
struct AttnShape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kCtasPerSm = W > 4 ? 1 : NT == 1 ? 3 : 2;
  static constexpr int kSlots = NT == 1 ? 2 : 3;
  static constexpr int kSlotBytes = kTileTokens * D;
  static constexpr int kRing = W * kSlots * kSlotBytes;
  // Joined partial of the CTA (read by the cluster's peers), apart from the
  // ring: rows of D floats, then maxima, sums and the unit of the outputs.
  static constexpr int part = kRing;
  static constexpr int ml = part + 8 * NT * D * 4;
  static constexpr int bytes = ml + (2 * 16 + 4) * 4;
  // The warps' partials take the ring's place.
  static_assert(W * (8 * NT * ((D + 4) * 4 + 8) + 4) <= kRing, "partials fit the ring");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Over the eight lanes of one t (the rows of a score tile).
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
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

template <int FMT, int D, int NT, int W>
__global__ void __launch_bounds__(32 * W, AttnShape<D, NT, W>::kCtasPerSm)
    kv8_attention_rows_kernel(const AttnArgs a, unsigned* err) {
  using SM = AttnShape<D, NT, W>;
  constexpr int kWarps = W, kAttnThreads = 32 * W, kSlots = SM::kSlots;
  constexpr int kRows = 8 * NT;
  constexpr int kSteps = D / 16;    // k-steps of the score product
  constexpr int kChunks = D / 64;   // 16-byte pieces of a key row per lane
  constexpr int kDTiles = D / 16;   // 16-channel tiles of the output
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
  pdl_launch_dependents();
  pdl_wait();
  const int32_t* table = a.bt.table + static_cast<int64_t>(b) * a.bt.max_pages;
  // Without a split a warp's first two tiles do not depend on the length:
  // their page ids are read along with it (and used if it reaches there).
  int first[2] = {-1, -1};
  if (ks == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = ((warp + i * kWarps) * kTileTokens + 16 * (g >> 1)) >> a.c.log_page;
      if (at < a.bt.max_pages) first[i] = __ldg(table + at);
    }
  }
  const Kv8Seq s = kv8_sequence(a.bt, b, a.c.log_page);
  if (s.bad && threadIdx.x == 0 && h == 0 && rt == 0 && rank == 0)
    record_error(err, kErrBadIndex, kKernelIdAttn);
  const int n_rows = s.n * a.group;
  const int r0 = rt * kRows;
  if (r0 >= n_rows) return;  // the whole cluster
  const int live_rows = n_rows - r0 < kRows ? n_rows - r0 : kRows;

  // Tiles of this CTA: the cluster's tiles in contiguous shares.
  const int keys = s.len - s.n + (r0 + live_rows - 1) / a.group + 1;  // <= 0: nothing is seen
  const int first_limit = s.len - s.n + r0 / a.group;
  const int tiles = keys > 0 ? (keys + kTileTokens - 1) / kTileTokens : 0;
  const int t_begin = static_cast<int>(static_cast<int64_t>(rank) * tiles / ks);
  const int t_end = static_cast<int>(static_cast<int64_t>(rank + 1) * tiles / ks);
  const int my_tiles = t_end - t_begin > warp ? (t_end - t_begin - warp + kWarps - 1) / kWarps : 0;

  const int page_mask = (1 << a.c.log_page) - 1;
  const uint32_t ring = smem_u32(smem) + warp * (kSlots * SM::kSlotBytes) + lane * 16;
  bool bad_page = false;
  // The page that holds the lane's granule (16 tokens) g / 2 of tile i, -1 if
  // none does.  The value granule t of a lane is that of the lanes g = 2 t.
  auto page_of = [&](int i, bool read = true, int p = 0) {
    const int tok = (t_begin + warp + i * kWarps) * kTileTokens + 16 * (g >> 1);
    if (i >= my_tiles || tok >= keys) return -1;
    if (read) p = __ldg(table + (tok >> a.c.log_page));
    if (p < 0 || p >= a.c.num_pages) {
      bad_page = true;
      return -1;
    }
    return p;
  };
  const int64_t page_bytes = (static_cast<int64_t>(a.c.heads) << a.c.log_page) * D;
  const int64_t head_bytes = (static_cast<int64_t>(h) << a.c.log_page) * D;
  const uint8_t* k_lane = a.c.k + head_bytes + (g & 1) * D + 16 * t;
  const uint8_t* v_lane = a.c.v + head_bytes + (static_cast<int64_t>(g) << a.c.log_page);
  const int64_t v_step = static_cast<int64_t>(8) << a.c.log_page;
  // Unit u: keys (even) or values (odd) of tile u / 2, whose granule lies in
  // `page`, into slot u % kSlots.
  auto issue_k = [&](int i, int slot, int page) {
    if (i < my_tiles) {
      const uint32_t dst = ring + slot * SM::kSlotBytes;
      const int tok = (t_begin + warp + i * kWarps) * kTileTokens + 16 * (g >> 1);
      // tokens g % 2, g % 2 + 2, + 4, ... of the granule
      const uint8_t* src = k_lane + (page < 0 ? 0 : page) * page_bytes + (tok & page_mask) * D;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          kv8_copy16(dst + (j * kChunks + c) * 512, src + 2 * j * D + 64 * c, page >= 0);
    }
    kv8_copy_commit();
  };
  auto issue_v = [&](int i, int slot, int k_page) {
    const int page = __shfl_sync(0xffffffffu, k_page, 8 * t);
    if (i < my_tiles) {
      const uint32_t dst = ring + slot * SM::kSlotBytes;
      const int tok = (t_begin + warp + i * kWarps) * kTileTokens + 16 * t;
      // channels g, g + 8, g + 16, ... of the lane's 16 tokens
      const uint8_t* src = v_lane + (page < 0 ? 0 : page) * page_bytes + (tok & page_mask);
#pragma unroll
      for (int j = 0; j < 2 * kDTiles; ++j, src += v_step)
        kv8_copy16(dst + j * 512, src, page >= 0);
    }
    kv8_copy_commit();
  };
  // With two slots a tile's keys and values are on their way while it is
  // waited for; with three also the next tile's keys.
  int page = page_of(0, ks > 1, first[0]), page_next = page_of(1, ks > 1, first[1]);
  issue_k(0, 0, page);
  issue_v(0, 1, page);
  if (kSlots > 2) issue_k(1, 2, page_next);
  auto scales_of = [&](int p, float& sk, float& sv) {
    const int64_t at = static_cast<int64_t>(p < 0 ? 0 : p) * a.c.heads + h;
    // Not through the non-coherent path: this kernel may be resident while an
    // append writes these scales and reads their neighbours.
    sk = p < 0 ? 0.f : a.c.ks[at];
    sv = p < 0 ? 0.f : a.c.vs[at];
  };
  float sk_next, sv_next;
  scales_of(page, sk_next, sv_next);
  int slot_k = 0, slot_v = 1;  // of this tile

  // Query fragments: row 8 nt + g, scaled by a power of two.
  uint32_t qb[NT][kSteps][2];
  float q_back[NT][2];  // of rows 8 nt + 2 t, + 1: undoes the scaling, times the softmax scale
  int limit[NT][2];     // the last position that each of these rows sees
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 8 * nt + g;
    const bool live = r < n_rows;
    const int tok = live ? r / a.group : 0;
    const __nv_bfloat16* qr = a.q + static_cast<int64_t>(s.row0 + tok) * a.ldq +
                              (h * a.group + (live ? r - tok * a.group : 0)) * D;
    uint32_t raw[kSteps][2];
    uint32_t big = 0;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(
                                 qr + 64 * (st / 4) + 16 * t + 4 * (st % 4)))
                           : make_uint2(0, 0);
      raw[st][0] = v.x;
      raw[st][1] = v.y;
      big = __vmaxu2(big, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
    }
    big = max(big & 0xFFFFu, big >> 16);
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // Largest magnitude in [2^e, 2^(e+1)); scaled by 2^(7 - e).
    const int e = static_cast<int>(big >> 7) - 127;
    const float up = __int_as_float((min(7 - e, 126) + 127) << 23);
    const float back = __int_as_float((max(e - 7, -126) + 127) << 23) * a.scale_log2;
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const __half2 x = __floats2half2_rn(__uint_as_float(raw[st][w] << 16) * up,
                                            __uint_as_float(raw[st][w] & 0xFFFF0000u) * up);
        qb[nt][st][w] = *reinterpret_cast<const uint32_t*>(&x);
      }
    const int lim = live ? s.len - s.n + tok : -1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {  // row 2 t + x lies with the lanes g = 2 t + x
      q_back[nt][x] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + x));
      limit[nt][x] = __shfl_sync(0xffffffffu, lim, 4 * (2 * t + x));
    }
  }

  float o[NT][kDTiles][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < kDTiles; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[nt][j][x] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }
  // Largest value scale so far, which o is in units of; not under 2^-126, so
  // that its reciprocal is a number.
  float v_ref = 0x1p-126f;

  for (int i = 0; i < my_tiles; ++i) {
    const int tok0 = (t_begin + warp + i * kWarps) * kTileTokens;
    const float sk = sk_next, sv = sv_next;
    page = page_next;  // of tile i + 1
    page_next = page_of(i + 2);
    scales_of(page, sk_next, sv_next);
    // ---- scores: sc[nt][i4][x], tokens 16 (g/2) + 4 i4 + g%2 (+ 2 for x >= 2)
    // of rows 2 t + x % 2 ----
    kv8_copy_wait<kSlots - 1>();
    float sc[NT][4][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[nt][j][x] = 0.f;
    {
      const uint32_t src = ring + slot_k * SM::kSlotBytes;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t kw[8][4];  // the lane's eight tokens
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 w = kv8_lds128(src + (j * kChunks + c) * 512);
          kw[j][0] = w.x, kw[j][1] = w.y, kw[j][2] = w.z, kw[j][3] = w.w;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t f[4];
            kv8_codes_to_f16<FMT>(kw[2 * j][x], f[0], f[2]);
            kv8_codes_to_f16<FMT>(kw[2 * j + 1][x], f[1], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(sc[nt][j], f, qb[nt][4 * c + x][0], qb[nt][4 * c + x][1]);
          }
      }
    }
    if (kSlots == 2) issue_k(i + 1, slot_k, page); else issue_v(i + 1, slot_k, page);
    // ---- online softmax ----
    const bool all_seen = tok0 + kTileTokens - 1 <= first_limit;
    const float v_new = fmaxf(v_ref, column_max(sv));
    const float v_inv = __frcp_rn(v_new);
    const float v_old = v_ref * v_inv, v_rel = sv * v_inv;
    v_ref = v_new;
    uint32_t pb[NT][4][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float keep[2], base[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float f = q_back[nt][x] * sk;
        const int seen = limit[nt][x] - (tok0 + 16 * (g >> 1) + (g & 1));
        float top = -INFINITY;
        auto scale_scores = [&](auto masks) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              float v = sc[nt][j][2 * hi + x] * f;
              // A masked score may be anything, so it is replaced, not added to.
              if (decltype(masks)::value && 4 * j + 2 * hi > seen) v = -INFINITY;
              sc[nt][j][2 * hi + x] = v;
              top = fmaxf(top, v);
            }
        };
        if (all_seen) scale_scores(std::false_type{}); else scale_scores(std::true_type{});
        const float mn = fmaxf(m[nt][x], column_max(top));
        const float at = mn == -INFINITY ? 0.f : mn;
        keep[x] = ex2(m[nt][x] - at);
        m[nt][x] = mn;
        base[x] = at - kShift;
        l[nt][x] *= keep[x];
        keep[x] *= v_old;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const float p0 = ex2(sc[nt][j][2 * hi] - base[0]);
          const float p1 = ex2(sc[nt][j][2 * hi + 1] - base[1]);
          l[nt][0] += p0;
          l[nt][1] += p1;
          const __half2 p = __floats2half2_rn(p0 * v_rel, p1 * v_rel);
          pb[nt][j][hi] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p));
        }
#pragma unroll
      for (int j = 0; j < kDTiles; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nt][j][x] *= keep[x & 1];
    }
    // ---- outputs ----
    kv8_copy_wait<kSlots - 1>();
    {
      const uint32_t src = ring + slot_v * SM::kSlotBytes;
      // Bytes behind the last key may hold anything, NaN codes included.
      const int held = keys - tok0 - 16 * t;  // tokens of this lane's 16 that count
      const bool ragged = tok0 + kTileTokens > keys;
#pragma unroll
      for (int j0 = 0; j0 < kDTiles; j0 += 4) {
        uint32_t vw[8][4];  // four output tiles: channels g and g + 8 of each
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 w = kv8_lds128(src + (2 * j0 + j) * 512);
          vw[j][0] = w.x, vw[j][1] = w.y, vw[j][2] = w.z, vw[j][3] = w.w;
        }
        if (ragged) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int nb = held - 4 * x;  // bytes of this word that count
            const uint32_t mask = nb >= 4 ? 0xFFFFFFFFu : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
#pragma unroll
            for (int j = 0; j < 8; ++j) vw[j][x] &= mask;
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t f[4];
            kv8_codes_to_f16<FMT>(vw[2 * j][x], f[0], f[2]);
            kv8_codes_to_f16<FMT>(vw[2 * j + 1][x], f[1], f[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(o[nt][j0 + j], f, pb[nt][x][0], pb[nt][x][1]);
          }
        }
      }
    }
    if (kSlots == 2) {
      issue_v(i + 1, slot_v, page);
    } else {
      issue_k(i + 2, slot_v, page_next);
      // Unit u lies in slot u % 3.
      const int was_k = slot_k;
      slot_k = 3 - slot_k - slot_v;
      slot_v = was_k;
    }
  }
  kv8_copy_wait<0>();
  if (bad_page) record_error(err, kErrBadIndex, kKernelIdAttn);

  // ---- join the warps of the CTA ----
  __syncthreads();  // every ring is idle
  constexpr int kLd = D + 4;  // floats between rows
  float* wo = reinterpret_cast<float*>(smem) + warp * (kRows * kLd);  // [row][channel]
  float* wm = reinterpret_cast<float*>(smem) + kWarps * kRows * kLd;  // [warp][row] maxima, sums
  float* wv = wm + 2 * kWarps * kRows;  // [warp] units (v_ref)
  // Outputs stay in units of the largest v_ref until they have been divided by
  // the sum: before, they carry the probabilities' 2^14 and the number of keys,
  // and in units of 1 they could pass binary32's range where the result does not.
  if (lane == 0) wv[warp] = v_ref;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 8 * nt + 2 * t + x;
      const float sum = column_sum(l[nt][x]);
      if (g == 0) {
        wm[warp * kRows + row] = m[nt][x];
        wm[(kWarps + warp) * kRows + row] = sum;
      }
#pragma unroll
      for (int j = 0; j < kDTiles; ++j) {
        wo[row * kLd + 16 * j + g] = o[nt][j][x];
        wo[row * kLd + 16 * j + 8 + g] = o[nt][j][2 + x];
      }
    }
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem + SM::part);
  float* part_ml = reinterpret_cast<float*>(smem + SM::ml);
  const float* all_o = reinterpret_cast<const float*>(smem);
  float unit = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) unit = fmaxf(unit, wv[w]);
  const float per_unit = __frcp_rn(unit);
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
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, wm[w * kRows + row]);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      float f = ex2(wm[w * kRows + row] - at);
      sum += f * wm[(kWarps + w) * kRows + row];
      f *= wv[w] * per_unit;
      const float4 x = *reinterpret_cast<const float4*>(all_o + (w * kRows + row) * kLd + d);
      v.x += f * x.x;
      v.y += f * x.y;
      v.z += f * x.z;
      v.w += f * x.w;
    }
    if (ks == 1) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      store(row, d, make_float4(v.x * inv * unit, v.y * inv * unit, v.z * inv * unit,
                                v.w * inv * unit));
    } else {
      *reinterpret_cast<float4*>(part + row * D + d) = v;
      if (d == 0) {
        part_ml[row] = mx;
        part_ml[16 + row] = sum;
        part_ml[32] = unit;
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
    for (int p = 0; p < ks; ++p) {
      const float* ml = cluster.map_shared_rank(part_ml, p);
      mx = fmaxf(mx, ml[row]);
      unit = fmaxf(unit, ml[32]);
    }
    const float per_unit = __frcp_rn(unit);
    const float at = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < ks; ++p) {
      const float* ml = cluster.map_shared_rank(part_ml, p);
      float f = ex2(ml[row] - at);
      sum += f * ml[16 + row];
      f *= ml[32] * per_unit;
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, p) + row * D + d);
      v.x += f * x.x;
      v.y += f * x.y;
      v.z += f * x.z;
      v.w += f * x.w;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    store(row, d, make_float4(v.x * inv * unit, v.y * inv * unit, v.z * inv * unit,
                              v.w * inv * unit));
  }
  cluster.sync();  // peers keep their partials until every reader is done
}

template <int FMT, int D, int NT, int W>
void set_cluster(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, int64_t ctas, int ks) {
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(AttnShape<D, NT, W>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = AttnShape<D, NT, W>::bytes;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
}

// Clusters of each size that the device holds at once (clusters do not pack
// its GPCs evenly: 148 SMs hold 15 clusters of 8 or 9 CTAs, 11 of 10 and 7 of
// 16 at one CTA per SM).  Asked for once per device; also where the kernel's
// attributes are set.
struct Fit {
  int clusters[kMaxSplit + 1];
};
template <int FMT, int D, int NT, int W>
cudaError_t clusters_at_once(Fit& fit) {
  constexpr auto kern = kv8_attention_rows_kernel<FMT, D, NT, W>;
  constexpr int kDevices = 64;
  static Fit known[kDevices];
  static int state[kDevices];  // 2: known (every thread that asks finds the same)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && __atomic_load_n(&state[dev], __ATOMIC_ACQUIRE) == 2) {
    fit = known[dev];
    return cudaSuccess;
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           AttnShape<D, NT, W>::bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  fit.clusters[0] = 0;
  for (int ks = 1; ks <= kMaxSplit && e == cudaSuccess; ++ks) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    set_cluster<FMT, D, NT, W>(cfg, attr, ks, ks);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&fit.clusters[ks], kern, &cfg);
  }
  if (e != cudaSuccess) return e;
  int none = 0;
  if (dev < kDevices && __atomic_compare_exchange_n(&state[dev], &none, 1, false,
                                                    __ATOMIC_ACQ_REL, __ATOMIC_RELAXED)) {
    known[dev] = fit;
    __atomic_store_n(&state[dev], 2, __ATOMIC_RELEASE);
  }
  return cudaSuccess;
}

// The split of K for W warps per CTA that takes the least time by a model in
// microseconds, fitted to launches of 8 ... 1024 problems of 5 ... 1024 tiles
// (within 25 %): waves x (start, join and per-tile rounds of a warp), a round
// taking longer the more warps share an SM and the more SMs are at work.
// 8 problems x 512 tiles: 16 x 4 warps 25.3 us, 8 x 12 25.5, 10 x 12 23.1;
// x 32 tiles: 8 x 4 7.8, 4 x 12 8.5; 256 problems x 64: 1 x 4 48, 2 x 4 42.
// Waves count in parts where an SM takes several CTAs (lengths differ, so
// they end at different times), in full where it takes one.
template <int NT, int W>
double best_split(const Fit& fit, int64_t probs, int64_t tiles, int num_sms, int& best) {
  double least = 0;
  best = 0;
  for (int ks = 1; ks <= kMaxSplit; ++ks) {
    if (ks > 1 && (ks - 1) * W >= tiles) break;
    if (fit.clusters[ks] < 1) continue;
    const int64_t at_once = probs < fit.clusters[ks] ? probs : fit.clusters[ks];
    const double per_sm = static_cast<double>(at_once * ks) / num_sms;
    double waves = static_cast<double>(probs) / fit.clusters[ks];
    if (W > 4) waves = static_cast<double>((probs + fit.clusters[ks] - 1) / fit.clusters[ks]);
    if (waves < 1) waves = 1;
    const double round = (NT == 1 ? 1. : 1.3) * (0.75 + 0.19 * W * (per_sm > 1 ? per_sm : 1) +
                                                 0.65 * (per_sm < 1 ? per_sm : 1));
    const double t = waves * ((ks == 1 ? 3. : 5.2 + 0.12 * ks) +
                              round * (static_cast<double>(tiles) / (ks * W) + 0.5));
    if (best == 0 || t < least) {
      least = t;
      best = ks;
    }
  }
  return least;
}

template <int FMT, int D, int NT, int W>
cudaError_t launch_shape(const AttnArgs& a, int ks, cudaStream_t stream, unsigned* err) {
  const int64_t probs = static_cast<int64_t>(a.bt.batch) * a.c.heads * a.row_tiles;
  if (ks < 1 || probs * ks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  set_cluster<FMT, D, NT, W>(cfg, attr[1], probs * ks, ks);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kv8_attention_rows_kernel<FMT, D, NT, W>, a, err);
}

template <int FMT, int D, int NT>
cudaError_t launch_rows(AttnArgs a, cudaStream_t stream, int num_sms, unsigned* err) {
  a.row_tiles = static_cast<int>((static_cast<int64_t>(a.bt.max_new) * a.group + 8 * NT - 1) /
                                 (8 * NT));
  const int64_t probs = static_cast<int64_t>(a.bt.batch) * a.c.heads * a.row_tiles;
  // The table's width bounds the lengths.
  const int64_t tiles = ((static_cast<int64_t>(a.bt.max_pages) << a.c.log_page) + kTileTokens - 1) /
                        kTileTokens;
  Fit fit;
  cudaError_t e = clusters_at_once<FMT, D, NT, 4>(fit);
  if (e != cudaSuccess) return e;
  int ks;
  const double four = best_split<NT, 4>(fit, probs, tiles, num_sms, ks);
  if constexpr (NT == 1) {
    e = clusters_at_once<FMT, D, NT, 12>(fit);
    if (e != cudaSuccess) return e;
    int ks12;
    if (best_split<NT, 12>(fit, probs, tiles, num_sms, ks12) < four && ks12 > 0)
      return launch_shape<FMT, D, NT, 12>(a, ks12, stream, err);
  }
  return launch_shape<FMT, D, NT, 4>(a, ks, stream, err);
}

}  // namespace

cudaError_t launch_kv8_attention(const Kv8Cache& c, const Kv8Batch& bt, const void* q, int64_t ldq,
                                 int q_heads, int D, int fmt, float scale, void* out,
                                 cudaStream_t stream, int num_sms, unsigned* err) {
  if (kv8_attention_prefers_tc(c, bt, q_heads / c.heads, num_sms))
    return launch_kv8_attention_tc(c, bt, q, ldq, q_heads, D, fmt, scale, out, stream, err);
  AttnArgs a;
  a.c = c;
  a.bt = bt;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ldq = ldq;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.row_tiles = 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  const bool one = static_cast<int64_t>(bt.max_new) * a.group <= 8;
  if (fmt == kKvInt8) {
    if (D == 64)
      return one ? launch_rows<kKvInt8, 64, 1>(a, stream, num_sms, err)
                 : launch_rows<kKvInt8, 64, 2>(a, stream, num_sms, err);
    return one ? launch_rows<kKvInt8, 128, 1>(a, stream, num_sms, err)
               : launch_rows<kKvInt8, 128, 2>(a, stream, num_sms, err);
  }
  if (D == 64)
    return one ? launch_rows<kKvE4m3, 64, 1>(a, stream, num_sms, err)
               : launch_rows<kKvE4m3, 64, 2>(a, stream, num_sms, err);
  return one ? launch_rows<kKvE4m3, 128, 1>(a, stream, num_sms, err)
             : launch_rows<kKvE4m3, 128, 2>(a, stream, num_sms, err);
}

}  // namespace w4
