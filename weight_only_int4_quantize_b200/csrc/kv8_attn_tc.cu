// Causal attention over the 8-bit paged cache (layout: kv8.cuh), tcgen05
// kernel: long runs of new tokens (prompts and their chunks).
//
// One CTA owns 256 rows (row = token * group + head of the group), two tiles
// of 128, of one sequence and kv head and walks the keys in tiles of 64:
//
//   S = Q K^T            (fp16 operands, fp32 in TMEM)
//   P = exp2(f S - m)    (fp16 in TMEM, weighted by the value scales)
//   O += P V             (A operand P from TMEM, fp32 accumulator in TMEM)
//
// Warp roles: 0..3 and 4..7 softmax of the two row tiles (a thread owns a
// row), 8 and 9 MMA issue for one row tile each, 10..13 dequantization: a
// lane copies (cp.async) the pieces of codes that it will turn three tiles
// ahead, turns this tile's into fp16 and writes the swizzled operand tiles, so
// codes cross L2 once per 256 rows.
//
// Per row tile and 64 keys (D = 128) the tensor pipe needs 512 cycles (640
// with the shared-memory reads of the score product) and the exponential unit
// 512; what has to be kept out of the way is latency.  Scores have two
// buffers, and P takes the place of the scores that it was made of, so the
// scores of the next tile lie ready while a tile's exponentials run and a row
// tile's softmax never waits for its outputs; each row tile has its own
// issuing warp, so one does not wait for the other's softmax.
// 2 x 2048 tokens over up to 8192 keys, 16 / 8 heads: 128 rows per CTA and
// two CTAs per SM 371 us; 256 rows, one issuing warp, codes fetched into
// registers one tile ahead 340 us; an issuing warp per row tile and copies
// three tiles ahead 260 us; two S buffers with P in place 252 us, now 248, 0.6
// PFLOP/s (27 % of the tensor pipe).  What is left is the softmax arithmetic of eight
// warps, two per scheduler: 128-key tiles took 353 us, 128 us without that
// arithmetic; 16 softmax warps of half a row each 381 us.
//
// Numerics as in the rows kernel (kv8_attn.cu): codes are exact in fp16; a
// query row is scaled by a power of two; key scales (one per 16 keys at the
// finest) multiply the fp32 scores; value scales weight the probabilities
// relative to a running reference v_ref.  The running maximum that O is kept
// relative to is moved only when a row's maximum has grown by more than 2^5,
// and v_ref only when a value scale exceeds twice it, so O is rescaled in TMEM
// rarely; P is at most 2^9 * 2^5 * 2 = 2^15 (fp16), full precision from 2^-14.
#include <cuda_fp16.h>

#include <type_traits>

#include "kv8.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace {

constexpr int kTcThreads = 448;
constexpr int kTcRows = 128;         // rows of one MMA; two such tiles per CTA
constexpr int kTcStages = 3;         // key and value tiles in shared memory
constexpr int kTcAhead = 3;          // tiles of codes on their way
constexpr int kKeys = 64;            // keys of a tile
constexpr float kTcShift = 9.f;      // probabilities are kept times 2^9
constexpr float kTcGrow = 5.f;       // the maximum moves once a row's has grown by 2^5
constexpr unsigned kKernelIdAttnTc = 64;

template <int D>
struct TcSmem {
  static constexpr uint32_t kQ = kTcRows * D * 2;  // D / 64 tiles of 128 rows x 128 bytes
  static constexpr uint32_t kK = kKeys * D * 2;    // D / 64 tiles of 64 rows x 128 bytes
  static constexpr uint32_t kV = D * kKeys * 2;    // D rows x 128 bytes
  static constexpr uint32_t k = 2 * kQ;
  static constexpr uint32_t v = k + kTcStages * kK;
  static constexpr uint32_t codes = v + kTcStages * kV;  // keys, values in turn
  static constexpr uint32_t kCodes = kKeys * D;
  static constexpr uint32_t bars = codes + 2 * kTcAhead * kCodes;
  static constexpr uint32_t misc = bars + (14 + 4 * kTcStages) * 8;
  static constexpr size_t bytes = misc + 32 + 1024;
};

// TMEM columns: O of both row tiles, two S each (P, two fp16 per column, in
// the first half of the S it replaces).
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemAll = 512;

__device__ __forceinline__ void umma_f16_ta(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// Two fp32 operations at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ bool elect_lane() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
               : "=r"(ok));
  return ok != 0;
}

struct TcArgs {
  Kv8Cache c;
  Kv8Batch bt;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t ldq;
  int q_heads, group, row_tiles;
  float scale_log2;  // softmax scale * log2(e)
};

template <int FMT, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    kv8_attention_tc_kernel(const TcArgs a, unsigned* err) {
  using SM = TcSmem<D>;
  constexpr int kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw_addr);
  const uint32_t bar = base + SM::bars;
  // One of each per row tile.
  auto q_full = [&](int t) { return bar + 8u * t; };
  // S and P have a barrier per buffer: a softmax warp may be a key tile ahead
  // of another, and its arrival must not count for the slower one's tile.
  auto s_full = [&](int t, int buf) { return bar + 16u + 8u * (2 * t + buf); };
  auto p_full = [&](int t, int buf) { return bar + 48u + 8u * (2 * t + buf); };
  auto pv_done = [&](int t) { return bar + 80u + 8u * t; };
  auto done_bar = [&](int t) { return bar + 96u + 8u * t; };
  auto k_full = [&](int s) { return bar + 112u + 8u * s; };
  auto k_empty = [&](int s) { return bar + 112u + 8u * (kTcStages + s); };
  auto v_full = [&](int s) { return bar + 112u + 8u * (2 * kTcStages + s); };
  auto v_empty = [&](int s) { return bar + 112u + 8u * (3 * kTcStages + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + SM::misc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + SM::misc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Row tiles from the last to the first: later ones see more keys.
  const int rt = a.row_tiles - 1 - static_cast<int>(blockIdx.x);
  const int h = blockIdx.y % a.c.heads, b = blockIdx.y / a.c.heads;

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 4);
      mbar_init(s_full(t, 0), 1);
      mbar_init(s_full(t, 1), 1);
      mbar_init(p_full(t, 0), 4);
      mbar_init(p_full(t, 1), 4);
      mbar_init(pv_done(t), 1);
      mbar_init(done_bar(t), 1);
    }
    for (int s = 0; s < kTcStages; ++s) {
      mbar_init(k_full(s), 4);
      mbar_init(k_empty(s), 2);  // both issuing warps
      mbar_init(v_full(s), 4);
      mbar_init(v_empty(s), 2);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), kTmemAll);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Not before this CTA holds its TMEM: a dependent kernel that allocated
  // first would wait for this one while it waits for its TMEM.
  pdl_launch_dependents();
  pdl_wait();

  const Kv8Seq s = kv8_sequence(a.bt, b, a.c.log_page);
  if (s.bad && threadIdx.x == 0 && h == 0 && rt == 0) record_error(err, kErrBadIndex, kKernelIdAttnTc);
  const int n_rows = s.n * a.group;
  // Rows, keys seen (by the last row) and key tiles of each row tile; the
  // second's rows are later tokens, so it has at least as many key tiles
  // unless it has no rows.
  auto rows_of = [&](int t) {
    const int left = n_rows - (2 * rt + t) * kTcRows;
    return left < 0 ? 0 : left < kTcRows ? left : kTcRows;
  };
  auto keys_of = [&](int t) {
    const int n = rows_of(t);
    const int k = n > 0 ? s.len - s.n + ((2 * rt + t) * kTcRows + n - 1) / a.group + 1 : 0;
    return k > 0 ? k : 0;
  };
  const int keys0 = keys_of(0), keys1 = keys_of(1);
  const int keys = keys0 > keys1 ? keys0 : keys1;
  const int tiles0 = (keys0 + kKeys - 1) / kKeys, tiles1 = (keys1 + kKeys - 1) / kKeys;
  const int tiles = (keys + kKeys - 1) / kKeys;
  const int32_t* table = a.bt.table + static_cast<int64_t>(b) * a.bt.max_pages;
  bool bad_page = false;
  // The page of the 16 tokens from `tok` on, -1 if none holds them.
  auto page_of = [&](int tok) {
    if (tok >= keys) return -1;
    const int p = __ldg(table + (tok >> a.c.log_page));
    if (p < 0 || p >= a.c.num_pages) {
      bad_page = true;
      return -1;
    }
    return p;
  };

  if (warp < 8) {
    // -------------------------------------------------------- softmax --
    const int rtile = warp >> 2;
    const int row = threadIdx.x & 127;
    const int r0 = (2 * rt + rtile) * kTcRows;
    const int r = r0 + row;
    const bool live = row < rows_of(rtile);
    const int my_tiles = rtile ? tiles1 : tiles0;
    const int first_limit = s.len - s.n + r0 / a.group;  // what every row sees
    const int tok = live ? r / a.group : 0;
    const int limit = live ? s.len - s.n + tok : -1;
    const int64_t out_row = static_cast<int64_t>(s.row0 + tok) * a.q_heads + h * a.group +
                            (live ? r - tok * a.group : 0);
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t t_o = lane_addr + kTmemO + 128 * rtile, t_s0 = lane_addr + kTmemS + 128 * rtile;
    float back = 0.f;  // undoes the query scaling, times the softmax scale
    if (my_tiles > 0) {
      // This row of Q, scaled by a power of two, into the swizzled tiles; a
      // negative softmax scale goes into the queries' signs.
      const uint4* qr = reinterpret_cast<const uint4*>(
          a.q + static_cast<int64_t>(s.row0 + tok) * a.ldq +
          (h * a.group + (live ? r - tok * a.group : 0)) * D);
      uint32_t big = 0;
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = live ? __ldg(qr + i) : make_uint4(0, 0, 0, 0);
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                                     __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
      }
      big = max(big & 0xFFFFu, big >> 16);
      const int e = static_cast<int>(big >> 7) - 127;  // largest magnitude in [2^e, 2^(e+1))
      const float mag = __int_as_float((min(7 - e, 126) + 127) << 23);
      const float up = a.scale_log2 < 0.f ? -mag : mag;
      back = __int_as_float((max(e - 7, -126) + 127) << 23) * fabsf(a.scale_log2);
      for (int i = 0; i < D / 8; ++i) {
        const uint4 u = live ? __ldg(qr + i) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const __half2 p = __floats2half2_rn(__uint_as_float(w[x] << 16) * up,
                                              __uint_as_float(w[x] & 0xFFFF0000u) * up);
          o[x] = *reinterpret_cast<const uint32_t*>(&p);
        }
        sts128(base + rtile * SM::kQ + (i >> 3) * (kTcRows * 128) + sw128_offset(row, i & 7), o[0],
               o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(rtile));
    }
    float m = -INFINITY;  // what O and l are relative to
    float v_ref = 0x1p-126f;  // at least: its reciprocal is a number
    uint64_t l2 = pack2(0.f, 0.f);  // the sum, in two halves
    // Scales of the tile's four granules: lane g < 4 fetches those of granule
    // g one tile ahead.
    float sk_next = 0.f, sv_next = 0.f;
    auto scales_of = [&](int j) {
      const int p = (lane < 4 && j < my_tiles) ? page_of(j * kKeys + 16 * lane) : -1;
      const int64_t at = static_cast<int64_t>(p < 0 ? 0 : p) * a.c.heads + h;
      // Not through the non-coherent path: this kernel may be resident while an
      // append writes these scales and reads their neighbours.
      sk_next = p < 0 ? 0.f : a.c.ks[at];
      sv_next = p < 0 ? 0.f : a.c.vs[at];
    };
    scales_of(0);
    bool ok = true;
    for (int j = 0; j < my_tiles; ++j) {
      const int tok0 = j * kKeys;
      float f[4], w[4];
      float v_top = 0.f;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f[g] = __shfl_sync(0xffffffffu, sk_next, g) * back;
        w[g] = __shfl_sync(0xffffffffu, sv_next, g);
        v_top = fmaxf(v_top, w[g]);
      }
      scales_of(j + 1);
      const bool all_seen = tok0 + kKeys - 1 <= first_limit;  // by every live row
      const int seen = limit - tok0;  // columns 0 .. seen of the tile count

      const uint32_t t_s = t_s0 + 64 * (j & 1);
      ok = mbar_wait(s_full(rtile, j & 1), (j >> 1) & 1u, abort_flag, err, kKernelIdAttnTc);
      if (!ok) break;
      tc_fence_after();
      uint32_t sc[2][32];
      tmem_ld32(t_s, sc[0]);
      tmem_ld32(t_s + 32, sc[1]);
      tmem_ld_wait();

      // Largest score; masked scores (which may be anything) do not count.
      float top = -INFINITY;
      auto largest = [&](auto masks) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float t = -INFINITY;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float v = __uint_as_float(sc[g >> 1][(g & 1) * 16 + x]);
            if (!decltype(masks)::value || 16 * g + x <= seen) t = fmaxf(t, v);
          }
          top = fmaxf(top, t == -INFINITY ? t : t * f[g]);
        }
      };
      if (all_seen) largest(std::false_type{}); else largest(std::true_type{});
      // Move the reference maximum only where it has grown by 2^5 or there
      // is none yet, and v_ref only where a value scale exceeds twice it.
      const bool move_m = top > m + kTcGrow || (m == -INFINITY && top > -INFINITY);
      const bool move_v = v_top > 2.f * v_ref;
      float keep = 1.f;
      if (move_m) {
        keep = m == -INFINITY ? 0.f : ex2(m - top);
        l2 = mul2(l2, pack2(keep, keep));
        m = top;
      }
      if (move_v) {
        keep *= v_ref / v_top;
        v_ref = v_top;
      }
      const float off = kTcShift - (m == -INFINITY ? 0.f : m);
      const uint64_t off2 = pack2(off, off);
      const float inv_v = __frcp_rn(v_ref);
      uint32_t p[32];
      auto weights = [&](auto masks) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float wv = w[g] * inv_v;
          const uint64_t f2 = pack2(f[g], f[g]), w2 = pack2(wv, wv);
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const uint64_t e2 =
                fma2(pack2(__uint_as_float(sc[g >> 1][(g & 1) * 16 + x]),
                           __uint_as_float(sc[g >> 1][(g & 1) * 16 + x + 1])), f2, off2);
            float p0, p1;
            unpack2(e2, p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            if (decltype(masks)::value) {
              if (16 * g + x > seen) p0 = 0.f;
              if (16 * g + x + 1 > seen) p1 = 0.f;
            }
            const uint64_t p2 = pack2(p0, p1);
            l2 = add2(l2, p2);
            unpack2(mul2(p2, w2), p0, p1);
            const __half2 q = __floats2half2_rn(p0, p1);
            p[8 * g + x / 2] = *reinterpret_cast<const uint32_t*>(&q);
          }
        }
      };
      if (all_seen) weights(std::false_type{}); else weights(std::true_type{});
      // O is moved between products: all up to the last tile's are done and
      // this tile's waits for P.
      // The last tile's product is waited for before the last P in any case:
      // once that is there two more products may end, and a wait for the
      // first of them would find its phase gone by.
      const bool move = __any_sync(0xffffffffu, move_m || move_v);
      if (j > 0 && (move || j == my_tiles - 1)) {
        ok = mbar_wait(pv_done(rtile), (j - 1) & 1u, abort_flag, err, kKernelIdAttnTc);
        if (!ok) break;
        tc_fence_after();
      }
      if (j > 0 && move) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
          tmem_st32(t_o + c, o);
        }
      }
      tmem_st32(t_s, p);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(rtile, j & 1));
    }
    if (ok && my_tiles > 0)
      ok = mbar_wait(pv_done(rtile), (my_tiles - 1) & 1u, abort_flag, err, kKernelIdAttnTc);
    tc_fence_after();
    if (ok && rows_of(rtile) > 0) {
      // l is times 2^9 like P, so the factors cancel.
      float la, lb;
      unpack2(l2, la, lb);
      const float l = la + lb;
      const bool none = l == 0.f;
      const float inv = 1.f / l;
      __nv_bfloat16* dst = a.out + out_row * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (my_tiles > 0) {
          tmem_ld32(t_o + c, o);
          tmem_ld_wait();
        }
        uint32_t y[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          // A row that sees nothing (l = 0) gets zeros whatever O holds; a sum
          // that is not a number stays one.  v_ref comes last: v_ref / l could
          // underflow where the result does not.
          const float y0 = none ? 0.f : __uint_as_float(o[2 * x]) * inv * v_ref;
          const float y1 = none ? 0.f : __uint_as_float(o[2 * x + 1]) * inv * v_ref;
          const __nv_bfloat162 q = __floats2bfloat162_rn(y0, y1);
          y[x] = *reinterpret_cast<const uint32_t*>(&q);
        }
        if (live) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + c);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            d4[x] = make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
        }
      }
    }
  } else if (warp < 10) {
    // ------------------------------------------------------------ MMA --
    const bool one = elect_lane();
    const int t = warp - 8;
    constexpr uint32_t idesc_s = idesc_f16(kTcRows, kKeys, false);
    constexpr uint32_t idesc_o = idesc_f16(kTcRows, D, false);
    const int my_tiles = t ? tiles1 : tiles0;
    const uint32_t t_s0 = tmem + kTmemS + 128 * t, t_o = tmem + kTmemO + 128 * t;
    bool issued = false;
    // Scores of key tile j, which come two by two ahead of the outputs: the
    // buffer's last user, the outputs of tile j - 2, was issued before.
    int kst = 0;
    uint32_t kph = 0;
    auto scores = [&](int j) {
      if (!mbar_wait(k_full(kst), kph, abort_flag, err, kKernelIdAttnTc)) return false;
      tc_fence_after();
      if (one) {
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const uint64_t da = sdesc_k_sw128(base + t * SM::kQ + half * (kTcRows * 128));
          const uint64_t db = sdesc_k_sw128(base + SM::k + kst * SM::kK + half * (kKeys * 128));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16(t_s0 + 64 * (j & 1), da + 2ull * kk, db + 2ull * kk, idesc_s,
                     (half | kk) != 0);
        }
        umma_commit(s_full(t, j & 1));
        umma_commit(k_empty(kst));
      }
      issued = true;
      if (++kst == kTcStages) kst = 0, kph ^= 1u;
      return true;
    };
    bool ok = true;
    if (my_tiles > 0) {
      ok = mbar_wait(q_full(t), 0, abort_flag, err, kKernelIdAttnTc) && scores(0);
      if (ok && my_tiles > 1) ok = scores(1);
    }
    int st = 0;
    uint32_t ph = 0;
    for (int j = 0; ok && j < my_tiles; ++j) {
      ok = mbar_wait(v_full(st), ph, abort_flag, err, kKernelIdAttnTc) &&
           mbar_wait(p_full(t, j & 1), (j >> 1) & 1u, abort_flag, err, kKernelIdAttnTc);
      if (!ok) break;
      tc_fence_after();
      if (one) {
        const uint64_t db = sdesc_k_sw128(base + SM::v + st * SM::kV);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          umma_f16_ta(t_o, t_s0 + 64 * (j & 1) + 8 * kk, db + 2ull * kk, idesc_o, (j | kk) != 0);
        umma_commit(pv_done(t));
        umma_commit(v_empty(st));
      }
      if (++st == kTcStages) st = 0, ph ^= 1u;
      if (j + 2 < my_tiles) ok = scores(j + 2);
    }
    // Key tiles that only the other row tile has: release them as they come.
    for (int j = my_tiles; ok && j < tiles && !*abort_flag; ++j) {
      const int s3 = j % kTcStages;
      const uint32_t p3 = (j / kTcStages) & 1u;
      if (!mbar_wait(k_full(s3), p3, abort_flag, err, kKernelIdAttnTc)) break;
      if (one) mbar_arrive(k_empty(s3));
      if (!mbar_wait(v_full(s3), p3, abort_flag, err, kKernelIdAttnTc)) break;
      if (one) mbar_arrive(v_empty(s3));
    }
    if (*abort_flag && issued && one) {
      umma_commit(done_bar(t));  // in-flight MMAs end before TMEM is freed
      volatile int dummy = 0;
      mbar_wait(done_bar(t), 0, &dummy, err, kKernelIdAttnTc, kWaitLimitNs / 4);
    }
  } else {
    // ------------------------------------------------- dequantization --
    const int t = threadIdx.x - 320;  // 0 .. 127
    // Pieces of 16 codes: eight neighbouring lanes hold eight rows (tokens of
    // keys, channels of values) of one 16-code chunk, so their 16-byte stores
    // meet different banks of the swizzled tile.
    constexpr int kPieces = kKeys * D / 16 / 128;  // per thread and side: 4 or 2
    constexpr int kChunks = D / 16;                // chunks of a key row
    const int sub = t & 7, grp8 = t >> 3;  // 16 groups of 8 lanes
    // Keys: piece i is token k_row(i), chunk k_chunk; values: channel v_row(i),
    // tokens 16 v_chunk ..
    const int k_chunk = grp8 % kChunks;
    auto k_row = [&](int i) { return (grp8 / kChunks + i * (16 / kChunks)) * 8 + sub; };
    const int v_chunk = grp8 & 3;
    auto v_row = [&](int i) { return ((grp8 >> 2) + 4 * i) * 8 + sub; };
    const int page_mask = (1 << a.c.log_page) - 1;
    // Bytes from page to page (keys and values alike), and of this head.
    const int64_t page_bytes = (static_cast<int64_t>(a.c.heads) << a.c.log_page) * D;
    const int64_t head_bytes = (static_cast<int64_t>(h) << a.c.log_page) * D;
    // Page ids of a tile's four granules, in the lanes g < 4.
    auto pages = [&](int j) {
      return (lane < 4 && j < tiles) ? page_of(j * kKeys + 16 * lane) : -1;
    };
    // Each lane's own ring: keys and values of kTcAhead tiles, read back only
    // by the lane that copied them.
    const uint32_t own = base + SM::codes + 16u * t;
    auto copy_k = [&](int j, int slot, int id) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = k_row(i);
        const int p = __shfl_sync(0xffffffffu, id, row >> 4);
        kv8_copy16(own + slot * 2 * SM::kCodes + i * 2048u,
                   a.c.k + (p < 0 ? 0 : p) * page_bytes + head_bytes +
                       ((j * kKeys + row) & page_mask) * D + 16 * k_chunk,
                   p >= 0);
      }
      kv8_copy_commit();
    };
    auto copy_v = [&](int j, int slot, int id) {
      const int p = __shfl_sync(0xffffffffu, id, v_chunk);
      const uint8_t* src = a.c.v + (p < 0 ? 0 : p) * page_bytes + head_bytes +
                           ((j * kKeys + 16 * v_chunk) & page_mask);
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        kv8_copy16(own + (slot * 2 + 1) * SM::kCodes + i * 2048u,
                   src + (v_row(i) << a.c.log_page), p >= 0);
      kv8_copy_commit();
    };
    auto put = [&](uint32_t tile, int row, int chunk, uint4 c) {
      // 16 codes are two 16-byte chunks of the row's 128 bytes.
      uint32_t o[8];
      kv8_codes_to_f16<FMT>(c.x, o[0], o[1]);
      kv8_codes_to_f16<FMT>(c.y, o[2], o[3]);
      kv8_codes_to_f16<FMT>(c.z, o[4], o[5]);
      kv8_codes_to_f16<FMT>(c.w, o[6], o[7]);
      const uint32_t at = tile + sw128_offset(row, 2 * chunk);
      sts128(at, o[0], o[1], o[2], o[3]);
      sts128(at ^ 16u, o[4], o[5], o[6], o[7]);  // the neighbouring chunk
    };
    for (int j = 0; j < kTcAhead; ++j) {
      const int id = pages(j);
      copy_k(j, j, id);
      copy_v(j, j, id);
    }
    int id_next = pages(kTcAhead);
    int st = 0, slot = 0;
    uint32_t ph = 1;  // phase of the stage's release to wait for
    for (int j = 0; j < tiles; ++j) {
      const int id = id_next;  // of tile j + kTcAhead
      id_next = pages(j + kTcAhead + 1);
      if (j >= kTcStages && !mbar_wait(k_empty(st), ph, abort_flag, err, kKernelIdAttnTc)) break;
      kv8_copy_wait<2 * kTcAhead - 1>();
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        put(base + SM::k + st * SM::kK + (k_chunk >> 2) * (kKeys * 128), k_row(i), k_chunk & 3,
            kv8_lds128(own + slot * 2 * SM::kCodes + i * 2048u));
      copy_k(j + kTcAhead, slot, id);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(st));
      if (j >= kTcStages && !mbar_wait(v_empty(st), ph, abort_flag, err, kKernelIdAttnTc)) break;
      kv8_copy_wait<2 * kTcAhead - 1>();
      const int held = keys - (j * kKeys + 16 * v_chunk);  // tokens of these 16 that count
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint4 c = kv8_lds128(own + (slot * 2 + 1) * SM::kCodes + i * 2048u);
        if (held < 16) {
          // Bytes behind the last key may hold anything, NaN codes included.
          auto mask = [&](uint32_t v, int x) {
            const int nb = held - 4 * x;
            return nb >= 4 ? v : nb <= 0 ? 0u : v & ((1u << (8 * nb)) - 1u);
          };
          c = make_uint4(mask(c.x, 0), mask(c.y, 1), mask(c.z, 2), mask(c.w, 3));
        }
        put(base + SM::v + st * SM::kV, v_row(i), v_chunk, c);
      }
      copy_v(j + kTcAhead, slot, id);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
      if (++st == kTcStages) st = 0, ph ^= 1u;
      if (++slot == kTcAhead) slot = 0;
    }
    kv8_copy_wait<0>();
  }
  if (bad_page) record_error(err, kErrBadIndex, kKernelIdAttnTc);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

template <int FMT, int D>
cudaError_t launch_tc(const TcArgs& a, cudaStream_t stream, unsigned* err) {
  using SM = TcSmem<D>;
  constexpr auto kern = kv8_attention_tc_kernel<FMT, D>;
  static unsigned long long done = 0;  // bit d: device d
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(__atomic_load_n(&done, __ATOMIC_ACQUIRE) & (1ull << dev))) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(SM::bytes));
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.row_tiles),
                     static_cast<unsigned>(a.bt.batch) * a.c.heads, 1);
  cfg.blockDim = dim3(kTcThreads, 1, 1);
  cfg.dynamicSmemBytes = SM::bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a, err);
}

}  // namespace

// Which kernel: per 64 keys the tcgen05 kernel takes 1.2 us (one row tile) or
// 1.95 us (two) for each wave of CTAs, the rows kernel about 0.003 us for each
// 16 rows of each problem.  The host knows neither the lengths, which enter
// both alike, nor each sequence's new tokens: all are taken to have max_new,
// so a batch of single tokens and one long run goes to the tcgen05 kernel,
// which walks each single token's keys unsplit (one run of 512 and 63 single
// tokens over 4096 keys each: 340 us, in two calls 207).
// Measured, rows / tcgen05 kernel: 8 x 128
// tokens over 4096 keys (16 / 8 heads) 156 / 100 us, 8 x 64 90 / 78, 8 x 16
// 35 / 76; 1 x 256 over 16384 205 / 360; 2 x 2048 over 8192 917 / 249.
bool kv8_attention_prefers_tc(const Kv8Cache& c, const Kv8Batch& bt, int group, int num_sms) {
  const int64_t problems = static_cast<int64_t>(bt.batch) * c.heads;
  if (problems > 65535) return false;  // a grid axis
  const int64_t rows = static_cast<int64_t>(bt.max_new) * group;
  const double ctas = static_cast<double>(problems) * ((rows + 2 * kTcRows - 1) / (2 * kTcRows));
  const double waves = ctas > num_sms ? ctas / num_sms : 1.0;
  return waves * (rows > kTcRows ? 1.95 : 1.2) < 0.003 * ((rows + 15) / 16) * problems;
}

cudaError_t launch_kv8_attention_tc(const Kv8Cache& c, const Kv8Batch& bt, const void* q,
                                    int64_t ldq, int q_heads, int D, int fmt, float scale,
                                    void* out, cudaStream_t stream, unsigned* err) {
  TcArgs a;
  a.c = c;
  a.bt = bt;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ldq = ldq;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  a.row_tiles = static_cast<int>((static_cast<int64_t>(bt.max_new) * a.group + 2 * kTcRows - 1) /
                                 (2 * kTcRows));
  a.scale_log2 = scale * 1.4426950408889634f;
  if (fmt == kKvInt8)
    return D == 64 ? launch_tc<kKvInt8, 64>(a, stream, err) : launch_tc<kKvInt8, 128>(a, stream, err);
  return D == 64 ? launch_tc<kKvE4m3, 64>(a, stream, err) : launch_tc<kKvE4m3, 128>(a, stream, err);
}

}  // namespace w4
