// bf16 -> microscaled 4-bit floating point (e2m1 codes with block scales).
//
// mx: blocks of 32 channels, the scale a power of two two binades under the
//     block's largest magnitude: s = 2^e, e = clamp(floor(log2 amax) - 2,
//     -127, 127) (-127 for a block of zeros).
// nv: blocks of 16 channels, an e4m3 scale in units of a power of two of the
//     row: 2^E the least with max|row| <= 6 * 448 * 2^E (E >= -126, E = 0
//     for a row of zeros), s = e4m3(amax / (6 * 2^E)).
// code = e2m1(x / (s 2^E)), ties to even, saturating at 6; a block whose
// scale rounds to 0 has codes of magnitude 0.  Signs are kept, also on 0.
//
// Every decision is taken on exact values.  mx: x 2^-e is exact.  nv: 6 t
// for an e4m3 rounding border t has 7 significant bits, and b s for an e2m1
// border b has 7, while x has 8: a quotient that is not on its border is at
// least 2^-9 (relative) away from it.  So the products amax * (1 / 6) and x * (1 / s),
// with factors a little large (by 2^-20, more than all their rounding errors
// together) and cut to 13 significant bits, lie on the side of every border
// that the true quotient lies on, and on it where that does.  The values (2 + 4 significant
// bits, or 2) are exact in bf16 from 2^-126 up.
//
// Bound: HBM (2 bytes read and 0.53 / 0.56 written per weight, 2 more with
// values).  A thread owns 16 consecutive channels; the largest magnitude of
// an mx block takes one shuffle, of an nv block none.  The four scale bytes
// of a tile word are gathered by shuffles and stored as one word.  The nv
// row maximum is a first pass over the row, which stays in registers: a row's
// CTA has as many warps as it takes at one to three pieces per thread (8192 x
// 17408: 69 us, 5.2 TB/s, with 384 threads of three pieces, two CTAs per SM, up
// to 77 back to back; 83 with 544 of two and one CTA; 140 with 256 threads
// whatever the row).  Rows of more than 18432 channels have two pieces and one
// CTA per SM again, those of more than 32768 are read twice.  mx with values
// runs at 97 % of the copy rate (17408 x 5120: 63 us).
#include <type_traits>

#include "fp4.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace {

constexpr int kQuantThreads = 256;
struct Piece {
  uint32_t u[8];  // 16 bf16
};

__device__ __forceinline__ Piece load_piece(const uint4* p) {
  Piece r;
  const uint4 a = __ldg(p), b = __ldg(p + 1);
  r.u[0] = a.x, r.u[1] = a.y, r.u[2] = a.z, r.u[3] = a.w;
  r.u[4] = b.x, r.u[5] = b.y, r.u[6] = b.z, r.u[7] = b.w;
  return r;
}

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t u) {
  return *reinterpret_cast<const __nv_bfloat162*>(&u);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Largest magnitude of the 16 channels.
__device__ __forceinline__ float piece_amax(const Piece& p) {
  __nv_bfloat162 m = as_bf2(p.u[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2(m, as_bf2(p.u[i] & 0x7FFF7FFFu));
  const uint32_t u = as_u32(m);
  return fmaxf(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

// The 16 channels times a power of two (exact in bf16, except results under
// 2^-126, whose codes are 0 either way), as floats.
__device__ __forceinline__ void scaled(const Piece& p, float pow2, float (&v)[16]) {
  const __nv_bfloat162 f = __float2bfloat162_rn(pow2);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = as_u32(__hmul2(as_bf2(p.u[i]), f));
    v[2 * i] = __uint_as_float(u << 16);
    v[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
  }
}

// v cut to 13 significant bits (towards zero).
__device__ __forceinline__ float cut(float v) {
  return __uint_as_float(__float_as_uint(v) & 0xFFFFF800u);
}

// 1 / 6 and 1 / s (s normal), 2^-20 large: the approximate reciprocal is off
// by at most one unit in the last place, the products by half of one each.
constexpr float kSixth = 0.16666666666f * (1.f + 0x1p-20f);
__device__ __forceinline__ float reciprocal_up(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r * (1.f + 0x1p-20f);
}

__device__ __forceinline__ uint2 codes_of(const float (&v)[16]) {
  const float a[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  const float b[8] = {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]};
  return make_uint2(e2m1x8(a), e2m1x8(b));
}

// The values that codes stand for at scale s, as 16 bf16.
__device__ __forceinline__ void store_values(uint2 c, float s, uint4* out) {
  uint32_t o[8];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(e2m1_pair_to_f16(half ? c.y : c.x, i));
      o[4 * half + i] = as_u32(__floats2bfloat162_rn(f.x * s, f.y * s));
    }
  }
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Address of the scale word of (row, blocks 4 w .. 4 w + 3); `words` per row.
__device__ __forceinline__ uint32_t* scale_word(uint8_t* scales, int64_t row, int64_t w,
                                                int64_t words) {
  return reinterpret_cast<uint32_t*>(scales + ((row >> 7) * words + w) * 512 + (row & 31) * 16 +
                                     ((row >> 5) & 3) * 4);
}

// mx: piece i of the matrix is channels 16 (i % (K/16)) .. of row i / (K/16).
// K / 16 is a multiple of 8, so the eight lanes of a scale word share a row.
template <bool VALUES>
__global__ void __launch_bounds__(kQuantThreads)
    fp4_quantize_mx_kernel(const __nv_bfloat16* __restrict__ x, int64_t pieces, int per_row,
                           int64_t ldx, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                           __nv_bfloat16* __restrict__ values) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kQuantThreads;
  // Whole warps stay in the loop for the shuffles; pieces is a multiple of 8.
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kQuantThreads + (threadIdx.x & ~31);
       i0 < pieces; i0 += stride) {
    const int64_t i = i0 + lane;
    const bool live = i < pieces;
    const int64_t row = live ? ((i >> 32) ? i / per_row
                                          : static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row))
                             : 0;
    const int c = live ? static_cast<int>(i - row * per_row) : 0;
    Piece p = {};
    if (live) p = load_piece(reinterpret_cast<const uint4*>(x + row * ldx) + 2 * c);
    float amax = piece_amax(p);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    // The exponent field is floor(log2 amax) + 127, 0 for zero and subnormal
    // magnitudes, whose scale is 2^-127.
    const int field = static_cast<int>(__float_as_uint(amax) >> 23);
    const int byte = field > 2 ? field - 2 : 0;  // e + 127
    float v[16];
    scaled(p, __uint_as_float(static_cast<uint32_t>(254 - byte) << 23), v);  // 2^-e
    const uint2 q = codes_of(v);
    const int b1 = __shfl_down_sync(0xffffffffu, byte, 2);
    const int b2 = __shfl_down_sync(0xffffffffu, byte, 4);
    const int b3 = __shfl_down_sync(0xffffffffu, byte, 6);
    if (!live) continue;
    reinterpret_cast<uint2*>(codes)[i] = q;
    if ((lane & 7) == 0)
      *scale_word(scales, row, c >> 3, per_row >> 3) =
          static_cast<uint32_t>(byte) | (b1 << 8) | (b2 << 16) | (static_cast<uint32_t>(b3) << 24);
    if (VALUES) store_values(q, exp2_int(byte - 127), reinterpret_cast<uint4*>(values) + 2 * i);
  }
}

constexpr int nv_registers(int held) { return held == 1 ? 48 : held == 2 ? 64 : 80; }

// nv: a warp (WARP) or the CTA owns one row; a thread keeps HELD pieces in
// registers between the passes (the rest of a longer row is read again).
template <bool VALUES, bool WARP, int HELD>
__global__ void __maxnreg__(nv_registers(HELD))
    fp4_quantize_nv_kernel(const __nv_bfloat16* __restrict__ x, int64_t rows, int per_row,
                           int64_t ldx, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                           float* __restrict__ row_scale, __nv_bfloat16* __restrict__ values) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int G = WARP ? 32 : static_cast<int>(blockDim.x);
  const int t = WARP ? lane : static_cast<int>(threadIdx.x);
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * (kQuantThreads / 32) : gridDim.x;
  int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (kQuantThreads / 32) + (threadIdx.x >> 5)
                     : static_cast<int64_t>(blockIdx.x);

  // The next row is on its way while this one is reduced and written.
  Piece next[HELD];
  auto fetch = [&](int64_t at) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + at * ldx);
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int c = t + j * G;
      next[j] = Piece{};
      if (at < rows && c < per_row) next[j] = load_piece(xr + 2 * c);
    }
  };
  fetch(row);
  for (int turn = 0; row < rows; row += step, turn ^= 1) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + row * ldx);
    Piece held[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) held[j] = next[j];
    fetch(row + step);
    float amax = 0.f, top[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      top[j] = piece_amax(held[j]);
      amax = fmaxf(amax, top[j]);
    }
    for (int c = t + HELD * G; c < per_row; c += G)
      amax = fmaxf(amax, piece_amax(load_piece(xr + 2 * c)));
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!WARP) {
      // Two sets of maxima in turn: a warp may be a row ahead, not two.
      if (lane == 0) red[turn][threadIdx.x >> 5] = amax;
      __syncthreads();
      amax = lane < (G >> 5) ? red[turn][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    // amax = f 2^n with 1 <= f < 2, and 2688 = 1.3125 * 2^11.
    int E = 0;
    if (amax > 0.f) {
      const uint32_t u = __float_as_uint(amax);
      E = static_cast<int>(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x280000u ? 11 : 10);
      if (E < -126) E = -126;  // also every subnormal maximum
    }
    const float up = exp2_int(E), down = exp2_int(-E);
    if (t == 0) row_scale[row] = up;

    const int64_t words = per_row >> 2;
    auto emit = [&](int c, const Piece& p, float largest) {
      // Called by whole groups of 4 lanes (per_row is a multiple of 8).
      const uint32_t byte = e4m3_of(cut(largest * down * kSixth));
      const float s = e4m3_value(byte);
      const float r = s > 0.f ? reciprocal_up(s) : 0.f;
      float v[16];
      scaled(p, down, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = cut(v[i] * r);
      const uint2 q = codes_of(v);
      const uint32_t four = 0xFu << (lane & ~3);
      const uint32_t b1 = __shfl_down_sync(four, byte, 1, 4);
      const uint32_t b2 = __shfl_down_sync(four, byte, 2, 4);
      const uint32_t b3 = __shfl_down_sync(four, byte, 3, 4);
      const int64_t i = row * per_row + c;
      reinterpret_cast<uint2*>(codes)[i] = q;
      if ((lane & 3) == 0)
        *scale_word(scales, row, c >> 2, words) = byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
      if (VALUES) store_values(q, s * up, reinterpret_cast<uint4*>(values) + 2 * i);
    };
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int c = t + j * G;
      if (c < per_row) emit(c, held[j], top[j]);
    }
    for (int c = t + HELD * G; c < per_row; c += G) {
      const Piece p = load_piece(xr + 2 * c);
      emit(c, p, piece_amax(p));
    }
  }
}

template <auto kern, typename... Args>
cudaError_t launch_pdl(int64_t grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <bool VALUES>
cudaError_t quantize(const __nv_bfloat16* x, int64_t R, int64_t K, int64_t ldx, int fmt,
                     uint8_t* codes, uint8_t* scales, float* row_scale, __nv_bfloat16* values,
                     cudaStream_t stream, int num_sms) {
  const int per_row = static_cast<int>(K / 16);
  if (fmt == kFp4Mx) {
    const int64_t pieces = R * per_row;
    const int64_t want = (pieces + kQuantThreads - 1) / kQuantThreads;
    const int64_t grid = want < int64_t{num_sms} * 64 ? want : int64_t{num_sms} * 64;
    return launch_pdl<fp4_quantize_mx_kernel<VALUES>>(grid, kQuantThreads, stream, x, pieces,
                                                      per_row, ldx, codes, scales, values);
  }
  if (per_row <= 64) {
    const int64_t want = (R + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
    const int64_t grid = want < int64_t{num_sms} * 4 ? want : int64_t{num_sms} * 4;
    return launch_pdl<fp4_quantize_nv_kernel<VALUES, true, 2>>(
        grid, kQuantThreads, stream, x, R, per_row, ldx, codes, scales, row_scale, values);
  }
  // Pieces per thread: one up to 512 threads (few rows: the latency of one
  // round), else two, but three where two would leave one CTA of some 20 warps
  // per SM and three make two CTAs fit; as many CTAs as are resident at once.
  auto launch = [&](auto held) {
    constexpr int kHeld = decltype(held)::value;
    const int pieces = (per_row + kHeld - 1) / kHeld;
    const int threads = pieces < 1024 ? (pieces + 31) & ~31 : 1024;
    const int64_t most = int64_t{num_sms} * (65536 / (nv_registers(kHeld) * threads));
    return launch_pdl<fp4_quantize_nv_kernel<VALUES, false, kHeld>>(
        R < most ? R : most, threads, stream, x, R, per_row, ldx, codes, scales, row_scale, values);
  };
  if (per_row <= 512) return launch(std::integral_constant<int, 1>{});
  if (per_row <= 1024 || per_row > 1152) return launch(std::integral_constant<int, 2>{});
  return launch(std::integral_constant<int, 3>{});
}

}  // namespace

cudaError_t launch_fp4_quantize(const void* x, int64_t R, int64_t K, int64_t ldx, int fmt,
                                uint8_t* codes, uint8_t* scales, float* row_scale, void* values,
                                cudaStream_t stream, int num_sms) {
  const auto* xp = static_cast<const __nv_bfloat16*>(x);
  auto* vp = static_cast<__nv_bfloat16*>(values);
  return vp ? quantize<true>(xp, R, K, ldx, fmt, codes, scales, row_scale, vp, stream, num_sms)
            : quantize<false>(xp, R, K, ldx, fmt, codes, scales, row_scale, vp, stream, num_sms);
}

}  // namespace w4
