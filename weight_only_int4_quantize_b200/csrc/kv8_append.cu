// New keys and values into the 8-bit paged cache (layout: kv8.cuh).
//
// For every page and kv head that a new token falls into, with a the largest
// magnitude of the page's new tokens and s0 the page's scale (0 where the
// page held no earlier token of the sequence):
//
//   s = max(s0, up(a / qmax)),  up: the next value that bf16 holds, at least
//                               2^-126 (0 for a = 0)
//   new codes      round(x / s)                (ties to even; s = 0: 0)
//   earlier codes  round(code * s0 / s)        only where s > s0
//
// Every rounding is decided exactly.  With s (and s0) of 8 significant bits,
// which is what this kernel writes, a code's rounding border times s has at
// most 16 bits (and so has code * s0), x has 8, so a quotient that is not on
// its border is at least 2^-17 (relative) away from it.  x * (1 / s), off by
// less than 2^-22, rounded to 20 significant bits, therefore falls on the same
// side, and back onto the border where it is on it; no division is needed.
// A page's scale may also have come from elsewhere, with 24 bits: then both
// sides have at most 32 bits, a quotient is at least 2^-33 away, and the same
// is done in binary64 with 41 bits (write_exact).  That takes a page that held
// earlier tokens, so one page of a sequence, head and side at most.
//
// A warp owns 16 tokens (a granule) of one page, kv head and side; the
// page_size / 16 warps of a page share its largest magnitude through shared
// memory.  A lane owns D / 32 neighbouring channels of all 16 tokens: rows are
// read coalesced, key codes leave as words of a row, and the 16 codes of a
// channel, which lie side by side in a value row, as one 16-byte store; nothing
// is turned in shared memory.  Bound: for prompts the instructions of the
// exact decisions at the occupancy that 64 registers leave (58 % of the issue
// slots, 43 % of the warps; 4 of up to 4000 tokens, 8 heads of 128: 16.6 us,
// where their 69 MB take 10.5; some 4 us more without the path for granules that
// are new from end to end; a CTA per page 52), for single tokens the chain of
// dependent loads (length, page id, rows and scale), in which write_exact adds
// nothing that shows (64 tokens: 5.9 us either way).
#include "kv8.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kGranule = 16;
constexpr unsigned kKernelIdAppend = 16;

// v rounded to 20 significant bits.
__device__ __forceinline__ float snap(float v) {
  return __uint_as_float((__float_as_uint(v) + 0x8u) & 0xFFFFFFF0u);
}

// Codes of four values (in units of the scale), one per byte.
template <int FMT>
__device__ __forceinline__ uint32_t kv_codes(float v0, float v1, float v2, float v3) {
  if constexpr (FMT == kKvInt8) {
    // + 1.5 * 2^23 rounds to an integer, ties to even, into the low bits.
    // |v| <= 127 by the choice of the scale.
    const float big = 12582912.f;
    const uint32_t a = __byte_perm(__float_as_uint(v0 + big), __float_as_uint(v1 + big), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(v2 + big), __float_as_uint(v3 + big), 0x0040);
    return __byte_perm(a, b, 0x5410);
  } else {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(v1), "f"(v0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(v3), "f"(v2));
    return static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
  }
}

template <int FMT>
__device__ __forceinline__ float kv_value(uint32_t code) {
  if constexpr (FMT == kKvInt8) {
    return static_cast<float>(static_cast<int8_t>(code));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code & 0xFFu)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xFFFFu)));
  }
}

// The four codes of a word times f (= s0 / s, as s0 * (1 / s): both factors
// are applied one after the other and only the last product is not exact).
template <int FMT>
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float s0, float inv) {
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = snap(kv_value<FMT>(w >> (8 * i)) * s0 * inv);
  return kv_codes<FMT>(v[0], v[1], v[2], v[3]);
}

// A quotient off by less than 2^-51 as a float on the same side of every
// border, or on it: to 41 significant bits, then rounded to odd.
__device__ __forceinline__ float snap_exact(double v) {
  const double w = __longlong_as_double((__double_as_longlong(v) + 0x800ll) & ~0xFFFll);
  const float f = __double2float_rz(w);
  return static_cast<double>(f) == w ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Tokens first .. last - 1 of a granule at scales of any number of bits: a lane's
// CH channels, `token` and `channel` bytes apart from `cell` on; tokens from
// `fresh` on are new (rows `ld` apart from x on), those before are rescaled.
template <int FMT, int CH>
__device__ __noinline__ void write_exact(uint8_t* cell, int token, int channel, int first, int last,
                                         int fresh, const __nv_bfloat16* x, int64_t ld, float s0,
                                         float s1) {
  const double inv = 1.0 / static_cast<double>(s1);
#pragma unroll 1
  for (int t = first; t < last; ++t) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      uint8_t* at = cell + t * token + i * channel;
      const double v = t >= fresh
                           ? static_cast<double>(__bfloat162float(x[t * ld + i]))
                           : static_cast<double>(kv_value<FMT>(*at)) * static_cast<double>(s0);
      *at = static_cast<uint8_t>(kv_codes<FMT>(snap_exact(v * inv), 0.f, 0.f, 0.f));
    }
  }
}

// Bytes of `after` where tokens first .. first + 3 are new or rescaled
// earlier ones, of `before` elsewhere.
__device__ __forceinline__ uint32_t byte_mask(int first, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (first + i >= lo && first + i < hi) m |= 0xFFu << (8 * i);
  return m;
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads, 4)
    kv8_append_kernel(const Kv8Cache c, const Kv8Batch bt, const __nv_bfloat16* __restrict__ k,
                      const __nv_bfloat16* __restrict__ v, int64_t ldk, int64_t ldv, int touched,
                      int64_t units, unsigned* err) {
  constexpr int CH = D / 32;  // channels of a lane
  __shared__ float red[kAppendThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int log_warps = c.log_page - 4;  // warps of a unit (page, head, side)
  const int w = warp & ((1 << log_warps) - 1);
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) << (3 - log_warps)) + (warp >> log_warps);
  pdl_launch_dependents();
  pdl_wait();
  if (unit >= units) return;
  const bool is_v = (unit & 1) != 0;
  const int h = static_cast<int>((unit >> 1) % c.heads);
  const int bj = static_cast<int>((unit >> 1) / c.heads);
  const int b = bj / touched, jt = bj % touched;
  const Kv8Seq s = kv8_sequence(bt, b, c.log_page);
  if (s.bad && lane == 0 && h == 0 && jt == 0 && !is_v && w == 0)
    record_error(err, kErrBadIndex, kKernelIdAppend);
  const int old = s.len > s.n ? s.len - s.n : 0;
  const int skip = s.n - (s.len - old);  // new tokens in front of position 0: not held
  const int j = (old >> c.log_page) + jt;  // page of the sequence
  const int64_t p0 = static_cast<int64_t>(j) << c.log_page;
  if (s.n == 0 || p0 >= s.len) return;  // all warps of the unit
  const int page_size = 1 << c.log_page;
  const int lo = old > p0 ? static_cast<int>(old - p0) : 0;  // new tokens [lo, hi) of the page
  const int hi = s.len - p0 < page_size ? static_cast<int>(s.len - p0) : page_size;
  const int page = __ldg(bt.table + static_cast<int64_t>(b) * bt.max_pages + j);
  const int t0 = kGranule * w;  // this warp's tokens of the page
  const int64_t ld = is_v ? ldv : ldk;
  // Row of token t0 (only those of new tokens are read).  The rows are on
  // their way while the page id is.
  const __nv_bfloat16* x = (is_v ? v : k) + static_cast<int64_t>(h) * D + lane * CH +
                           (static_cast<int64_t>(s.row0) + skip + (p0 + t0 - old)) * ld;
  uint32_t raw[kGranule][CH / 2];
  auto fetch = [&](int t, const __nv_bfloat16* at) {
    if constexpr (CH == 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
      raw[t][0] = u.x;
      raw[t][1] = u.y;
    } else {
      raw[t][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
  };
  // A prompt's granules are new from end to end, but for two.
  const bool whole = t0 >= lo && t0 + kGranule <= hi;
  if (whole) {
    const __nv_bfloat16* at = x;
#pragma unroll
    for (int t = 0; t < kGranule; ++t, at += ld) fetch(t, at);
  } else {
#pragma unroll
    for (int t = 0; t < kGranule; ++t) {
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) raw[t][i] = 0;
      if (t0 + t >= lo && t0 + t < hi) fetch(t, x + t * ld);
    }
  }
  if (page < 0 || page >= c.num_pages) {
    if (lane == 0) record_error(err, kErrBadIndex, kKernelIdAppend);
    return;
  }
  const int64_t slot = static_cast<int64_t>(page) * c.heads + h;
  float* scale = (is_v ? c.vs : c.ks) + slot;
  const float s0 = lo > 0 ? *scale : 0.f;
  uint32_t big = 0;
#pragma unroll
  for (int t = 0; t < kGranule; ++t)
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) big = __vmaxu2(big, raw[t][i] & 0x7FFF7FFFu);
  big = max(big & 0xFFFFu, big >> 16);
  big = __reduce_max_sync(0xffffffffu, big);
  if (log_warps > 0) {
    if (lane == 0) red[warp] = __uint_as_float(big << 16);
    const int id = 1 + (warp >> log_warps);
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 << log_warps) : "memory");
    float m = 0.f;
    for (int i = 0; i < (1 << log_warps); ++i) m = fmaxf(m, red[warp - w + i]);
    big = __float_as_uint(m) >> 16;
  }
  const float amax = __uint_as_float(big << 16);
  float up = __uint_as_float(
      (__float_as_uint(__fdiv_rn(amax, kv8_qmax(FMT))) + 0xFFFFu) & 0xFFFF0000u);
  if (amax > 0.f) up = fmaxf(up, __uint_as_float(0x00800000u));  // 2^-126: 1 / s is finite
  const float s1 = fmaxf(s0, up);
  // Every warp of the unit has read the old scale before the barrier above.
  if (w == 0 && lane == 0) *scale = s1;
  const float inv = s1 > 0.f ? __frcp_rn(s1) : 0.f;
  const bool again = lo > 0 && s1 > s0;
  const int from = again ? 0 : lo;  // bytes of tokens [from, hi) are written
  if (t0 >= hi || t0 + kGranule <= from) return;

  // More than 8 significant bits, or no binary32 reciprocal.
  if (((__float_as_uint(s1) | (again ? __float_as_uint(s0) : 0u)) & 0xFFFFu) != 0 ||
      (s1 > 0.f && s1 < __uint_as_float(0x00800000u))) {
    const int first = from > t0 ? from - t0 : 0, last = hi - t0 < kGranule ? hi - t0 : kGranule;
    uint8_t* cell = is_v ? c.v + ((slot * D + lane * CH) << c.log_page) + t0
                         : c.k + ((slot << c.log_page) + t0) * D + lane * CH;
    write_exact<FMT, CH>(cell, is_v ? 1 : D, is_v ? page_size : 1, first, last, lo - t0, x, ld, s0,
                         s1);
    return;
  }

  auto value = [&](int t, int i) {  // channel i of the lane, in units of the scale
    const uint32_t u = raw[t][i / 2];
    return snap(__uint_as_float((i & 1) ? (u & 0xFFFF0000u) : (u << 16)) * inv);
  };
  if (is_v) {
    uint8_t* col = c.v + ((slot * D + lane * CH) << c.log_page) + t0;
    const int first = lo > t0 ? lo - t0 : 0, last = hi - t0 < kGranule ? hi - t0 : kGranule;
    if (!whole && !again && last - first <= 4) {
      // A few new tokens (a decode step's one): their bytes alone, so that
      // nothing of the page has to be fetched first.
#pragma unroll
      for (int t = 0; t < kGranule; ++t)
        if (t >= first && t < last) {
#pragma unroll
          for (int i = 0; i < CH; ++i)
            col[(i << c.log_page) + t] =
                static_cast<uint8_t>(kv_codes<FMT>(value(t, i), 0.f, 0.f, 0.f));
        }
      return;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      uint4* dst = reinterpret_cast<uint4*>(col + (i << c.log_page));
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = kv_codes<FMT>(value(4 * q, i), value(4 * q + 1, i), value(4 * q + 2, i),
                             value(4 * q + 3, i));
      if (!whole) {
        const uint4 was = *dst;
        const uint32_t e[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t fresh = byte_mask(t0 + 4 * q, lo, hi);
          const uint32_t earlier = again ? byte_mask(t0 + 4 * q, 0, lo) : 0u;
          const uint32_t re = again ? rescaled<FMT>(e[q], s0, inv) : 0u;
          o[q] = (o[q] & fresh) | (re & earlier) | (e[q] & ~(fresh | earlier));
        }
      }
      *dst = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    uint8_t* row = c.k + ((slot << c.log_page) + t0) * D + lane * CH;
    if (whole) {
#pragma unroll
      for (int t = 0; t < kGranule; ++t) {
        if constexpr (CH == 4)
          *reinterpret_cast<uint32_t*>(row + t * D) =
              kv_codes<FMT>(value(t, 0), value(t, 1), value(t, 2), value(t, 3));
        else
          *reinterpret_cast<uint16_t*>(row + t * D) =
              static_cast<uint16_t>(kv_codes<FMT>(value(t, 0), value(t, 1), 0.f, 0.f));
      }
      return;
    }
#pragma unroll
    for (int t = 0; t < kGranule; ++t) {
      const int tok = t0 + t;
      if (tok < from || tok >= hi) continue;
      uint32_t code;
      if constexpr (CH == 4) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(row + t * D);
        code = tok >= lo ? kv_codes<FMT>(value(t, 0), value(t, 1), value(t, 2), value(t, 3))
                         : rescaled<FMT>(*dst, s0, inv);
        *dst = code;
      } else {
        uint16_t* dst = reinterpret_cast<uint16_t*>(row + t * D);
        code = tok >= lo ? kv_codes<FMT>(value(t, 0), value(t, 1), 0.f, 0.f)
                         : rescaled<FMT>(*dst, s0, inv);
        *dst = static_cast<uint16_t>(code);
      }
    }
  }
}

template <int FMT, int D>
cudaError_t launch_append(const Kv8Cache& c, const Kv8Batch& bt, const __nv_bfloat16* k,
                          const __nv_bfloat16* v, int64_t ldk, int64_t ldv, cudaStream_t stream,
                          unsigned* err) {
  const int page = 1 << c.log_page;
  const int touched = (bt.max_new + page - 2) / page + 1;  // pages of one sequence, at most
  const int64_t units = static_cast<int64_t>(bt.batch) * touched * c.heads * 2;
  const int per_cta = (kAppendThreads / 32) * kGranule / page;
  const int64_t grid = (units + per_cta - 1) / per_cta;
  if (grid > 0x7FFFFFFF || static_cast<int64_t>(bt.batch) * touched > 0x7FFFFFFF)
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_append_kernel<FMT, D>, c, bt, k, v, ldk, ldv, touched, units,
                            err);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Cache& c, const Kv8Batch& bt, const void* k, const void* v,
                              int64_t ldk, int64_t ldv, int D, int fmt, cudaStream_t stream,
                              unsigned* err) {
  const auto* kp = static_cast<const __nv_bfloat16*>(k);
  const auto* vp = static_cast<const __nv_bfloat16*>(v);
  if (fmt == kKvInt8)
    return D == 64 ? launch_append<kKvInt8, 64>(c, bt, kp, vp, ldk, ldv, stream, err)
                   : launch_append<kKvInt8, 128>(c, bt, kp, vp, ldk, ldv, stream, err);
  return D == 64 ? launch_append<kKvE4m3, 64>(c, bt, kp, vp, ldk, ldv, stream, err)
                 : launch_append<kKvE4m3, 128>(c, bt, kp, vp, ldk, ldv, stream, err);
}

}  // namespace w4
