// New keys and values into the 8-bit paged cache (layout: kv8.cuh).
//
// For every page and kv head that a new token falls into, with a the largest
// magnitude of the page's new tokens and s0 the page's scale (0 where the
// page held no earlier token of the sequence):
//
//   s = max(s0, up(a / qmax)),  up: the next fp32 value that bf16 holds
//   new codes      round(x / s)                (ties to even; s = 0: 0)
//   earlier codes  round(code * s0 / s)        only where s > s0
//
// With s of 8 significant bits every rounding is decided exactly: a code's
// rounding border times s has at most 16 bits, code * s0 at most 16, so a
// product is exact in fp32 and the correctly rounded quotient lies on its
// border only if the true one does.
//
// One CTA per (sequence, page it touches, kv head); keys and values are two
// CTAs (blockIdx.z).  The page's new rows pass through shared memory as
// bf16: rows are read as they lie in x, and written as they lie in the page
// (values turned: [channel][token]).  Bound: HBM / L2 (2 bytes read and 1
// written per element), for single tokens launch latency.
#include "kv8.cuh"
#include "w4_kernels.h"

namespace w4 {

namespace {

constexpr int kAppendThreads = 128;
constexpr unsigned kKernelIdAppend = 16;

template <int FMT>
__device__ __forceinline__ uint32_t kv_code(float v) {
  if constexpr (FMT == kKvInt8) {
    const int q = __float2int_rn(v);
    return static_cast<uint32_t>(min(127, max(-127, q))) & 0xFFu;
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
    return r & 0xFFu;
  }
}

template <int FMT>
__device__ __forceinline__ float kv_value(uint32_t code) {
  if constexpr (FMT == kKvInt8) {
    return static_cast<float>(static_cast<int8_t>(code));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xFFFFu)));
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads)
    kv8_append_kernel(const Kv8Cache c, const Kv8Batch bt, const __nv_bfloat16* __restrict__ k,
                      const __nv_bfloat16* __restrict__ v, int64_t ldk, int64_t ldv,
                      unsigned* err) {
  // New rows [token][channel]; a row is padded by one 4-byte word so that a
  // column walk (values) hits distinct banks.
  extern __shared__ uint32_t tile[];
  constexpr int kRowWords = D / 2 + 1;
  __shared__ float red[kAppendThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x / c.heads, h = blockIdx.x % c.heads;
  const bool is_v = blockIdx.z != 0;
  const int page_size = 1 << c.log_page;
  const Kv8Seq s = kv8_sequence(bt, b, c.log_page);
  if (s.bad && threadIdx.x == 0 && blockIdx.y == 0) record_error(err, kErrBadIndex, kKernelIdAppend);
  const int old = s.len > s.n ? s.len - s.n : 0;
  const int skip = s.n - (s.len - old);  // new tokens in front of position 0: not held
  const int j = (old >> c.log_page) + static_cast<int>(blockIdx.y);  // page of the sequence
  const int64_t p0 = static_cast<int64_t>(j) << c.log_page;
  if (s.n == 0 || p0 >= s.len) return;
  const int lo = old > p0 ? static_cast<int>(old - p0) : 0;  // new tokens [lo, hi) of the page
  const int hi = s.len - p0 < page_size ? static_cast<int>(s.len - p0) : page_size;
  const int page = bt.table[static_cast<int64_t>(b) * bt.max_pages + j];
  if (page < 0 || page >= c.num_pages) {
    if (threadIdx.x == 0) record_error(err, kErrBadIndex, kKernelIdAppend);
    return;
  }
  const int64_t row0 = static_cast<int64_t>(s.row0) + skip + (p0 + lo - old);
  const __nv_bfloat16* x = (is_v ? v : k) + static_cast<int64_t>(h) * D;
  const int64_t ld = is_v ? ldv : ldk;
  const int64_t slot = static_cast<int64_t>(page) * c.heads + h;
  uint8_t* out = (is_v ? c.v : c.k) + (slot << c.log_page) * D;
  float* scale = (is_v ? c.vs : c.ks) + slot;

  // Rows into shared memory, and their largest magnitude.
  const int n_new = hi - lo;
  float amax = 0.f;
  constexpr int kChunks = D / 8;
  for (int e = threadIdx.x; e < n_new * kChunks; e += kAppendThreads) {
    const int r = e / kChunks, ch = e % kChunks;
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(x + (row0 + r) * ld) + ch);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tile[r * kRowWords + 4 * ch + i] = u[i];
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[i] << 16)),
                               fabsf(__uint_as_float(u[i] & 0xFFFF0000u))));
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  const float s0 = lo > 0 ? *scale : 0.f;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const float up = __uint_as_float(
      (__float_as_uint(__fdiv_rn(amax, kv8_qmax(FMT))) + 0xFFFFu) & 0xFFFF0000u);
  const float s1 = fmaxf(s0, up);
  if (threadIdx.x == 0) *scale = s1;

  const bool again = lo > 0 && s1 > s0;
  auto element = [&](int t, int d) {  // token t of the page, channel d
    const uint32_t u = tile[(t - lo) * kRowWords + d / 2];
    return __uint_as_float((d & 1) ? (u & 0xFFFF0000u) : (u << 16));
  };
  // The page's bytes in words of four along its contiguous axis: every word
  // that holds a new token, and those of earlier ones where the scale grew.
  const int words = is_v ? D * page_size / 4 : hi * (D / 4);
  const int w0 = is_v ? 0 : (again ? 0 : lo * (D / 4));
  uint32_t* ow = reinterpret_cast<uint32_t*>(out);
  const int log_vw = c.log_page - 2;  // words of a value row
  for (int w = w0 + threadIdx.x; w < words; w += kAppendThreads) {
    int t, d;
    if (is_v) {
      d = w >> log_vw;
      t = (w & ((1 << log_vw) - 1)) * 4;
      if (t >= hi || (t + 4 <= lo && !again)) continue;
    } else {
      t = w / (D / 4);
      d = (w % (D / 4)) * 4;
    }
    const bool mixed = is_v ? t < lo || t + 4 > hi : t < lo;
    uint32_t before = mixed ? ow[w] : 0u, after = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ti = is_v ? t + i : t, di = is_v ? d : d + i;
      uint32_t code = (before >> (8 * i)) & 0xFFu;
      if (ti >= lo && ti < hi)
        code = s1 > 0.f ? kv_code<FMT>(__fdiv_rn(element(ti, di), s1)) : 0u;
      else if (ti < lo && again)
        code = kv_code<FMT>(__fdiv_rn(__fmul_rn(kv_value<FMT>(code), s0), s1));
      after |= code << (8 * i);
    }
    ow[w] = after;
  }
}

template <int FMT, int D>
cudaError_t launch_append(const Kv8Cache& c, const Kv8Batch& bt, const __nv_bfloat16* k,
                          const __nv_bfloat16* v, int64_t ldk, int64_t ldv, cudaStream_t stream,
                          unsigned* err) {
  const int page = 1 << c.log_page;
  const int touched = (bt.max_new + page - 2) / page + 1;
  const int most = bt.max_new < page ? bt.max_new : page;
  const size_t smem = static_cast<size_t>(most) * (D / 2 + 1) * 4;  // at most 33 KB
  constexpr auto kern = kv8_append_kernel<FMT, D>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(bt.batch) * c.heads, touched, 2);
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, c, bt, k, v, ldk, ldv, err);
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
