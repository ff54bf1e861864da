// Shared definitions of the 8-bit paged KV cache kernels.
//
// Layout: keys [page][kv head][token in page][channel], values
// [page][kv head][channel][token in page], one byte each (int8 or e4m3), and
// one fp32 scale for each page and kv head of either side.  With both sides
// contiguous along the axis that their product sums over, 16 bytes of a key
// row (channels) and 16 bytes of a value row (tokens) are each an operand
// fragment that a lane can use as loaded.
#pragma once

#include "w4_common.cuh"

namespace w4 {

enum : int { kKvInt8 = 0, kKvE4m3 = 1 };

// Device error word, bit 1: a page id, a length or a row offset outside the
// caller's buffers was met; what it addressed was skipped.
constexpr unsigned kErrBadIndex = 2u;

__host__ __device__ constexpr float kv8_qmax(int fmt) { return fmt == kKvInt8 ? 127.f : 448.f; }

// Asynchronous copies of 16 bytes (zeros unless live), waited for by the lane
// that issued them.
__device__ __forceinline__ void kv8_copy16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void kv8_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void kv8_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 kv8_lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Four codes -> two packed pairs of fp16 values.
template <int FMT>
__device__ __forceinline__ void kv8_codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
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

struct Kv8Cache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int num_pages, heads, log_page;
};

struct Kv8Batch {
  const int32_t* table;   // [batch, max_pages]
  const int32_t* lens;    // [batch] tokens in the cache, the new ones included
  const int32_t* starts;  // [batch + 1] rows of the new tokens; NULL: row b alone
  int batch, max_pages, rows;  // rows: of the q / k / v buffers
  int max_new;
};

// One sequence's length, new tokens and first row, checked against the
// buffers: anything outside them counts as no new tokens.
struct Kv8Seq {
  int len, n, row0;
  bool bad;
};

__device__ __forceinline__ Kv8Seq kv8_sequence(const Kv8Batch& p, int b, int log_page) {
  Kv8Seq s;
  s.len = p.lens[b];
  s.row0 = p.starts ? p.starts[b] : b;
  const int end = p.starts ? p.starts[b + 1] : b + 1;
  const int64_t room = static_cast<int64_t>(p.max_pages) << log_page;
  s.bad = s.len < 0 || s.len > room || s.row0 < 0 || end < s.row0 || end > p.rows ||
          static_cast<int64_t>(end) - s.row0 > p.max_new;
  s.n = s.bad ? 0 : end - s.row0;
  if (s.bad) s.len = 0;
  return s;
}

}  // namespace w4
