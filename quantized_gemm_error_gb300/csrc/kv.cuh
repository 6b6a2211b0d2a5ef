// kv.cuh -- device views of the paged key/value cache and of the sequences a
// call works on, and the address arithmetic shared by the kernels that write,
// move and read pages.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace spear {

// Launch of a kernel that begins with enter(): it may be set up while the
// kernel before it on the stream finishes (programmatic dependent launch), and
// reads and writes nothing before that one is done.
template <typename... P, typename... A>
inline int launch_dependent(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const char* what,
                            A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, fn, P(args)...), what);
}
__device__ __forceinline__ void enter() {
  pdl_launch_dependents();
  pdl_wait();
}

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 by a multiplication: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1 the quotient is
// (floor(m n / 2^32) + n) >> l; the sum stays below 2^32 because n < 2^31.
struct FastDiv {
  uint32_t d, m, l;
  __host__ static FastDiv of(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.l = 0;
    while ((1ull << f.l) < d) ++f.l;
    f.m = (uint32_t)(((1ull << 32) * ((1ull << f.l) - d)) / d + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

// The cache: element (page, head, slot, d) of K or V is at
// page page_stride + head head_stride + slot slot_stride + d (64-bit, in
// elements): a pool passes 2^31 elements at 4 GB.
struct KvView {
  const uint16_t* k;
  const uint16_t* v;
  int64_t page_stride, head_stride, slot_stride;
  FastDiv page;
  int num_pages, heads;
};

// The call's sequences: sequence b is row ids[b] (or b) of the block table.
struct SeqView {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* ids;
  int64_t table_stride;
  int n, max_pages, rows;
};

inline KvView kv_view(const spear_kv_cache& c) {
  return {c.k, c.v, c.page_stride, c.head_stride, c.slot_stride, FastDiv::of((uint32_t)c.page_size), c.num_pages,
          c.num_kv_heads};
}
inline SeqView seq_view(const spear_kv_seqs& s) {
  return {s.block_table, s.seq_lens, s.seq_ids, s.table_stride, s.num_seqs, s.max_pages, s.table_rows};
}

// Row of sequence b, or -1 (recorded) where seq_ids names none.
__device__ __forceinline__ int seq_row(const SeqView& s, int b, unsigned* status) {
  const int r = s.ids ? s.ids[b] : b;
  if (r < 0 || r >= s.rows) {
    record_status(status, DEV_ERR_INVALID);
    return -1;
  }
  return r;
}
// Length of that row, at most what its table row can hold.
__device__ __forceinline__ int seq_len(const SeqView& s, const KvView& c, int row, unsigned* status) {
  if (row < 0) return 0;
  const int n = s.lens[row];
  const long long cap = (long long)s.max_pages * c.page.d;
  if (n < 0 || n > cap) {
    record_status(status, DEV_ERR_INVALID);
    return n < 0 ? 0 : (int)cap;
  }
  return n;
}
// Offset of cached row (pos, head 0), or -1 (recorded) where the table names no page.
__device__ __forceinline__ int64_t kv_row_offset(const KvView& c, const int32_t* table_row, int pos,
                                                 unsigned* status) {
  const uint32_t pg = c.page.div((uint32_t)pos);
  const int p = table_row[pg];
  if ((unsigned)p >= (unsigned)c.num_pages) {
    record_status(status, DEV_ERR_INVALID);
    return -1;
  }
  return (int64_t)p * c.page_stride + (int64_t)(pos - (int)(pg * c.page.d)) * c.slot_stride;
}

// The keys a token at position `pos` sees, as two ranges [0, sink_end) and
// [win_begin, pos] (sink_end <= win_begin; without a window all in the second).
struct Visible {
  int sink_end, win_begin;
};
__device__ __forceinline__ Visible visible_keys(int pos, int window, int sinks) {
  Visible r{0, 0};
  if (window > 0 && pos >= window) {
    r.win_begin = pos - window + 1;
    r.sink_end = min(sinks, r.win_begin);
  }
  return r;
}

__device__ __forceinline__ float f16_bits_to_f32(uint16_t b) { return __half2float(__ushort_as_half(b)); }
template <bool F16>
__device__ __forceinline__ float elem_to_f32(uint16_t b) {
  return F16 ? f16_bits_to_f32(b) : __uint_as_float((uint32_t)b << 16);
}
// Two floats rounded to nearest even, `lo` in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t pack_elem2(float lo, float hi) {
  if (F16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}

constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes to shared memory, zeros where there are none.
__device__ __forceinline__ void cp_async16_zfill(uint32_t s, const void* g, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(g), "r"(valid ? 16 : 0) : "memory");
}
// p / z for 0 <= p < 2^63 and z > 0; in 32 bits where both fit.
__device__ __forceinline__ long long divide(long long p, long long z) {
  if ((((unsigned long long)p | (unsigned long long)z) >> 32) == 0) return (uint32_t)p / (uint32_t)z;
  return (long long)((unsigned long long)p / (unsigned long long)z);
}

}  // namespace spear
