// What the cache kernels share: the sequences of a batch, and where a row's token is cached.
#pragma once

#include <climits>

#include "common.cuh"
#include "internal.h"

namespace marble {

struct SeqsParams {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* start;  // null: one row a sequence
  int32_t* status;       // or null
  long long table_stride, n;
  int n_seqs, page, n_pages;
  int top;               // positions that the table reaches
};

inline SeqsParams seqs_params(const marble_seqs_t& s, const marble_cache_t& c, int64_t n) {
  SeqsParams p;
  p.table = s.table;
  p.lens = s.lens;
  p.start = s.start;
  p.status = s.status;
  p.table_stride = s.table_stride;
  p.n = n;
  p.n_seqs = s.n_seqs;
  p.page = c.page_tokens;
  p.n_pages = (int)c.n_pages;
  // (so far below 2^31 that a chunk's last position still is)
  const int64_t top = (int64_t)s.table_pages * c.page_tokens, most = INT_MAX - 65535;
  p.top = (int)(top < most ? top : most);
  return p;
}

static_assert(kErrTimeout == MARBLE_SEQS_TIMEOUT, "waits set this bit of the status");

__device__ __forceinline__ void seqs_bad(const SeqsParams& p) {
  if (p.status) atomicOr(p.status, MARBLE_SEQS_BAD);
}

// The rows [first, first + count) and the length of sequence b, cut to what the arrays hold.
struct Seq {
  int first, count, len;
};
// is a sequence's length or its rows [s0, s1) out of bounds?
__device__ __forceinline__ bool seq_off(const SeqsParams& p, int len, int s0, int s1) {
  return len < 0 || len > p.top || s0 < 0 || s1 < s0 || s1 > (int)p.n;
}
template <bool kTell>
__device__ __forceinline__ Seq seq_at(const SeqsParams& p, int b) {
  const int len = p.lens[b];
  int s0 = b, s1 = b + 1;
  if (p.start) {
    s0 = p.start[b];
    s1 = p.start[b + 1];
  }
  const int n = (int)p.n;
  if (kTell && seq_off(p, len, s0, s1)) seqs_bad(p);
  Seq s;
  s.first = min(max(s0, 0), n);
  s.count = min(max(s1, s.first), n) - s.first;
  s.len = min(max(len, 0), p.top);
  return s;
}

// the table's entry for position `pos` of sequence b, and the page that it is (-1: none)
__device__ __forceinline__ int table_at(const SeqsParams& p, int b, int pos) {
  return __ldg(p.table + (int64_t)b * p.table_stride + pos / p.page);
}
__device__ __forceinline__ int page_at(const SeqsParams& p, int b, int pos) {
  const int g = table_at(p, b, pos);
  return (unsigned)g < (unsigned)p.n_pages ? g : -1;
}

// two e4m3 codes as halves, and those as fp32 (all exact)
__device__ __forceinline__ uint32_t e4m3_halves(uint32_t two) {  // low 16 bits
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(h)
      : "r"(two));
  return h;
}

__device__ __forceinline__ void halves_to_float(uint32_t h, float* lo, float* hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(*lo), "=f"(*hi)
      : "r"(h));
}

}  // namespace marble
