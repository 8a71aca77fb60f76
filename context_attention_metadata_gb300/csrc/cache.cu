// The paged key-value cache: rows written into it, quantised on the way, and read back.
//
// With `top` the largest |channel| of a token's head, x a channel:
//   e4m3:  s = 2^e, the smallest with top <= 448 s;   code = x / s rounded to e4m3
//   int8:  s = top / 127;                             code = x * 127 / top rounded to an integer
// and back: bf16(code * s).
//
// Bound by memory: 2 bytes a channel on one side, 2 or 1 on the other.  A thread holds 16 channels
// of a head, d / 16 lanes a head, so that `top` is a butterfly and a code's store or load is 16
// bytes.  A CTA takes a tile of up to 16 rows: one warp finds where the next tile's tokens are cached
// (a chain of three loads, a lane each) while all move the present one's heads, a warp one head
// of k or v of all rows.  Those are contiguous in a page, and the warps' heads are contiguous in
// the rows, so that both sides' accesses fall together: with a warp for all heads of a row the
// figures below were 271, 324 and 293 us.  Measured, heads of 8 x 128: 213,194 rows in plan order into
// e4m3 208 us (6.35 TB/s, 95% of a plain copy's rate), into bf16 268 (97%); 262,144 rows out of int8
// 250 us (97%), out of bf16 328 (98%).
#include <algorithm>
#include <cstring>

#include "seqs.cuh"

namespace marble {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 16;  // rows of a CTA's tile, at most
constexpr int kLooks = 4;  // sequences that a thread looks over at a time

struct CachePart {
  char* rows;              // bf16 [n, hkv, d], null: not in the call
  char* pages;
  float* scale;
  long long row_bytes, page_bytes, scale_stride;
};

struct CacheParams {
  CachePart part[2];       // k, v
  SeqsParams seqs;
  const int32_t* perm;     // plan index -> original index, or null
  int hkv;
  int run;                 // rows of a tile
  unsigned ctas;           // that move rows
};

// where the token of row i is: its page (-1: none, -2: the row belongs to no sequence) and slot
struct Place {
  int page, slot;
};
__device__ __forceinline__ Place place_of(const SeqsParams& s, long long row) {
  int b = (int)row;
  if (s.start) {
    // the sequence whose rows end first behind `row`
    int lo = 0, hi = s.n_seqs;
    while (lo < hi) {
      const int mid = lo + ((hi - lo) >> 1);  // (the sum may pass 2^31)
      if (__ldg(s.start + mid + 1) <= row) lo = mid + 1; else hi = mid;
    }
    b = lo;
  }
  if (b >= s.n_seqs) return {-2, 0};
  const Seq q = seq_at<true>(s, b);
  const long long at = row - q.first;
  if (at < 0 || at >= q.count) return {-2, 0};
  const long long pos = (long long)q.len - q.count + at;
  if (pos < 0) return {-1, 0};
  const int page = page_at(s, b, (int)pos);
  if (page < 0) seqs_bad(s);
  return {page, (int)(pos % s.page)};
}

__device__ __forceinline__ uint32_t hmax2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// the largest |channel| of a head, as bf16 bits (a NaN's if there is one)
template <int D>
__device__ __forceinline__ uint32_t top_bits(const uint32_t (&w)[8]) {
  uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = hmax2_nan(m, w[i] & 0x7fff7fffu);
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) m = hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  return hmax2_nan(m, m >> 16 | m << 16) & 0xffffu;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bf16 channels -> 16 codes; the scale of their head
template <int D, int kType>
__device__ __forceinline__ uint4 quantise(const uint32_t (&w)[8], float* scale) {
  const uint32_t top = top_bits<D>(w);
  uint32_t c[4] = {0, 0, 0, 0};
  if (top >= 0x7f80u) {
    *scale = __uint_as_float(0x7fc00000u);
    return make_uint4(0, 0, 0, 0);
  }
  if constexpr (kType == MARBLE_CACHE_E4M3) {
    // 448 = 1.75 * 2^8; top's mantissa (7 bits) says whether its binade reaches beyond
    const int e = max((int)(top >> 7) - ((top & 0x7fu) <= 0x60u ? 8 : 7), 1);
    *scale = top ? __uint_as_float((uint32_t)e << 23) : 0.f;
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint16_t two;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(two)
          : "f"(hi_f(w[i]) * inv), "f"(lo_f(w[i]) * inv));
      c[i >> 1] |= (uint32_t)two << (16 * (i & 1));
    }
  } else {
    *scale = __fdiv_rn(__uint_as_float(top << 16), 127.f);
    // In units of 2^e, in which top is `at`, in [1, 2) (less for a top below 2^-119), y = x * 127
    // has 15 bits, at 8.  The quotient is estimated and put right by one Newton step: what the
    // estimate leaves, rest, is exact (two of the estimate's last places times at), so the step is
    // off by 2^-22 of a last place before it is rounded.  A quotient halfway between whole
    // numbers is therefore met exactly, and the others lie 2^-17 or more away from halfway, where a
    // last place is 2^-17 at most: the sum below rounds every one as the exact quotient.
    const int e = max((int)(top >> 7) - 127, -119);
    const float one = e < 127 ? __uint_as_float((uint32_t)(127 - e) << 23) : 0x1p-127f;
    const float at = __uint_as_float(top << 16) * one, r = top ? __frcp_rn(at) : 0.f;
    const float by = 127.f * one;
    constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it leaves the nearest integer
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      uint32_t m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t two = w[(i + k) >> 1];
        const float y = (k & 1 ? hi_f(two) : lo_f(two)) * by, q = y * r;
        const float rest = fmaf(-q, at, y);
        m[k] = __float_as_uint(fmaf(rest, r, q) + kWhole);
      }
      c[i >> 2] = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
    }
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// 16 codes and their head's scale -> 16 bf16 channels
template <int kType>
__device__ __forceinline__ void restore(const uint4& codes, float scale, uint32_t (&w)[8]) {
  const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    if constexpr (kType == MARBLE_CACHE_E4M3) {
      halves_to_float(e4m3_halves(c[i >> 1] >> (16 * (i & 1))), &lo, &hi);
    } else {
      // the byte above 2^23 with its sign bit turned is 2^23 + 128 + code
      const uint32_t u = c[i >> 1] ^ 0x80808080u;
      lo = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 | (2 * (i & 1)))) - 8388736.f;
      hi = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 | (2 * (i & 1) + 1))) - 8388736.f;
    }
    w[i] = pack_bf16(lo * scale, hi * scale);
  }
}

// Sequences that no row leads to may be out of bounds too.  Several a time, whose loads are under way
// together.
__device__ __forceinline__ void look_over(const SeqsParams& s, int cta, int ctas) {
  bool off = false;
#pragma unroll kLooks
  for (long long b = cta * kThreads + threadIdx.x; b < s.n_seqs; b += ctas * kThreads)
    off |= seq_off(s, __ldg(s.lens + b), __ldg(s.start + b), __ldg(s.start + b + 1));
  if (off) seqs_bad(s);
}

// kLook: there are CTAs behind those of the rows that look the sequences over.  (A variant of its
// own, as the e4m3 write is at the limit of its registers: with them in
// one kernel the large write above takes 209.4 instead of 208.4 us, inlined among the rows' 212.)
template <int D, int kType, bool kWrite, bool kLook>
__global__ void __launch_bounds__(kThreads, 4) k_cache(const __grid_constant__ CacheParams p) {
  constexpr int kTpr = D / 16, kRows = 32 / kTpr, kEs = kType == MARBLE_CACHE_BF16 ? 2 : 1;
  // passes of kRows rows whose loads are under way together (of 1, 2 and 4, by time: more loads do
  // not help, where the accesses of a CTA lie close together does)
  constexpr int kPasses = kWrite ? (kEs == 2 ? 2 : 4) : (kEs == 2 ? 1 : 2);
  __shared__ Place places[2][kRun];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % kTpr, sub = lane / kTpr;
  const SeqsParams& s = p.seqs;
  if (kLook && blockIdx.x >= p.ctas) {
    look_over(s, blockIdx.x - p.ctas, gridDim.x - p.ctas);
    return;
  }
  const int ctas = kLook ? p.ctas : gridDim.x;
  const int tiles = (int)((s.n + p.run - 1) / p.run);
  const int steps = (p.run + kRows * kPasses - 1) / (kRows * kPasses);  // of a head's rows
  auto look = [&](int tile, int buf) {
    const long long i = (long long)tile * p.run + lane;
    if (tile < tiles && lane < p.run)
      places[buf][lane] = i < s.n ? place_of(s, p.perm ? p.perm[i] : i) : Place{-2, 0};
  };
  if (warp == 0) look(blockIdx.x, 0);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += ctas, buf ^= 1) {
    __syncthreads();
    if (warp == 0) look(tile + ctas, buf ^ 1);
    const long long i0 = (long long)tile * p.run;
    for (int unit = warp; unit < steps * 2 * p.hkv; unit += kWarps) {
      const int step = unit % steps, x = unit / steps & 1, h = unit / steps >> 1;
      const CachePart& c = p.part[x];
      if (!c.rows) continue;
      const int r0 = step * kRows * kPasses + sub;
      char* const row = c.rows + (i0 + r0) * c.row_bytes + ((long long)h * D + 16 * j) * 2;
      uint4 a[kPasses][kEs == 2 || kWrite ? 2 : 1];
      float scale[kPasses];
      Place at[kPasses];
#pragma unroll
      for (int u = 0; u < kPasses; ++u) {
        const int r = r0 + u * kRows;
        at[u] = r < p.run ? places[buf][r] : Place{-2, 0};
        const bool there = at[u].page >= 0;
        if constexpr (kWrite) {
          const uint4* src = reinterpret_cast<const uint4*>(row + (long long)u * kRows * c.row_bytes);
          a[u][0] = there ? __ldg(src) : make_uint4(0, 0, 0, 0);
          a[u][1] = there ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
        } else {
          const long long slot = (long long)h * s.page + at[u].slot;
          const uint4* src = reinterpret_cast<const uint4*>(c.pages + at[u].page * c.page_bytes +
                                                            (slot * D + 16 * j) * kEs);
          a[u][0] = there ? __ldg(src) : make_uint4(0, 0, 0, 0);
          if constexpr (kEs == 2) a[u][1] = there ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
          if constexpr (kEs == 1) scale[u] = there ? c.scale[at[u].page * c.scale_stride + slot] : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < kPasses; ++u) {
        if constexpr (kWrite) {
          const long long slot = (long long)h * s.page + at[u].slot;
          uint4* dst = reinterpret_cast<uint4*>(c.pages + at[u].page * c.page_bytes +
                                                (slot * D + 16 * j) * kEs);
          if constexpr (kEs == 2) {
            if (at[u].page >= 0) {
              dst[0] = a[u][0];
              dst[1] = a[u][1];
            }
          } else {
            const uint32_t v[8] = {a[u][0].x, a[u][0].y, a[u][0].z, a[u][0].w,
                                   a[u][1].x, a[u][1].y, a[u][1].z, a[u][1].w};
            float sc;
            const uint4 codes = quantise<D, kType>(v, &sc);
            if (at[u].page >= 0) {
              *dst = codes;
              if (j == 0) c.scale[at[u].page * c.scale_stride + slot] = sc;
            }
          }
        } else if (at[u].page != -2) {
          uint4* dst = reinterpret_cast<uint4*>(row + (long long)u * kRows * c.row_bytes);
          if constexpr (kEs == 1) {
            uint32_t o[8];
            restore<kType>(a[u][0], scale[u], o);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
          } else {
            dst[0] = a[u][0];
            dst[1] = a[u][1];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache(bool write, const marble_plan_t* plan, int64_t n, const marble_cache_t* c,
                         const marble_seqs_t* seqs, const marble_heads_t* rows, cudaStream_t s) {
  CacheParams p;
  memset(&p, 0, sizeof(p));
  const int es = c->type == MARBLE_CACHE_BF16 ? 2 : 1;
  p.part[0] = CachePart{static_cast<char*>(rows->k), static_cast<char*>(c->k), c->k_scale,
                        rows->k_stride * 2, c->k_stride * es, c->k_scale_stride};
  p.part[1] = CachePart{static_cast<char*>(rows->v), static_cast<char*>(c->v), c->v_scale,
                        rows->v_stride * 2, c->v_stride * es, c->v_scale_stride};
  p.seqs = seqs_params(*seqs, *c, n);
  p.perm = plan ? plan->perm : nullptr;
  p.hkv = c->hkv;
  // Tiles of up to kRun rows, fewer where that leaves SMs without work; as many CTAs as run at once,
  // or fewer that take the same number of rounds.  With start and a status, one CTA for 1024
  // sequences beside them (without start each sequence has its row).
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.run = kRun;
  while (p.run > 512 / c->d && n < (int64_t)p.run * sms * 4) p.run /= 2;
  const int64_t lookers = !seqs->start || !seqs->status ? 0
                          : std::min<int64_t>((seqs->n_seqs - 1) / (kThreads * kLooks) + 1, sms);
  const int64_t tiles = (n + p.run - 1) / p.run, most = (int64_t)sms * 4 - (lookers ? 1 : 0);
  const int64_t rounds = (tiles + most - 1) / most;
  p.ctas = (unsigned)((tiles + rounds - 1) / rounds);
  const unsigned grid = (unsigned)(p.ctas + lookers);
  auto pick = [&](auto dd, auto ll) {
    constexpr int D = decltype(dd)::value;
    constexpr bool L = decltype(ll)::value;
    if (c->type == MARBLE_CACHE_BF16)
      return write ? k_cache<D, MARBLE_CACHE_BF16, true, L> : k_cache<D, MARBLE_CACHE_BF16, false, L>;
    if (c->type == MARBLE_CACHE_E4M3)
      return write ? k_cache<D, MARBLE_CACHE_E4M3, true, L> : k_cache<D, MARBLE_CACHE_E4M3, false, L>;
    return write ? k_cache<D, MARBLE_CACHE_INT8, true, L> : k_cache<D, MARBLE_CACHE_INT8, false, L>;
  };
  auto at_d = [&](auto ll) {
    return c->d == 128 ? pick(std::integral_constant<int, 128>{}, ll)
                       : pick(std::integral_constant<int, 64>{}, ll);
  };
  auto kernel = lookers ? at_d(std::true_type{}) : at_d(std::false_type{});
  kernel<<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace marble
