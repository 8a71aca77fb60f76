// Attention of every sequence's last tokens over its paged, cached keys and values.
//
//   s_j = scale q.k_j (capped, lowered by a slope times the distance, in base 2),
//   m = running maximum, p_j = 2^(s_j - m), l = sum p_j, O = sum p_j v_j,   o = O / l.
//
// Bound by memory for few rows (new tokens x q heads of a group) of a kv head: every key and value
// is read once, at 2 or 1 bytes a channel.  One sequence of 1,048,576 tokens, 8 kv heads of
// 128, microseconds, and the time that a plain copy's rate gives:
//   rows        4       12      20      64     copy
//   bf16       593     628     657    1142      642
//   e4m3       336     388     580    1115      331
//   int8       338     398     600    1159      331
// and with heads of 64, 4 rows: bf16 306 (321), e4m3 180 to 184 (171).  From 12 rows on for 8-bit
// types, above 20 for bf16, the computing warps' instructions are the bound.
//
// - An item is a (sequence, kv head, tile of 8, 16, 32 or 64 rows); its cost is its chunks of keys
//   and a constant.  Every CTA takes an equal range of the sum of all costs, so that ragged
//   batches keep all SMs busy to the end; it finds its range from the sequences' lengths itself.
//   An item that a range cuts leaves unnormalised pieces (O, m, l) in the workspace, at most two a
//   CTA whatever the batch, and a second kernel, already launched when the first ends, joins
//   them in order.
// - A CTA is a warp that fetches (page table look-ups, chunks by TMA into a ring, the next pieces'
//   q) and four that compute; two CTAs share an SM, so that one's item boundaries hide behind
//   the other's streaming.
// - A chunk belongs to one warp of the item's 8 or 16 rows (two or four where there are more rows):
//   warps have their own m, l and O over their chunks and meet only at an item's end.  Where the
//   batch has items of more than 16 rows, those of fewer still have their keys dealt to all four
//   warps.  A place of the ring then passes between warps, and one that waits for its next
//   filling has to know that the one before is over, or the barrier's parity misleads it: the
//   fetching warp tells how many chunks it has issued.
// - The products are m16n8k16 matrix instructions with the keys (channels) as the 16 rows and the q
//   rows as the 8 columns: tcgen05's 128 x 8 would have the same shape, but its operands come from
//   shared memory, where 8-bit codes would have to be written as fp16 first, and what memory
//   feeds for 8 rows is 15% of the warp-level instructions' rate.  (e4m3 products with
//   q in two e4m3 terms were exact too, but slower: twice the sums.)
// - 8-bit codes become fp16 exactly in registers; k's scales multiply scores, v's scales the
//   weights, so that nothing but the weights (and q, by a power of two a row) is rounded to fp16.
#pragma once

#include <math.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "score.cuh"
#include "seqs.cuh"
#include "tma_host.h"

namespace marble {
namespace cached {

constexpr int kWorkers = 4;   // computing warps
// One more warp fetches; it has three idle ones beside it, so that registers can be moved between
// two groups of four warps: of the 128 a thread that two CTAs on an SM leave, the computing warps
// get 200 (five warps alone could have no more than 168, which 16 rows of 128 channels spill).
constexpr int kThreads = 64 * kWorkers;
constexpr int kFetchRegs = 56, kWorkRegs = 200;
constexpr int kUnitOver = 3;  // an item's constant cost, in chunks (1 to 6: 3 and 4 are the fastest)
constexpr int kMergeArrivals = 6;  // of the warps whose O is handed over: 3 or 2
constexpr float kLazy = 8.f;  // O is rescaled when m grows by more (base 2)
constexpr float kPUp = 64.f;  // fp16 weights are raised by this (see below)
constexpr uint32_t kLeastUnit = (127 - 120) << 23;  // 2^-120 as fp32's bits: v's scales' least unit

// kNt: tiles of 8 rows that a warp computes
template <int D, int kType, int kNt>
struct Cfg {
  static constexpr bool kQuant = kType != MARBLE_CACHE_BF16;
  static constexpr int kRow = D * (kQuant ? 1 : 2);          // bytes of a key
  static constexpr int kPitch = kRow > 128 ? 128 : kRow;     // of its rows in shared memory
  static constexpr int kHalves = kRow / kPitch;
  static constexpr int kKeys = kRow > 128 ? 32 : 64;         // of a chunk
  // keys that a warp works on at once: what its registers hold beside O and q
  static constexpr int kSub = kNt == 2 && kQuant && D == 128 ? 32 : kKeys;
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kStages = kTile == 8192 ? 4 : 8;
  static_assert(kStages % kWorkers == 0, "a place keeps its warps while chunks are dealt the same way");
  static constexpr int kScales = kQuant ? kStages * 2 * kKeys * 4 : 0;
  // pieces that the fetching warp may be ahead; their q; the warps' O, m and l on their way together
  static constexpr int kPieces = kNt == 1 ? 4 : 2;
  static constexpr int kQPitch = D * 2 + 16;
  static constexpr int kMerge = 32 * (D / 4 * kNt + 4 * kNt) * 4;
  static constexpr int kMergeBufs = kNt == 1 ? 2 : 1;
  static constexpr int smem(int row_warps) {
    const int writers = row_warps == kWorkers ? 0 : kWorkers - 1;
    return 1024 + kStages * 2 * kTile + kScales + kPieces * 8 * kNt * row_warps * kQPitch +
           kMergeBufs * writers * kMerge;
  }
};

struct AttnParams {
  CUtensorMap kmap, vmap;
  SeqsParams seqs;
  const float* k_scale;
  const float* v_scale;
  long long k_scale_stride, v_scale_stride;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  long long q_stride, o_stride;
  const float* slopes;
  float scale2;      // scale * log2 e
  float inv_cap2;    // 1 / cap2
  float cap2;        // cap * log2 e, 0: none
  int hkv, group;
  int window, span;
  int row_warps;     // warps that an item's rows are split over, at most: 1, 2 or 4
  int rows, rows_log;  // of an item: 8 * kNt * row_warps
  int box;           // keys of a TMA box
  int grain;         // as many CTAs work as the sum of units holds grains, rounded up
  float* part_o;     // [2 * CTAs][rows][D] pieces
  float2* part_ml;   // [2 * CTAs][rows]
  int4* joins;       // [CTAs][2]: pieces (0: none), the sequence's first row and rows; kv head, first row
  unsigned* err;
  uint64_t limit_ns, drain_ns;
};

// one sequence's items: `items` of `units` each; all of them walk the chunks
// [chunk0, chunk0 + chunks) of the keys [lo, hi)
struct Work {
  Seq s;
  int lo, hi, chunk0, chunks, tiles, items;
  int weight;  // units of a chunk
  long long units;
};

// The time of a chunk by the rows of its item, in quarters: 8-bit items whose keys go to two warps at
// a time, among others whose keys go to four, take longer.
__device__ __forceinline__ int weight_of(const AttnParams& p, int count) {
  const long long rows = min((long long)count * p.group, (long long)p.rows);
  return !p.k_scale || p.row_warps == kWorkers || rows <= 16 ? 4 : 6;
}

// the positions that the row at `pos` sees: [lo, hi)
__device__ __forceinline__ void sees(const AttnParams& p, const Seq& s, int pos, int* lo, int* hi) {
  *lo = (int)max((long long)pos - p.window + 1, 0ll);
  *hi = pos + 1;
  if (p.span) {
    *lo = min(*lo, max(s.len - s.count, 0));
    *hi = s.len;
  }
  if (pos < 0) *lo = *hi = 0;
}

template <int kKeys, int kNt, bool kTell>
__device__ __forceinline__ Work work_of(const AttnParams& p, int b) {
  Work w;
  w.s = seq_at<kTell>(p.seqs, b);
  int hi;
  sees(p, w.s, max(w.s.len - w.s.count, 0), &w.lo, &hi);
  w.hi = p.window > 0 || p.span ? w.s.len : w.lo;  // (no window: no keys at all)
  w.chunk0 = w.lo / kKeys;
  w.chunks = w.lo < w.hi ? (w.hi - 1) / kKeys - w.chunk0 + 1 : 0;
  w.tiles = (int)(((long long)w.s.count * p.group + p.rows - 1) >> p.rows_log);
  w.items = w.tiles * p.hkv;
  w.weight = kNt == 1 ? 1 : weight_of(p, w.s.count);
  w.units = w.items ? (long long)(w.chunks + kUnitOver) * w.weight : 0;
  return w;
}

// a / b of non-negative numbers; most fit 32 bits, whose quotient takes a fifth of the time
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// chunks before offset x of an item
template <int kNt>
__device__ __forceinline__ int cut(const Work& w, long long x) {
  return (int)max((kNt == 1 ? x : quotient(x, w.weight)) - kUnitOver, 0ll);
}

// the walk over a CTA's range of units, piece by piece
template <int kKeys, int kNt>
struct Walk {
  const AttnParams& p;
  long long left, off;  // units left, those of the present item that are behind
  int b;
  Work w;
  // of the present piece
  int item, c0, c1;
  long long rest;       // units of its item behind it
  // from unit `at` of sequence b_ on
  __device__ __forceinline__ Walk(const AttnParams& p_, int b_, long long at, long long left_)
      : p(p_), left(left_), b(b_) {
    w = work_of<kKeys, kNt, false>(p, b);
    next_item = (int)quotient(at, w.units);
    off = at - next_item * w.units;
  }
  __device__ __forceinline__ bool next() {
    while (left > 0) {
      if (next_item >= w.items) {
        if (++b >= p.seqs.n_seqs) return false;
        w = work_of<kKeys, kNt, false>(p, b);
        next_item = 0;
        continue;
      }
      item = next_item;
      const long long from = off, to = min(w.units, from + left);
      left -= to - from;
      const bool ends = to == w.units;
      next_item += ends ? 1 : 0;
      off = ends ? 0 : to;
      rest = w.units - to;
      c0 = cut<kNt>(w, from);
      c1 = cut<kNt>(w, to);
      if (c1 > c0 || (w.chunks == 0 && from == 0)) return true;
    }
    return false;
  }

 private:
  int next_item;
};

__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
__device__ __forceinline__ void ldsm4_t(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// the 8 x 8 matrix of 16-bit values turned over
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// c += a b, 16 x 8 x 16, of halves or bf16
template <bool kHalf>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (!kHalf)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// int8 codes with their sign bits turned (128 + code) at bytes of `u` -> two halves
__device__ __forceinline__ uint32_t int8_halves(uint32_t u, uint32_t sel) {
  uint32_t h = __byte_perm(u, 0x64646464u, sel), r;  // 1024 + 128 + code
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}
// four codes of consecutive channels of one key: the halves of the first two, and the others
template <int kType>
__device__ __forceinline__ void along(uint32_t c, uint32_t* a, uint32_t* b) {
  if constexpr (kType == MARBLE_CACHE_E4M3) {
    *a = e4m3_halves(c);
    *b = e4m3_halves(c >> 16);
  } else {
    const uint32_t u = c ^ 0x80808080u;
    *a = int8_halves(u, 0x4140);
    *b = int8_halves(u, 0x4342);
  }
}
// codes (key 0: channels 0, 1; key 1: channels 0, 1): the halves of channel 0, and of channel 1
template <int kType>
__device__ __forceinline__ void across(uint32_t c, uint32_t* a, uint32_t* b) {
  if constexpr (kType == MARBLE_CACHE_E4M3) {
    const uint32_t x = __byte_perm(c, 0, 0x3120);
    *a = e4m3_halves(x);
    *b = e4m3_halves(x >> 16);
  } else {
    const uint32_t u = c ^ 0x80808080u;
    *a = int8_halves(u, 0x4240);
    *b = int8_halves(u, 0x4341);
  }
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// arrive `n` times
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, int n) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(n)
      : "memory");
}
__device__ __forceinline__ void store_release(int* at, int v) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(smem_u32(at)), "r"(v) : "memory");
}
__device__ __forceinline__ int load_acquire(const int* at) {
  int v;
  asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(at)) : "memory");
  return v;
}
// whole warp: until chunk `n` has been issued (bounded like the barriers' waits)
__device__ __forceinline__ bool wait_issued(const int* issued, int n, const WaitCtx& w) {
  if (__all_sync(0xffffffffu, load_acquire(issued) > n)) return true;
  const uint64_t t0 = globaltimer_ns();
  bool ok = true;
  while (ok && load_acquire(issued) <= n) {
    if (*w.abort) ok = false;
    if (globaltimer_ns() - t0 > w.limit_ns) {
      atomicOr(w.err, kErrTimeout);
      *w.abort = 1;
      ok = false;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// over the 8 lanes that hold a row's keys
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// ln of the sum, from a base-2 maximum and a sum
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// row `x` of a kv head's rows (new token by new token, the group's q heads of each): its token's
// row in the call, its q head and its position
struct RowAt {
  int token, head, pos;
  bool live;
};
__device__ __forceinline__ RowAt row_at(const AttnParams& p, const Seq& s, int head, int x) {
  const int t = x / p.group;
  RowAt a;
  a.live = t < s.count;
  a.token = s.first + t;
  a.head = head * p.group + (x - t * p.group);
  a.pos = s.len - s.count + t;
  return a;
}

// what the computing warps need of a piece
struct Piece {
  Seq s;
  int lo, hi;           // the item's keys
  int key0, chunks;     // the piece's first key and chunks; chunks < 0: there are no more pieces
  int head, row0;       // the item's kv head and first row
  int row_warps;        // warps that the item's rows are split over
  int place;            // where the piece goes in the workspace, -1: it is the whole item
};

template <int D, int kType, int kNt, bool kScored>
__global__ void __launch_bounds__(kThreads, 2) k_attn_cached(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, kType, kNt>;
  constexpr bool kQuant = C::kQuant;
  constexpr int kKeys = C::kKeys, kStages = C::kStages, kMt = C::kSub / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(ring + kStages * 2 * C::kTile);
  uint8_t* qs = reinterpret_cast<uint8_t*>(scales) + C::kScales;
  float4* merge = reinterpret_cast<float4*>(qs + C::kPieces * p.rows * C::kQPitch);
  __shared__ uint64_t full[kStages], empty[kStages], piece_full[C::kPieces], piece_empty[C::kPieces];
  __shared__ uint64_t merge_full[C::kMergeBufs], merge_empty[C::kMergeBufs];
  __shared__ Piece pieces[C::kPieces];
  __shared__ int2 looked[32];
  __shared__ longlong2 looked_scales[kQuant ? 32 : 1];
  __shared__ int abort_flag, first_b, told;
  __shared__ long long first_at, range[2], sums[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // let the joining kernel's CTAs come up beside this one's
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's range of units
  // (n_seqs is at least 1; no sum here passes 2^31)
  const int ns = p.seqs.n_seqs, share = (ns - 1) / kThreads + 1;
  const int b0 = min(tid * share, ns), b1 = b0 + min(share, ns - b0);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Work w = blockIdx.x == 0 ? work_of<kKeys, kNt, true>(p, b) : work_of<kKeys, kNt, false>(p, b);
    mine += w.units * w.items;
  }
  long long upto = mine;  // of this warp's threads up to this one
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, off);
    upto += lane >= off ? v : 0;
  }
  if (lane == 31) sums[warp] = upto;
  if (tid == 0) {
    abort_flag = 0;
    told = 0;
    p.joins[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    tma_prefetch_desc(&p.kmap);
    tma_prefetch_desc(&p.vmap);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], p.row_warps);
    }
    for (int i = 0; i < C::kPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], kWorkers);
    }
    for (int i = 0; i < C::kMergeBufs; ++i) {
      mbar_init(&merge_full[i], kMergeArrivals);
      mbar_init(&merge_empty[i], kWorkers);
    }
    fence_mbar_init();
  }
  __syncthreads();
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    before += i < warp ? sums[i] : 0;
    total += sums[i];
  }
  const long long ctas = min((long long)gridDim.x, quotient(total + p.grain - 1, p.grain));
  if (blockIdx.x >= ctas) return;
  const long long u0 = quotient(total * blockIdx.x, ctas), u1 = quotient(total * (blockIdx.x + 1), ctas);
  if (before <= u0 && u0 < before + mine) {
    long long at = u0 - before;
    int b = b0;
    for (; b < b1; ++b) {
      const Work w = work_of<kKeys, kNt, false>(p, b);
      if (at < w.units * w.items) break;
      at -= w.units * w.items;
    }
    first_b = b;
    first_at = at;
    range[0] = total;
    range[1] = ctas;
  }
  __syncthreads();
  const WaitCtx wait = {p.limit_ns, p.err, &abort_flag};

  if (warp >= kWorkers) {
    regs_shrink<kFetchRegs>();
    if (warp > kWorkers) return;
    // ---- fetch.  The boxes of the next 32 / boxes chunks are looked up at once, a lane each;
    // one thread then issues all copies (its operands are uniform; lanes side by side would be
    // taken one by one, at twice the cost).
    const int boxes = kKeys / p.box, group = 32 / boxes;
    const bool leader = elect_one();
    // table entry and slot of box j of the chunk i behind chunk c of a piece; no slot: not needed
    auto look = [&](int c, const Walk<kKeys, kNt>& walk, int i, int j) {
      int2 at = make_int2(-1, -1);
      const int key = (walk.w.chunk0 + c + i) * kKeys + j * p.box;
      if (c + i < walk.c1 && key < walk.w.hi && key + p.box > walk.w.lo) {
        at.x = table_at(p.seqs, walk.b, key);
        at.y = key % p.seqs.page;
      }
      return at;
    };
    Walk<kKeys, kNt> walk(p, first_b, first_at, u1 - u0);
    int n = 0, np = 0, issued = 0;  // chunks and pieces so far
    bool ok = true;
    while (ok) {
      const bool more = walk.next();
      const int ps = np % C::kPieces;
      if (np >= C::kPieces && !warp_wait(&piece_empty[ps], ((np / C::kPieces) & 1) ^ 1, wait)) {
        ok = false;
        break;
      }
      const Work& w = walk.w;
      const int head = more ? walk.item / w.tiles : 0;
      const int row0 = more ? (walk.item - head * w.tiles) * p.rows : 0;
      // the first look-ups are under way while the piece is described
      int2 at = more ? look(walk.c0, walk, lane / boxes, lane % boxes) : make_int2(-1, -1);
      const int live = more ? min((int)min((long long)w.s.count * p.group - row0, 64ll), p.rows) : 0;
      if (lane == 0) {
        Piece& q = pieces[ps];
        q.chunks = -1;
        if (more) {
          const bool begins = walk.c0 == 0, ends = walk.c1 == w.chunks;
          q.s = w.s;
          q.lo = w.lo;
          q.hi = w.hi;
          q.key0 = (w.chunk0 + walk.c0) * kKeys;
          q.chunks = walk.c1 - walk.c0;
          q.head = head;
          q.row0 = row0;
          // (four row warps leave no room for merging)
          q.row_warps = p.row_warps == kWorkers || live > 8 * kNt ? p.row_warps : 1;
          // a CTA's first place is for an item that another CTA began, its second for one that
          // another goes on with
          q.place = begins && ends ? -1 : 2 * (int)blockIdx.x + (begins ? 1 : 0);
          if (begins && !ends) {
            // the CTAs that have the rest: the last one holds the item's last unit
            const long long end = u1 + walk.rest;
            const int last = (int)quotient(end * range[1] - 1, range[0]);
            p.joins[2 * blockIdx.x] = make_int4(last - (int)blockIdx.x + 1, w.s.first, w.s.count, head);
            p.joins[2 * blockIdx.x + 1] = make_int4(row0, 0, 0, 0);
          }
        }
        mbar_arrive_expect_tx(&piece_full[ps], live * D * 2);
      }
      __syncwarp();
      for (int r = lane; r < live; r += 32) {
        const RowAt at = row_at(p, w.s, head, row0 + r);
        bulk_load(smem_u32(qs + (ps * p.rows + r) * C::kQPitch),
                  p.q + at.token * p.q_stride + (long long)at.head * D, D * 2, &piece_full[ps]);
      }
      ++np;
      if (!more) break;

      for (int c = walk.c0; ok && c < walk.c1; c += group) {
        if (c > walk.c0) at = look(c, walk, lane / boxes, lane % boxes);
        const bool bad = at.y >= 0 && (unsigned)at.x >= (unsigned)p.seqs.n_pages;
        if (bad) seqs_bad(p.seqs);
        if constexpr (kQuant) {
          const long long page = bad || at.y < 0 ? 0 : at.x, row = (long long)head * p.seqs.page + max(at.y, 0);
          looked_scales[lane] = make_longlong2(
              reinterpret_cast<long long>(p.k_scale + page * p.k_scale_stride + row),
              reinterpret_cast<long long>(p.v_scale + page * p.v_scale_stride + row));
        }
        // (a page that is none lies outside the tensor map: zeros)
        if (bad) at.x = p.seqs.n_pages;
        looked[lane] = at;
        const unsigned needed = __ballot_sync(0xffffffffu, at.y >= 0);
        __syncwarp();
        const int last = min(group, walk.c1 - c);
        if (leader) {
          for (int i = 0; i < last; ++i) {
            const int at_n = n + i, st = at_n % kStages;
            if (at_n >= kStages && !mbar_wait(&empty[st], ((at_n / kStages) & 1) ^ 1, wait)) {
              ok = false;
              break;
            }
            issued = at_n + 1;
            const unsigned want = needed >> (i * boxes) & ((1u << boxes) - 1);
            mbar_arrive_expect_tx(&full[st],
                                  __popc(want) * p.box * (2 * C::kRow + (kQuant ? 8 : 0)));
            const uint32_t tile = smem_u32(ring) + st * 2 * C::kTile;
            auto issue = [&](int j, int2 place, longlong2 from) {
              const uint32_t to = tile + j * p.box * C::kPitch;
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h) {
                tma_load_4d(to + h * kKeys * C::kPitch, &p.kmap, &full[st], h * 64, place.y, head,
                            place.x);
                tma_load_4d(to + C::kTile + h * kKeys * C::kPitch, &p.vmap, &full[st], h * 64, place.y,
                            head, place.x);
              }
              if constexpr (kQuant) {
                const uint32_t s_to = smem_u32(scales + 2 * st * kKeys + j * p.box);
                bulk_load(s_to, reinterpret_cast<const void*>(from.x), p.box * 4, &full[st]);
                bulk_load(s_to + kKeys * 4, reinterpret_cast<const void*>(from.y), p.box * 4,
                          &full[st]);
              }
            };
            if constexpr (kNt > 1) store_release(&told, at_n + 1);
            if (boxes == 1) {
              issue(0, looked[i], looked_scales[kQuant ? i : 0]);
            } else {  // the boxes' operands first: reading them one by one takes longer than a copy
              int2 place[4];
              longlong2 from[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                place[j] = looked[(i * boxes + j) & 31];
                from[j] = looked_scales[kQuant ? (i * boxes + j) & 31 : 0];
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (want >> j & 1) issue(j, place[j], from[j]);
            }
          }
        }
        n += last;
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    if (leader) {
      // the last copies write to this CTA's shared memory, whoever still waits for them
      for (int i = max(0, issued - kStages); i < issued; ++i)
        drain_wait(&full[i % kStages], (i / kStages) & 1, p.drain_ns, p.err);
    }
    if (lane == 0) {
      for (int i = max(0, np - C::kPieces); i < np; ++i)
        drain_wait(&piece_full[i % C::kPieces], (i / C::kPieces) & 1, p.drain_ns, p.err);
    }
    return;
  }

  // ---- compute.  Products are taken with the keys as rows: S^T = K Q^T (16 keys x 8 rows), and
  // O^T = V^T P^T (16 channels x 8 rows), so that a group of up to 8 rows wastes nothing.  Lane 4 n
  // + t holds keys n and n + 8 of 16, rows 2 t and 2 t + 1 of 8.
  regs_grow<kWorkRegs>();
  const int qn = lane >> 2, qt = lane & 3, l7 = lane & 7, lm = lane >> 3;
  // where a lane's row of an ldmatrix begins: of keys (lm & 1 or lm >> 1: the second eight), and
  // the 16-byte chunk in it (the other bit), which the swizzle moves by the row
  const uint32_t swz = C::kPitch == 128 ? l7 : (l7 >> 1) & 3;
  const uint32_t k_row = ((lm & 1) * 8 + l7) * C::kPitch, k_x = ((lm >> 1) ^ swz) << 4;
  const uint32_t v_row = kQuant ? k_row : ((lm >> 1) * 8 + l7) * C::kPitch;
  const uint32_t v_x = kQuant ? k_x : ((lm & 1) ^ swz) << 4;
  int n = 0, nm = 0;  // chunks and merged pieces so far
  int dealt = 0, unsure = 0;  // row warps of the last piece; chunks whose places had other warps
  for (int np = 0;; ++np) {
    const int ps = np % C::kPieces;
    if (!wait_all(&piece_full[ps], (np / C::kPieces) & 1, wait)) return;
    const Piece pc = pieces[ps];
    if (pc.chunks < 0) return;
    if (kNt > 1 && pc.row_warps != dealt) {
      unsure = dealt ? n + kStages : 0;
      dealt = pc.row_warps;
    }
    const int row_warps = kNt == 1 ? 1 : pc.row_warps, kgs = kWorkers / row_warps;
    const int tile = warp % row_warps, kg = warp / row_warps;
    const int row0 = pc.row0 + 8 * kNt * tile;  // this warp's first row

    // q: bf16, channels (2 t, + 1, + 8, + 9) of 16; or fp16, channels 4 t .. + 3 of 16, the order in
    // which 8-bit codes come out of the ring
    uint32_t q[kNt][D / 16][2];
    F2 mul[kNt];                     // what the rows' products have to be multiplied by
    int pos[kNt][2];                 // -1: no row
    float slope[kNt][2];             // - slope * log2 e
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      const int r = 8 * (kNt * tile + t) + qn;
      const bool live = row_at(p, pc.s, pc.head, pc.row0 + r).live;
      const uint8_t* src = qs + (ps * p.rows + r) * C::kQPitch;
      float up = 1.f;
      if constexpr (!kQuant) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t* at = reinterpret_cast<const uint32_t*>(src + 32 * s + 4 * qt);
          q[t][s][0] = live ? at[0] : 0u;
          q[t][s][1] = live ? at[4] : 0u;
        }
      } else {
        uint2 v[D / 16];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          v[s] = live ? *reinterpret_cast<const uint2*>(src + 32 * s + 8 * qt) : make_uint2(0, 0);
          top = max(top, max(max(v[s].x & 0x7fffu, v[s].x >> 16 & 0x7fffu),
                             max(v[s].y & 0x7fffu, v[s].y >> 16 & 0x7fffu)));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest channel into [2^14, 2^15)
        const int e = min(max((int)(top >> 7) - 127 - 14, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          q[t][s][0] = pack_half(__uint_as_float(v[s].x << 16) * down,
                                 __uint_as_float(v[s].x & 0xffff0000u) * down);
          q[t][s][1] = pack_half(__uint_as_float(v[s].y << 16) * down,
                                 __uint_as_float(v[s].y & 0xffff0000u) * down);
        }
      }
      // from the lanes that read a row to those that hold its products
      float m2[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m2[x] = __shfl_sync(0xffffffffu, up, 4 * (2 * qt + x)) * p.scale2;
        const RowAt ra = row_at(p, pc.s, pc.head, row0 + 8 * t + 2 * qt + x);
        pos[t][x] = ra.live ? ra.pos : -1;
        slope[t][x] = 0.f;
        if constexpr (kScored)
          if (p.slopes && ra.live) slope[t][x] = p.slopes[ra.head] * -1.4426950408889634f;
      }
      mul[t] = f2(m2[0], m2[1]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[ps]);
    // the keys that all of this warp's rows see
    int all_lo, all_hi, dummy;
    {
      const RowAt a = row_at(p, pc.s, pc.head, row0);
      const RowAt z = row_at(p, pc.s, pc.head, row0 + 8 * kNt - 1);
      sees(p, pc.s, a.pos, &dummy, &all_hi);
      sees(p, pc.s, min(z.pos, pc.s.len - 1), &all_lo, &dummy);
    }

    float o[D / 16][kNt][4];
    float m[kNt][2];
    F2 l[kNt];
    float vref = 0.f;
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t] = f2(0.f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
    }

    // One chunk: S^T, the softmax's step, O^T += V^T P^T.  (Leaving out a second tile without rows, by a
    // second copy of this code, costs more in instruction fetches than it saves.)
    auto chunk_step = [&](int st, int base, bool masked) {
      const uint32_t kt = smem_u32(ring) + st * 2 * C::kTile, vt = kt + C::kTile;
      const float* ks = scales + 2 * st * kKeys;
      const float* vs = ks + kKeys;
      float inv = 0.f;
      if constexpr (kQuant) {
        // fp16 weights p * v's scale in units of vref, the power of two at or above the largest
        // scale so far, raised by kPUp: at most 2^(8 + 6 + 1), and nothing is lost above 2^-20
        // of the largest.  vref is at least 2^-120, so that kPUp / vref is finite: scales go down
        // to fp32's least, whose quotient would be infinite and, times a weight of 0, NaN.
        uint32_t big = 0;
#pragma unroll
        for (int x = 0; x < kKeys / 32; ++x)
          big = max(big, __float_as_uint(vs[32 * x + lane]) & 0x7fffffffu);
        big = __reduce_max_sync(0xffffffffu, big);
        if (big > __float_as_uint(vref)) {
          const float to = __uint_as_float(
              max(min((big + 0x7fffffu) & 0xff800000u, 0x7f000000u), kLeastUnit));
          if (to > vref) {
            const float by = vref / to;
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
              for (int t = 0; t < kNt; ++t)
#pragma unroll
                for (int y = 0; y < 4; ++y) o[d][t][y] *= by;
            vref = to;
          }
        }
        inv = vref > 0.f ? kPUp / vref : 0.f;
      }
#pragma unroll 1
      for (int sub = 0; sub < kKeys; sub += C::kSub) {
        // scores
        float s[kMt][kNt][4];
#pragma unroll
        for (int j = 0; j < kMt; ++j)
#pragma unroll
          for (int t = 0; t < kNt; ++t) s[j][t][0] = s[j][t][1] = s[j][t][2] = s[j][t][3] = 0.f;
#pragma unroll
        for (int x = 0; x < C::kRow / 32; ++x) {  // 32 bytes of the keys at a time
          const uint32_t row = kt + (x >> 2) * kKeys * C::kPitch + sub * C::kPitch + k_row +
                               (k_x ^ ((x & 3) << 5));
#pragma unroll
          for (int j = 0; j < kMt; ++j) {
            uint32_t f[4];
            ldsm4(row + j * 16 * C::kPitch, f);
            if constexpr (!kQuant) {
#pragma unroll
              for (int t = 0; t < kNt; ++t) mma<false>(s[j][t], f, q[t][x]);
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a[4];
                along<kType>(f[2 * y], &a[0], &a[2]);
                along<kType>(f[2 * y + 1], &a[1], &a[3]);
#pragma unroll
                for (int t = 0; t < kNt; ++t) mma<true>(s[j][t], a, q[t][2 * x + y]);
              }
            }
          }
        }

        // scale, cap, bias, mask: s becomes base-2 scores
        auto each = [&](auto f) {
#pragma unroll
          for (int j = 0; j < kMt; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int t = 0; t < kNt; ++t)
                split(f(f2(s[j][t][2 * y], s[j][t][2 * y + 1]), 16 * j + 8 * y, t), &s[j][t][2 * y],
                      &s[j][t][2 * y + 1]);
        };
        auto scaled = [&](F2 v, int key, int t) {
          return mul2(v, kQuant ? mul2(mul[t], f2(ks[sub + key + qn])) : mul[t]);
        };
        if constexpr (!kScored) {
          each(scaled);
        } else {
          float far[kNt][2];  // distances of this lane's first key
#pragma unroll
          for (int t = 0; t < kNt; ++t) {
            far[t][0] = (float)(pos[t][0] - base - sub - qn);
            far[t][1] = (float)(pos[t][1] - base - sub - qn);
          }
          auto biased = [&](F2 v, int key, int t) {
            float v0, v1;
            split(v, &v0, &v1);
            return f2(fmaf(slope[t][0], fabsf(far[t][0] - (float)key), v0),
                      fmaf(slope[t][1], fabsf(far[t][1] - (float)key), v1));
          };
          if (p.cap2 > 0.f) {
            each(scaled);
            // tanh by its polynomial where all of the warp's scores are within its reach (score.cuh).
            // The scores are divided by the cap only here: its quotient with the rows' and keys'
            // factors could be below fp32's range.
            const float reach = 0.875f * p.cap2;
            float top = 0.f;
            each([&](F2 v, int, int) {
              float v0, v1;
              split(v, &v0, &v1);
              top = fmaxf(top, fmaxf(fabsf(v0), fabsf(v1)));
              return v;
            });
            if (__any_sync(0xffffffffu, top > reach)) {
              each([&](F2 v, int, int) {
                float v0, v1;
                split(v, &v0, &v1);
                return f2(p.cap2 * tanhf(v0 * p.inv_cap2), p.cap2 * tanhf(v1 * p.inv_cap2));
              });
            } else {  // (a NaN's way too)
              each([&](F2 v, int, int) {
                const F2 y = mul2(v, f2(p.inv_cap2)), u = mul2(y, y);
                F2 r = f2((float)tanh_coef(5));
#pragma unroll
                for (int i = 4; i >= 0; --i) r = fma2(r, u, f2((float)tanh_coef(i)));
                return mul2(r, v);
              });
            }
            if (p.slopes) each(biased);
          } else {
            each([&](F2 v, int key, int t) { return biased(scaled(v, key, t), key, t); });
          }
        }
        if (masked) {
#pragma unroll
          for (int t = 0; t < kNt; ++t) {
            int lo[2], hi[2];
            sees(p, pc.s, pos[t][0], &lo[0], &hi[0]);
            sees(p, pc.s, pos[t][1], &lo[1], &hi[1]);
#pragma unroll
            for (int j = 0; j < kMt; ++j)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int key = base + sub + 16 * j + 8 * (y >> 1) + qn;
                if ((unsigned)(key - lo[y & 1]) >= (unsigned)(hi[y & 1] - lo[y & 1]))
                  s[j][t][y] = -INFINITY;
              }
          }
        }
        bool grow = false;
        float top[kNt][2];
#pragma unroll
        for (int t = 0; t < kNt; ++t) {
          top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
          for (int j = 0; j < kMt; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) top[t][y & 1] = fmaxf(top[t][y & 1], s[j][t][y]);
          grow |= top[t][0] > m[t][0] + kLazy || top[t][1] > m[t][1] + kLazy;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < kNt; ++t) {
            float by[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float to = fmaxf(m[t][x], row_max(top[t][x]));
              by[x] = to == m[t][x] ? 1.f : fast_exp2(m[t][x] - to);
              m[t][x] = to;
            }
            l[t] = mul2(l[t], f2(by[0], by[1]));
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
#pragma unroll
              for (int y = 0; y < 4; ++y) o[d][t][y] *= by[y & 1];
          }
        }

        // weights, as B operands: [row n][keys 2 t, + 1]
        uint32_t ph[kMt][kNt][2], pl[kQuant ? 1 : kMt][kNt][2];
#pragma unroll
        for (int t = 0; t < kNt; ++t) {
          const F2 off = f2(m[t][0] == -INFINITY ? 0.f : -m[t][0], m[t][1] == -INFINITY ? 0.f : -m[t][1]);
#pragma unroll
          for (int j = 0; j < kMt; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float a, b;
              split(add2(f2(s[j][t][2 * y], s[j][t][2 * y + 1]), off), &a, &b);
              a = fast_exp2(a);
              b = fast_exp2(b);
              l[t] = add2(l[t], f2(a, b));
              if constexpr (kQuant) {
                const float f = vs[sub + 16 * j + 8 * y + qn] * inv;
                ph[j][t][y] = turned(pack_half(a * f, b * f));
              } else {
                const uint32_t h = pack_bf16(a, b);
                ph[j][t][y] = turned(h);
                pl[j][t][y] = turned(pack_bf16(a - __uint_as_float(h << 16),
                                               b - __uint_as_float(h & 0xffff0000u)));
              }
            }
        }

        // O^T += V^T P^T, 16 keys at a time
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
#pragma unroll
          for (int x = 0; x < C::kRow / 32; ++x) {  // 32 bytes of the values at a time
            uint32_t f[4];
            ldsm4_t(vt + ((x >> 2) * kKeys + sub + 16 * j) * C::kPitch + v_row + (v_x ^ ((x & 3) << 5)),
                    f);
            if constexpr (!kQuant) {
#pragma unroll
              for (int t = 0; t < kNt; ++t) mma<false>(o[x][t], f, ph[j][t]);
#pragma unroll
              for (int t = 0; t < kNt; ++t) mma<false>(o[x][t], f, pl[j][t]);
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a[4];
                across<kType>(f[2 * y], &a[0], &a[1]);
                across<kType>(f[2 * y + 1], &a[2], &a[3]);
#pragma unroll
                for (int t = 0; t < kNt; ++t) mma<true>(o[2 * x + y][t], a, ph[j][t]);
              }
            }
          }
        }
      }
    };
    const bool any_rows = (long long)pc.s.count * p.group > row0;
    for (int i = (kg - n) & (kgs - 1); i < pc.chunks; i += kgs) {
      const int at = n + i, st = at % kStages, base = pc.key0 + i * kKeys;
      if ((kNt > 1 && at < unsure && !wait_issued(&told, at, wait)) ||
          !wait_all(&full[st], (at / kStages) & 1, wait))
        return;
      const bool masked = base < all_lo || base + kKeys > all_hi;
      if (base < pc.lo || base + kKeys > pc.hi) {
        // Keys outside the item: their weights are 0, and what the ring holds for their values
        // and scales becomes 0 too (another warp of the chunk writes the same).  With a cap so do
        // the keys: the way to tanh is chosen by all of a warp's scores.
        const bool keys_too = kScored && p.cap2 > 0.f;
        constexpr int kVecs = C::kTile / 16;
        uint4* tiles = reinterpret_cast<uint4*>(ring + 2 * st * C::kTile);  // k, v
        for (int x = (keys_too ? 0 : kVecs) + lane; x < 2 * kVecs; x += 32) {
          const int key = base + x / (C::kPitch / 16) % kKeys;
          if (key < pc.lo || key >= pc.hi) tiles[x] = make_uint4(0, 0, 0, 0);
        }
        if constexpr (kQuant)
          for (int x = (keys_too ? 0 : kKeys) + lane; x < 2 * kKeys; x += 32) {
            const int key = base + x % kKeys;
            if (key < pc.lo || key >= pc.hi) scales[2 * st * kKeys + x] = 0.f;
          }
        fence_proxy_async_smem();  // before the copies that follow these writes
        __syncwarp();
      }
      if (any_rows) chunk_step(st, base, masked);
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&empty[st], kNt == 1 ? 1 : p.row_warps / row_warps);
    }
    n += pc.chunks;

    float ls[kNt][2];
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
      split(l[t], &ls[t][0], &ls[t][1]);
      ls[t][0] = row_sum(ls[t][0]);
      ls[t][1] = row_sum(ls[t][1]);
    }
    if constexpr (kQuant) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int t = 0; t < kNt; ++t)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[d][t][y] = o[d][t][y] * (1.f / kPUp) * vref;
    }
    // the warps of the same rows: into one of them, which takes turns
    if (kgs > 1) {
      const int buf = nm % C::kMergeBufs, parity = (nm / C::kMergeBufs) & 1;
      const int from_one = (kg - nm) & (kgs - 1);  // 0: this warp's turn
      float4* bufs = merge + buf * (kWorkers - 1) * (C::kMerge / 16) + lane;
      // (every warp sees every phase of these barriers, one after the other)
      if (nm >= C::kMergeBufs && !wait_all(&merge_empty[buf], parity ^ 1, wait)) return;
      ++nm;
      if (from_one > 0) {
        float4* to = bufs + ((from_one - 1) * row_warps + tile) * (C::kMerge / 16);
#pragma unroll
        for (int t = 0; t < kNt; ++t) {
#pragma unroll
          for (int d = 0; d < D / 16; ++d, to += 32)
            *to = make_float4(o[d][t][0], o[d][t][1], o[d][t][2], o[d][t][3]);
          *to = make_float4(m[t][0], m[t][1], ls[t][0], ls[t][1]);
          to += 32;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&merge_full[buf], kMergeArrivals / (kWorkers - row_warps));
        continue;
      }
      if (!wait_all(&merge_full[buf], parity, wait)) return;
      for (int g = 1; g < kgs; ++g) {
        const float4* from = bufs + ((g - 1) * row_warps + tile) * (C::kMerge / 16);
#pragma unroll
        for (int t = 0; t < kNt; ++t, from += 32 * (D / 16 + 1)) {
          const float4 ml = from[32 * (D / 16)];
          float own[2], other[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float mo = x ? ml.y : ml.x, lo_ = x ? ml.w : ml.z;
            const float to = fmaxf(m[t][x], mo), ref = to == -INFINITY ? 0.f : to;
            own[x] = fast_exp2(m[t][x] - ref);
            other[x] = fast_exp2(mo - ref);
            ls[t][x] = ls[t][x] * own[x] + lo_ * other[x];
            m[t][x] = to;
          }
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const float4 v = from[32 * d];
            o[d][t][0] = o[d][t][0] * own[0] + v.x * other[0];
            o[d][t][1] = o[d][t][1] * own[1] + v.y * other[1];
            o[d][t][2] = o[d][t][2] * own[0] + v.z * other[0];
            o[d][t][3] = o[d][t][3] * own[1] + v.w * other[1];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_n(&merge_empty[buf], kWorkers / row_warps);
    }

    // channels of o[d][t][0 / 2] (row 2 t; [1 / 3]: row 2 t + 1): bf16 16 d + n and 16 d + 8 + n, 8-bit types
    // 16 d + 2 n and the next
#pragma unroll
    for (int t = 0; t < kNt; ++t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const RowAt ra = row_at(p, pc.s, pc.head, row0 + 8 * t + 2 * qt + x);
        if (!ra.live) continue;
        if (pc.place < 0) {
          const float by = ls[t][x] == 0.f ? 0.f : 1.f / ls[t][x];
          __nv_bfloat16* to = p.o + ra.token * p.o_stride + (long long)ra.head * D;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const uint32_t two = pack_bf16(o[d][t][x] * by, o[d][t][2 + x] * by);
            if constexpr (kQuant) {
              *reinterpret_cast<uint32_t*>(to + 16 * d + 2 * qn) = two;
            } else {
              reinterpret_cast<uint16_t*>(to)[16 * d + qn] = (uint16_t)two;
              reinterpret_cast<uint16_t*>(to)[16 * d + 8 + qn] = (uint16_t)(two >> 16);
            }
          }
          if (p.lse && qn == 0) p.lse[ra.head * p.seqs.n + ra.token] = lse_of(m[t][x], ls[t][x]);
        } else {
          const long long row = (long long)pc.place * p.rows + 8 * (kNt * tile + t) + 2 * qt + x;
          float* to = p.part_o + row * D;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            if constexpr (kQuant) {
              *reinterpret_cast<float2*>(to + 16 * d + 2 * qn) = make_float2(o[d][t][x], o[d][t][2 + x]);
            } else {
              to[16 * d + qn] = o[d][t][x];
              to[16 * d + 8 + qn] = o[d][t][2 + x];
            }
          }
          if (qn == 0) p.part_ml[row] = make_float2(m[t][x], ls[t][x]);
        }
      }
    }
  }
}

// Joins the pieces of the item that CTA blockIdx.x of the first kernel began.  A few pieces: a row a
// warp; more: a row a block, a quarter of the pieces a warp.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const __grid_constant__ AttnParams p) {
  constexpr int kPer = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 join = p.joins[2 * blockIdx.x];
  const int row0 = p.joins[2 * blockIdx.x + 1].x;
  if (join.x == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = p.rows;
  const Seq seq = {join.y, join.z, 0};
  auto place = [&](int i) { return 2 * ((int)blockIdx.x + i) + (i == 0 ? 1 : 0); };
  if (join.x <= 4) {
    for (int r = blockIdx.y * kJoinWarps + warp; r < rows; r += gridDim.y * kJoinWarps) {
      const RowAt at = row_at(p, seq, join.w, row0 + r);
      if (!at.live) break;  // rows are live up to the last token's
      float2 ml[4];
      float v[4][kPer], m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long row = (long long)place(min(i, join.x - 1)) * rows + r;
        ml[i] = i < join.x ? p.part_ml[row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int x = 0; x < kPer; ++x) v[i][x] = p.part_o[row * D + kPer * lane + x];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, ml[i].x);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= join.x) break;
        const float by = fast_exp2(ml[i].x - ref);
        l = fmaf(ml[i].y, by, l);
#pragma unroll
        for (int x = 0; x < kPer; ++x) o[x] = fmaf(v[i][x], by, o[x]);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint32_t* to = reinterpret_cast<uint32_t*>(p.o + at.token * p.o_stride + (long long)at.head * D) +
                     kPer / 2 * lane;
#pragma unroll
      for (int x = 0; x < kPer / 2; ++x) to[x] = pack_bf16(o[2 * x] * inv, o[2 * x + 1] * inv);
      if (p.lse && lane == 0) p.lse[at.head * p.seqs.n + at.token] = lse_of(m, l);
    }
    return;
  }
  __shared__ float so[kJoinWarps][D], sm[kJoinWarps], sl[kJoinWarps];
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const RowAt at = row_at(p, seq, join.w, row0 + r);
    if (!at.live) break;  // rows are live up to the last token's
    float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = 0.f;
    for (int i = warp; i < join.x; i += kJoinWarps) {
      const long long row = (long long)place(i) * rows + r;
      const float2 ml = p.part_ml[row];
      float v[kPer];
#pragma unroll
      for (int x = 0; x < kPer; ++x) v[x] = p.part_o[row * D + kPer * lane + x];
      const float to = fmaxf(m, ml.x), ref = to == -INFINITY ? 0.f : to;
      const float mine = fast_exp2(m - ref), other = fast_exp2(ml.x - ref);
      m = to;
      l = l * mine + ml.y * other;
#pragma unroll
      for (int x = 0; x < kPer; ++x) o[x] = o[x] * mine + v[x] * other;
    }
    __syncthreads();  // the row before is written
#pragma unroll
    for (int x = 0; x < kPer; ++x) so[warp][kPer * lane + x] = o[x];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    float to = -INFINITY, sum = 0.f;
#pragma unroll
    for (int g = 0; g < kJoinWarps; ++g) to = fmaxf(to, sm[g]);
    const float ref = to == -INFINITY ? 0.f : to;
    float by[kJoinWarps];
#pragma unroll
    for (int g = 0; g < kJoinWarps; ++g) {
      by[g] = fast_exp2(sm[g] - ref);
      sum += sl[g] * by[g];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < kJoinWarps; ++g) v += so[g][d] * by[g];
      p.o[at.token * p.o_stride + (long long)at.head * D + d] = __float2bfloat16_rn(v * inv);
    }
    if (p.lse && threadIdx.x == 0) p.lse[at.head * p.seqs.n + at.token] = lse_of(to, sum);
  }
}

// the pool of pages as (channel, token of a page, kv head, page), in boxes of `box` tokens
inline bool pages_map(CUtensorMap* map, const void* base, int type, int64_t stride, const marble_cache_t& c,
               int box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const int es = type == MARBLE_CACHE_BF16 ? 2 : 1, row = c.d * es;
  const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page_tokens, (cuuint64_t)c.hkv,
                              (cuuint64_t)c.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)row, (cuuint64_t)row * c.page_tokens,
                                 (cuuint64_t)stride * es};
  const cuuint32_t boxes[4] = {(cuuint32_t)std::min(c.d, 128 / es), (cuuint32_t)box, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
             const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row >= 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kType, int kNt, bool kScored>
marble_status_t launch(AttnParams& p, int grid, int join_rows, cudaStream_t s) {
  using C = Cfg<D, kType, kNt>;
  auto kernel = k_attn_cached<D, kType, kNt, kScored>;
  {
    // (held until it is set: a second thread's first call must not launch before)
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev & 63] || dev > 63) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(2));
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(k_attn_cached)");
      done[dev & 63] = true;
    }
  }
  kernel<<<grid, kThreads, C::smem(p.row_warps), s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "marble_attn_cached launch");
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, join_rows <= 8 ? join_rows : (join_rows + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_join<D>, p);
  if (e != cudaSuccess) return cuda_fail(e, "marble_attn_cached join launch");
  return MARBLE_OK;
}

// the kernel of a cache type, 8 or 16 rows a warp, with or without changed scores
template <int D>
marble_status_t launch_d(AttnParams& p, int type, int nt, bool scored, int grid, int join_rows,
                         cudaStream_t s) {
  auto at = [&](auto tt) {
    constexpr int T = decltype(tt)::value;
    switch (type * 2 + (scored ? 1 : 0)) {
      case 0: return launch<D, MARBLE_CACHE_BF16, T, false>(p, grid, join_rows, s);
      case 1: return launch<D, MARBLE_CACHE_BF16, T, true>(p, grid, join_rows, s);
      case 2: return launch<D, MARBLE_CACHE_E4M3, T, false>(p, grid, join_rows, s);
      case 3: return launch<D, MARBLE_CACHE_E4M3, T, true>(p, grid, join_rows, s);
      case 4: return launch<D, MARBLE_CACHE_INT8, T, false>(p, grid, join_rows, s);
      default: return launch<D, MARBLE_CACHE_INT8, T, true>(p, grid, join_rows, s);
    }
  };
  return nt == 1 ? at(std::integral_constant<int, 1>{}) : at(std::integral_constant<int, 2>{});
}

}  // namespace cached

// the two head dims, each in a translation unit of its own (attn_cached.cu, attn_cached_64.cu)
marble_status_t launch_d128(cached::AttnParams& p, int type, int nt, bool scored, int grid,
                            int join_rows, cudaStream_t s);
marble_status_t launch_d64(cached::AttnParams& p, int type, int nt, bool scored, int grid,
                           int join_rows, cudaStream_t s);

}  // namespace marble
