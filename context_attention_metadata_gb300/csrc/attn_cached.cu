// Attention of every sequence's last tokens over its paged, cached keys and values.
//
//   s_j = scale q.k_j (capped, lowered by a slope times the distance, in base 2),
//   m = running maximum, p_j = 2^(s_j - m), l = sum p_j, O = sum p_j v_j,   o = O / l.
//
// Bound by memory: every key and value is read once, at 2 or 1 bytes a channel, for the few rows
// (new tokens x q heads of a group) that share it.
//
// - An item is a (sequence, kv head, tile of 16, 32 or 64 rows); its cost is its chunks of keys
//   and a constant.  Every CTA takes an equal range of the sum of all costs, so that ragged
//   batches keep all SMs busy to the end; it finds its range from the sequences' lengths itself.
//   An item that a range cuts leaves unnormalised pieces (O, m, l) in the workspace, at most two a
//   CTA whatever the batch, and a second kernel, already launched when the first ends, joins
//   them in order.
// - A CTA is a warp that fetches chunks by TMA into a ring (a lane for each box of a page, page
//   table look-ups included) and four that compute; two CTAs share an SM, so that one's item
//   boundaries hide behind the other's streaming.
// - A chunk belongs to one warp of every 16 rows: warps have their own m, l and O over their
//   chunks and meet only at an item's end.  A place of the ring always belongs to the same warps
//   (its copies may land before those of an earlier place: whoever waits for a place's next
//   filling must have seen the one before, or the barrier's parity misleads it).  The products are m16n8k16 matrix instructions, whose
//   16 rows are what a kv head's group gives; tcgen05's 128 would be mostly padding, and the rate
//   of the warp-level ones is several times what memory can feed at these sizes.
// - 8-bit codes become fp16 exactly in registers; k's scales multiply scores, v's scales the
//   weights, so that nothing but the weights (and q, by a power of two a row) is rounded to fp16.
#include <math.h>

#include <algorithm>
#include <cstring>

#include "seqs.cuh"
#include "tma_host.h"

namespace marble {
namespace {

constexpr int kWorkers = 4;                     // computing warps
constexpr int kThreads = 32 * (kWorkers + 1);
constexpr int kUnitOver = 1;                    // an item's constant cost, in chunks
constexpr float kLazy = 8.f;                    // O is rescaled when m grows by more (base 2)
constexpr float kPUp = 64.f;                    // fp16 weights are raised by this (see below)

template <int D, int kType>
struct Cfg {
  static constexpr bool kQuant = kType != MARBLE_CACHE_BF16;
  static constexpr int kRow = D * (kQuant ? 1 : 2);          // bytes of a key
  static constexpr int kPitch = kRow > 128 ? 128 : kRow;     // of its rows in shared memory
  static constexpr int kHalves = kRow / kPitch;
  static constexpr int kKeys = kRow > 128 ? 32 : 64;         // of a chunk
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kStages = kTile == 8192 ? 4 : 8;
  static_assert(kStages % kWorkers == 0, "a place of the ring belongs to the same warps");
  static constexpr int kMerge = 32 * (D / 2 + 4) * 4;        // a warp's O, m, l
  static constexpr int kScales = kQuant ? kStages * 2 * kKeys * 4 : 0;
  static constexpr int kSmem =
      1024 + kStages * 2 * kTile + kScales + (kWorkers - 1) * kMerge + 2 * kStages * 8 + 64;
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
  float to_cap;      // scale / cap
  float cap2;        // cap * log2 e, 0: none
  int hkv, group, hq;
  int window, span;
  int tiles;         // 16-row tiles of an item: 1, 2 or 4
  int box;           // keys of a TMA box
  int grain;         // units a CTA takes at least
  float* part_o;     // [2 * CTAs][16 * tiles][D] pieces
  float2* part_ml;   // [2 * CTAs][16 * tiles]
  int4* joins;       // [CTAs]: sequence, item, pieces (0: none)
  unsigned* err;
  uint64_t limit_ns;
};

// one sequence's items: `items` of `units` each; all of them walk the chunks
// [chunk0, chunk0 + chunks) of the keys [lo, hi)
struct Work {
  Seq s;
  int lo, hi, chunk0, chunks, tiles, items;
  long long units;
};

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

template <int kKeys, bool kTell>
__device__ __forceinline__ Work work_of(const AttnParams& p, int b) {
  Work w;
  w.s = seq_at<kTell>(p.seqs, b);
  int hi;
  sees(p, w.s, max(w.s.len - w.s.count, 0), &w.lo, &hi);
  w.hi = p.window > 0 || p.span ? w.s.len : w.lo;  // (no window: no keys at all)
  w.chunk0 = w.lo / kKeys;
  w.chunks = w.lo < w.hi ? (w.hi - 1) / kKeys - w.chunk0 + 1 : 0;
  w.tiles = (int)(((long long)w.s.count * p.group + 16 * p.tiles - 1) / (16 * p.tiles));
  w.items = w.tiles * p.hkv;
  w.units = w.items ? w.chunks + kUnitOver : 0;
  return w;
}

// chunks before offset x of an item
__device__ __forceinline__ int cut(long long x) { return (int)max(x - kUnitOver, 0ll); }

// the walk over a CTA's range of units, piece by piece
template <int kKeys>
struct Walk {
  const AttnParams& p;
  long long left, at;  // units left, offset in the sequence's units
  int b;
  Work w;
  // of the present piece
  int item, c0, c1;
  __device__ __forceinline__ Walk(const AttnParams& p_, int b_, long long at_, long long left_)
      : p(p_), left(left_), at(at_), b(b_) {
    w = work_of<kKeys, false>(p, b);
  }
  __device__ __forceinline__ bool next() {
    while (left > 0) {
      if (at >= w.units * w.items) {
        at -= w.units * w.items;
        if (++b >= p.seqs.n_seqs) return false;
        w = work_of<kKeys, false>(p, b);
        continue;
      }
      item = (int)(at / w.units);
      const long long from = at - item * w.units, to = min(w.units, from + left);
      at += to - from;
      left -= to - from;
      c0 = cut(from);
      c1 = cut(to);
      if (c1 > c0 || (w.chunks == 0 && from == 0)) return true;
    }
    return false;
  }
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
// c += a b, 16 x 8 x 16
template <bool kHalf>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// ln of the sum, from a base-2 maximum and a sum
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// row `r` of an item: its token's row in the call and its q head
struct RowAt {
  int token, head, pos;
  bool live;
};
__device__ __forceinline__ RowAt row_at(const AttnParams& p, const Work& w, int item, int r) {
  const int head = item / w.tiles, x = (item - head * w.tiles) * 16 * p.tiles + r;
  const int t = x / p.group;
  RowAt a;
  a.live = t < w.s.count;
  a.token = w.s.first + t;
  a.head = head * p.group + (x - t * p.group);
  a.pos = w.s.len - w.s.count + t;
  return a;
}

template <int D, int kType, bool kScored>
__global__ void __launch_bounds__(kThreads, 2) k_attn_cached(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, kType>;
  constexpr bool kQuant = C::kQuant;
  constexpr int kKeys = C::kKeys, kStages = C::kStages, kNt = kKeys / 8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = align1024(smem_raw);
  float* scales = reinterpret_cast<float*>(ring + kStages * 2 * C::kTile);
  float4* merge = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(scales) + C::kScales);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(merge) +
                                               (kWorkers - 1) * C::kMerge);
  uint64_t* empty = full + kStages;
  __shared__ int abort_flag, first_b;
  __shared__ long long first_at, range[2], sums[kWorkers + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // let the joining kernel's CTAs come up beside this one's
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's range of units
  const int ns = p.seqs.n_seqs, share = (ns + kThreads - 1) / kThreads;
  const int b0 = min(tid * share, ns), b1 = min(b0 + share, ns);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Work w = blockIdx.x == 0 ? work_of<kKeys, true>(p, b) : work_of<kKeys, false>(p, b);
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
    p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], p.tiles);
    }
    fence_mbar_init();
  }
  __syncthreads();
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i <= kWorkers; ++i) {
    before += i < warp ? sums[i] : 0;
    total += sums[i];
  }
  const long long ctas = min((long long)gridDim.x, (total + p.grain - 1) / p.grain);
  if (blockIdx.x >= ctas) return;
  const long long u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
  if (before <= u0 && u0 < before + mine) {
    long long at = u0 - before;
    int b = b0;
    for (; b < b1; ++b) {
      const Work w = work_of<kKeys, false>(p, b);
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
  Walk<kKeys> walk(p, first_b, first_at, u1 - u0);
  int n = 0;  // chunks of the CTA so far

  if (warp == kWorkers) {
    // ---- fetch: lane 4 x + j takes box j of part x
    const int box = lane & 3, part = lane >> 2, boxes = kKeys / p.box;
    constexpr int kParts = kQuant ? 4 : 2 * C::kHalves;
    bool ok = true;
    while (ok && walk.next()) {
      const int head = walk.item / walk.w.tiles;
      for (int c = walk.c0; c < walk.c1; ++c, ++n) {
        const int st = n % kStages;
        const int key = (walk.w.chunk0 + c) * kKeys + box * p.box;
        const bool needed = box < boxes && key < walk.w.hi && key + p.box > walk.w.lo;
        int page = 0;
        if (needed && part < kParts) {
          page = page_at(p.seqs, walk.b, key);
          if (page < 0 && part == 0) seqs_bad(p.seqs);
        }
        if (n >= kStages && !warp_wait(&empty[st], ((n / kStages) & 1) ^ 1, wait)) {
          ok = false;
          break;
        }
        const int count = __popc(__ballot_sync(0xffffffffu, needed && part == 0));
        if (lane == 0)
          mbar_arrive_expect_tx(&full[st], count * p.box * (2 * C::kRow + (kQuant ? 8 : 0)));
        __syncwarp();
        if (needed && part < kParts) {
          const uint32_t tile = smem_u32(ring) + st * 2 * C::kTile;
          // (a page that is none lies outside the tensor map: zeros)
          const int g = page < 0 ? p.seqs.n_pages : page, slot = key % p.seqs.page;
          if constexpr (kQuant) {
            if (part < 2) {
              tma_load_4d(tile + part * C::kTile + box * p.box * C::kPitch,
                          part ? &p.vmap : &p.kmap, &full[st], 0, slot, head, g);
            } else {
              const float* src = part == 2 ? p.k_scale + max(page, 0) * p.k_scale_stride
                                           : p.v_scale + max(page, 0) * p.v_scale_stride;
              bulk_load(smem_u32(scales + (2 * st + part - 2) * kKeys + box * p.box),
                        src + (long long)head * p.seqs.page + slot, p.box * 4, &full[st]);
            }
          } else {
            const int which = part / C::kHalves, half = part % C::kHalves;
            tma_load_4d(tile + which * C::kTile + (half * kKeys + box * p.box) * C::kPitch,
                        which ? &p.vmap : &p.kmap, &full[st], half * 64, slot, head, g);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      // the last copies write to this CTA's shared memory, whoever still waits for them
      for (int i = max(0, n - kStages); i < n; ++i)
        drain_wait(&full[i % kStages], (i / kStages) & 1, p.limit_ns, p.err);
    }
    return;
  }

  // ---- compute
  const int tile = warp % p.tiles, kg = warp / p.tiles, kgs = kWorkers / p.tiles;
  const int qn = lane >> 2, qt = lane & 3, l7 = lane & 7, lm = lane >> 3;
  while (walk.next()) {
    const Work& w = walk.w;
    const RowAt ra[2] = {row_at(p, w, walk.item, 16 * tile + qn),
                         row_at(p, w, walk.item, 16 * tile + qn + 8)};
    // q in registers: bf16, channels (16 s + 2 t, + 1, + 8, + 9) of step s; or fp16, channels
    // 16 s + 4 t .. + 3, the order in which 8-bit codes come out of the ring
    uint32_t q[D / 16][4];
    int lo[2], hi[2];
    float up[2] = {1.f, 1.f};  // what the row's products have to be multiplied by
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      sees(p, w.s, ra[x].pos, &lo[x], &hi[x]);
      if (!ra[x].live) lo[x] = hi[x] = 0;
      const __nv_bfloat16* src =
          p.q + (ra[x].live ? ra[x].token * p.q_stride + (long long)ra[x].head * D : 0);
      if constexpr (!kQuant) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t* at = reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * qt);
          q[s][x] = ra[x].live ? at[0] : 0u;
          q[s][2 + x] = ra[x].live ? at[4] : 0u;
        }
      } else {
        uint2 v[D / 16];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          v[s] = ra[x].live ? *reinterpret_cast<const uint2*>(src + 16 * s + 4 * qt)
                            : make_uint2(0, 0);
          top = max(top, max(max(v[s].x & 0x7fffu, v[s].x >> 16 & 0x7fffu),
                             max(v[s].y & 0x7fffu, v[s].y >> 16 & 0x7fffu)));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest channel into [2^14, 2^15)
        const int e = min(max((int)(top >> 7) - 127 - 14, -126), 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        up[x] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          q[s][x] = pack_half(__uint_as_float(v[s].x << 16) * down,
                              __uint_as_float(v[s].x & 0xffff0000u) * down);
          q[s][2 + x] = pack_half(__uint_as_float(v[s].y << 16) * down,
                                  __uint_as_float(v[s].y & 0xffff0000u) * down);
        }
      }
    }
    float mul[2] = {up[0] * p.scale2, up[1] * p.scale2}, slope2[2] = {0.f, 0.f};
    if constexpr (kScored) {
      if (p.cap2 > 0.f) {
        mul[0] = up[0] * p.to_cap;
        mul[1] = up[1] * p.to_cap;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (p.slopes && ra[x].live) slope2[x] = p.slopes[ra[x].head] * 1.4426950408889634f;
    }
    // the keys that all of this warp's rows see
    int all_lo, all_hi, dummy;
    {
      const RowAt a = row_at(p, w, walk.item, 16 * tile);
      const RowAt z = row_at(p, w, walk.item, 16 * tile + 15);
      sees(p, w.s, a.pos, &dummy, &all_hi);
      sees(p, w.s, min(z.pos, w.s.len - 1), &all_lo, &dummy);
    }

    float o[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vref = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int i = (kg - n) & (kgs - 1); i < walk.c1 - walk.c0; i += kgs) {
      const int at = n + i, st = at % kStages, base = (w.chunk0 + walk.c0 + i) * kKeys;
      // (given up: the warps still meet at the items' ends)
      if (!wait_all(&full[st], (at / kStages) & 1, wait)) break;
      const uint32_t kt = smem_u32(ring) + st * 2 * C::kTile, vt = kt + C::kTile;
      const float* ks = scales + 2 * st * kKeys;
      const float* vs = ks + kKeys;
      const bool cut_v = base < w.lo || base + kKeys > w.hi;    // keys that no row may see
      const bool masked = base < all_lo || base + kKeys > all_hi;

      // scores: keys 8 j + 2 t, + 1 of rows n and n + 8
      float s[kNt][4];
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        const int row = 8 * j + l7;
#pragma unroll
        for (int x = 0; x < C::kRow / 64; ++x) {  // 64 bytes of the keys at a time
          const int chunk = 4 * x + lm;
          uint32_t f[4];
          if constexpr (C::kPitch == 128) {
            const int half = chunk >> 3;
            ldsm4(kt + (half * kKeys + row) * 128 + (((chunk & 7) ^ l7) << 4), f);
          } else {
            ldsm4(kt + row * 64 + ((chunk ^ ((l7 >> 1) & 3)) << 4), f);
          }
          if constexpr (!kQuant) {
            mma<false>(s[j], q[2 * x], f[0], f[1]);
            mma<false>(s[j], q[2 * x + 1], f[2], f[3]);
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t h0, h1;
              along<kType>(f[y], &h0, &h1);
              mma<true>(s[j], q[4 * x + y], h0, h1);
            }
          }
        }
      }

      // scale, cap, bias, mask
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
        float2 kscale = make_float2(1.f, 1.f);
        if constexpr (kQuant) kscale = *reinterpret_cast<const float2*>(ks + 8 * j + 2 * qt);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int x = y >> 1, key = base + 8 * j + 2 * qt + (y & 1);
          float v = s[j][y] * mul[x];
          if constexpr (kQuant) v *= (y & 1) ? kscale.y : kscale.x;
          if constexpr (kScored) {
            if (p.cap2 > 0.f) v = p.cap2 * tanhf(v);
            v = fmaf(-slope2[x], (float)abs(ra[x].pos - key), v);
          }
          if (masked && (unsigned)(key - lo[x]) >= (unsigned)(hi[x] - lo[x])) v = -INFINITY;
          s[j][y] = v;
          top[x] = fmaxf(top[x], v);
        }
      }
      top[0] = quad_max(top[0]);
      top[1] = quad_max(top[1]);
      if (__any_sync(0xffffffffu, top[0] > m[0] + kLazy || top[1] > m[1] + kLazy)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float to = fmaxf(m[x], top[x]), by = to == m[x] ? 1.f : fast_exp2(m[x] - to);
          m[x] = to;
          l[x] *= by;
#pragma unroll
          for (int d = 0; d < D / 8; ++d) {
            o[d][2 * x] *= by;
            o[d][2 * x + 1] *= by;
          }
        }
      }
      const float at0 = m[0] == -INFINITY ? 0.f : m[0], at1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
      for (int j = 0; j < kNt; ++j) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          s[j][y] = fast_exp2(s[j][y] - (y < 2 ? at0 : at1));
          l[y >> 1] += s[j][y];
        }
      }

      if constexpr (kQuant) {
        // fp16 weights p * v's scale in units of vref, the power of two at or above the largest
        // scale so far, raised by kPUp: at most 2^(8 + 6 + 1), and nothing is lost above 2^-20
        // of the largest.
        uint32_t big = 0;
#pragma unroll
        for (int x = 0; x < kKeys / 32; ++x) {
          const int key = base + 32 * x + lane;
          if (key >= w.lo && key < w.hi)
            big = max(big, __float_as_uint(vs[32 * x + lane]) & 0x7fffffffu);
        }
        big = __reduce_max_sync(0xffffffffu, big);
        if (big > __float_as_uint(vref)) {
          const float to = __uint_as_float(min((big + 0x7fffffu) & 0xff800000u, 0x7f000000u));
          if (to > vref) {
            const float by = vref / to;
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
#pragma unroll
              for (int y = 0; y < 4; ++y) o[d][y] *= by;
            vref = to;
          }
        }
        const float inv = vref > 0.f ? kPUp / vref : 0.f;
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
          float2 f = *reinterpret_cast<const float2*>(vs + 8 * j + 2 * qt);
          if (cut_v) {
            const int key = base + 8 * j + 2 * qt;
            if (key < w.lo || key >= w.hi) f.x = 0.f;
            if (key + 1 < w.lo || key + 1 >= w.hi) f.y = 0.f;
          }
          f.x *= inv;
          f.y *= inv;
          s[j][0] *= f.x;
          s[j][1] *= f.y;
          s[j][2] *= f.x;
          s[j][3] *= f.y;
        }
      }

      // O += P V, 16 keys at a time
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk) {
        uint32_t live[2] = {~0u, ~0u};
        if (cut_v) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = base + 16 * kk + 8 * x + 2 * qt;
            live[x] = (key >= w.lo && key < w.hi ? 0xffffu : 0u) |
                      (key + 1 >= w.lo && key + 1 < w.hi ? 0xffff0000u : 0u);
          }
        }
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float a = s[2 * kk + (x >> 1)][2 * (x & 1)], b = s[2 * kk + (x >> 1)][2 * (x & 1) + 1];
          if constexpr (kQuant) {
            ph[x] = pack_half(a, b);
          } else {
            ph[x] = pack_bf16(a, b);
            pl[x] = pack_bf16(a - __uint_as_float(ph[x] << 16),
                              b - __uint_as_float(ph[x] & 0xffff0000u));
          }
        }
        const int row = 16 * kk + (lm & 1) * 8 + l7;
#pragma unroll
        for (int x = 0; x < C::kRow / 32; ++x) {  // 32 bytes of the values at a time
          const int chunk = 2 * x + (lm >> 1);
          uint32_t f[4];
          if constexpr (C::kPitch == 128) {
            const int half = chunk >> 3;
            ldsm4_t(vt + (half * kKeys + row) * 128 + (((chunk & 7) ^ l7) << 4), f);
          } else {
            ldsm4_t(vt + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4), f);
          }
          if (cut_v) {
            f[0] &= live[0];
            f[1] &= live[1];
            f[2] &= live[0];
            f[3] &= live[1];
          }
          if constexpr (!kQuant) {
            mma<false>(o[2 * x], ph, f[0], f[1]);
            mma<false>(o[2 * x + 1], ph, f[2], f[3]);
            mma<false>(o[2 * x], pl, f[0], f[1]);
            mma<false>(o[2 * x + 1], pl, f[2], f[3]);
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a0, a1, c0, c1;
              across<kType>(f[2 * y], &a0, &c0);
              across<kType>(f[2 * y + 1], &a1, &c1);
              mma<true>(o[4 * x + 2 * y], ph, a0, a1);
              mma<true>(o[4 * x + 2 * y + 1], ph, c0, c1);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    n += walk.c1 - walk.c0;

    l[0] = quad_sum(l[0]);
    l[1] = quad_sum(l[1]);
    if constexpr (kQuant) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[d][y] = o[d][y] * (1.f / kPUp) * vref;
    }
    // the warps of the same rows: into the first of them
    if (kgs > 1) {
      const int bar = 1 + tile;
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * kgs) : "memory");
      if (kg > 0) {
        float4* to = merge + ((kg - 1) * p.tiles + tile) * (C::kMerge / 16) + lane;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) to[32 * d] = make_float4(o[d][0], o[d][1], o[d][2], o[d][3]);
        to[32 * (D / 8)] = make_float4(m[0], m[1], l[0], l[1]);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * kgs) : "memory");
      if (kg > 0) continue;
      for (int g = 1; g < kgs; ++g) {
        const float4* from = merge + ((g - 1) * p.tiles + tile) * (C::kMerge / 16) + lane;
        const float4 ml = from[32 * (D / 8)];
        float mine[2], other[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float mo = x ? ml.y : ml.x, lother = x ? ml.w : ml.z;
          const float to = fmaxf(m[x], mo), ref = to == -INFINITY ? 0.f : to;
          mine[x] = fast_exp2(m[x] - ref);
          other[x] = fast_exp2(mo - ref);
          l[x] = l[x] * mine[x] + lother * other[x];
          m[x] = to;
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          const float4 v = from[32 * d];
          o[d][0] = o[d][0] * mine[0] + v.x * other[0];
          o[d][1] = o[d][1] * mine[0] + v.y * other[0];
          o[d][2] = o[d][2] * mine[1] + v.z * other[1];
          o[d][3] = o[d][3] * mine[1] + v.w * other[1];
        }
      }
    }

    const bool begins = walk.c0 == 0, ends = walk.c1 == w.chunks;
    if (begins && ends) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ra[x].live) continue;
        const float by = l[x] == 0.f ? 0.f : 1.f / l[x];
        __nv_bfloat16* to = p.o + ra[x].token * p.o_stride + (long long)ra[x].head * D;
        if constexpr (!kQuant) {
#pragma unroll
          for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<uint32_t*>(to + 8 * d + 2 * qt) =
                pack_bf16(o[d][2 * x] * by, o[d][2 * x + 1] * by);
        } else {
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<uint2*>(to + 16 * d + 4 * qt) =
                make_uint2(pack_bf16(o[2 * d][2 * x] * by, o[2 * d + 1][2 * x] * by),
                           pack_bf16(o[2 * d][2 * x + 1] * by, o[2 * d + 1][2 * x + 1] * by));
        }
        if (p.lse && qt == 0) p.lse[ra[x].head * p.seqs.n + ra[x].token] = lse_of(m[x], l[x]);
      }
    } else {
      // a piece: the CTA's first place for one that another CTA began, its second otherwise
      const int place = 2 * blockIdx.x + (begins ? 1 : 0), rows = 16 * p.tiles;
      if (begins && tile == 0 && lane == 0) {
        // the CTAs that have the rest: the last one holds the item's last unit
        const long long rest = (long long)w.chunks - walk.c1;  // units behind this range
        const long long end = u1 + rest;
        const int last = (int)((end * range[1] - 1) / range[0]);
        p.joins[blockIdx.x] = make_int4(walk.b, walk.item, last - (int)blockIdx.x + 1, 0);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ra[x].live) continue;
        const long long row = (long long)place * rows + 16 * tile + qn + 8 * x;
        float* to = p.part_o + row * D;
        if constexpr (!kQuant) {
#pragma unroll
          for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2*>(to + 8 * d + 2 * qt) =
                make_float2(o[d][2 * x], o[d][2 * x + 1]);
        } else {
#pragma unroll
          for (int d = 0; d < D / 16; ++d)
            *reinterpret_cast<float4*>(to + 16 * d + 4 * qt) =
                make_float4(o[2 * d][2 * x], o[2 * d + 1][2 * x], o[2 * d][2 * x + 1],
                            o[2 * d + 1][2 * x + 1]);
        }
        if (qt == 0) p.part_ml[row] = make_float2(m[x], l[x]);
      }
    }
  }
}

// Joins the pieces of the item that CTA blockIdx.x of the first kernel began, a row a block (and
// every gridDim.y-th row after it), a quarter of the pieces a warp.
constexpr int kJoinWarps = 4;
template <int D, int kKeys>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join(const __grid_constant__ AttnParams p) {
  constexpr int kPer = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 join = p.joins[blockIdx.x];
  if (join.z == 0) return;
  __shared__ float so[kJoinWarps][D], sm[kJoinWarps], sl[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = 16 * p.tiles;
  const Work w = work_of<kKeys, false>(p, join.x);
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const RowAt at = row_at(p, w, join.y, r);
    if (!at.live) break;  // rows are live up to the last token's
    float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = 0.f;
    for (int i = warp; i < join.z; i += kJoinWarps) {
      const int place = 2 * (blockIdx.x + i) + (i == 0 ? 1 : 0);
      const long long row = (long long)place * rows + r;
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
bool pages_map(CUtensorMap* map, const void* base, int type, int64_t stride, const marble_cache_t& c,
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

template <int D, int kType, bool kScored>
marble_status_t launch(AttnParams& p, int grid, int join_rows, cudaStream_t s) {
  using C = Cfg<D, kType>;
  if (once_per_device(64 + (D == 128 ? 0 : 1) + 2 * kType + (kScored ? 8 : 0))) {
    const cudaError_t e = cudaFuncSetAttribute(k_attn_cached<D, kType, kScored>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(k_attn_cached)");
  }
  k_attn_cached<D, kType, kScored><<<grid, kThreads, C::kSmem, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "marble_attn_cached launch");
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, join_rows);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_join<D, C::kKeys>, p);
  if (e != cudaSuccess) return cuda_fail(e, "marble_attn_cached join launch");
  return MARBLE_OK;
}

}  // namespace

marble_status_t run_attn_cached(int64_t n, const marble_cache_t* c, const marble_seqs_t* seqs,
                                const marble_attn_cached_t* a, const marble_score_t* score,
                                cudaStream_t s) {
  AttnParams p;
  memset(&p, 0, sizeof(p));
  const bool quant = c->type != MARBLE_CACHE_BF16;
  const int keys = !quant && c->d == 128 ? 32 : 64;
  p.box = 16;
  while (p.box < keys && c->page_tokens % (2 * p.box) == 0) p.box *= 2;
  if (!pages_map(&p.kmap, c->k, c->type, c->k_stride, *c, p.box) ||
      !pages_map(&p.vmap, c->v, c->type, c->v_stride, *c, p.box))
    return fail(MARBLE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the cache");
  p.seqs = seqs_params(*seqs, *c, n);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.k_scale_stride = c->k_scale_stride;
  p.v_scale_stride = c->v_scale_stride;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.o = static_cast<__nv_bfloat16*>(a->o);
  p.lse = a->lse;
  p.q_stride = a->q_stride;
  p.o_stride = a->o_stride;
  const double scale = a->scale > 0.f ? a->scale : 1.0 / std::sqrt((double)c->d);
  p.scale2 = (float)(scale * 1.4426950408889634);
  const bool scored = score && (score->cap > 0.f || score->slopes);
  if (scored) {
    p.slopes = score->slopes;
    if (score->cap > 0.f) {
      p.to_cap = (float)(scale / score->cap);
      p.cap2 = (float)(score->cap * 1.4426950408889634);
    }
  }
  p.hkv = c->hkv;
  p.hq = a->hq;
  p.group = a->hq / c->hkv;
  p.window = a->window;
  p.span = a->span ? 1 : 0;
  const int64_t rows = std::min<int64_t>(64, (int64_t)p.group * std::max(1, a->new_tokens));
  p.tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  p.grain = 2;
  p.limit_ns = wait_limit_ns();
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // workspace: a word for timeouts without a status, the joins, the pieces
  const int64_t piece = 16 * p.tiles * (int64_t)(c->d + 2) * 4;
  const int64_t most = (MARBLE_ATTN_CACHED_WORKSPACE_BYTES - 65536) / (2 * piece);
  const int grid = (int)std::min<int64_t>(std::min<int64_t>(2 * sms, most), 4000);
  char* ws = static_cast<char*>(a->workspace);
  p.err = seqs->status ? reinterpret_cast<unsigned*>(seqs->status) : reinterpret_cast<unsigned*>(ws);
  p.joins = reinterpret_cast<int4*>(ws + 256);
  p.part_ml = reinterpret_cast<float2*>(ws + 65536);
  p.part_o = reinterpret_cast<float*>(ws + 65536 + 2 * (int64_t)grid * 16 * p.tiles * 8);
  auto at_d = [&](auto dd) {
    constexpr int D = decltype(dd)::value;
    switch (c->type * 2 + (scored ? 1 : 0)) {
      case 0: return launch<D, MARBLE_CACHE_BF16, false>(p, grid, (int)rows, s);
      case 1: return launch<D, MARBLE_CACHE_BF16, true>(p, grid, (int)rows, s);
      case 2: return launch<D, MARBLE_CACHE_E4M3, false>(p, grid, (int)rows, s);
      case 3: return launch<D, MARBLE_CACHE_E4M3, true>(p, grid, (int)rows, s);
      case 4: return launch<D, MARBLE_CACHE_INT8, false>(p, grid, (int)rows, s);
      default: return launch<D, MARBLE_CACHE_INT8, true>(p, grid, (int)rows, s);
    }
  };
  return c->d == 128 ? at_d(std::integral_constant<int, 128>{})
                     : at_d(std::integral_constant<int, 64>{});
}

}  // namespace marble
