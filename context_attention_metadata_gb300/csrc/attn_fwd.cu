// Forward ring step: update the fp32 online-softmax state (O_acc, m, l) of one q shard
// against the tiles the plan lists for one kv shard (or for all needed kv blocks).
//
// MARBLE post, s03 "Exact ring attention accumulation": each ring step is the usual
// FlashAttention loop over a different set of key/value blocks; the fp32 accumulator, m
// and l stay in HBM between calls and are resumed on every call but the first; only
// the last call normalises.  RingAttention tutorial, "The Online Softmax Formulation":
// the recurrence m_new = max(m, rowmax S), rescale by exp(m - m_new), add exp(S - m_new).
//
// Kernel structure (sm_103a): one persistent CTA per SM takes work units (q block, q head)
// from a shared ticket counter, in the plan's order for the step (longest tile list first),
// and runs them through a pipeline of warp roles that meet at mbarriers:
//   warp 2      scheduler: draws a ticket, turns it into a unit and its tile-list range and
//               posts it in a 4-entry queue in shared memory; every other role reads the
//               queue in order, and the epilogue frees an entry once all roles are past it.
//   warp 0      TMA producer: Q of each unit into one of two slots, K_j and V_j through
//               two-slot rings.
//   warp 1      allocates all 512 TMEM columns: S double buffer [0,128) and [128,256),
//               O double buffer [256,384) and [384,512) (units alternate); lane 0 issues
//               tcgen05.mma -- S = Q K^T up to two tiles ahead of the softmax, O += P V with P
//               as bf16 in TMEM over its S buffer and V read MN-major -- polling its inputs
//               and issuing whichever of the next PV and the next S is ready.
//   warps 4..11 softmax: two warps per TMEM lane quarter, each owning 64 of a row's 128
//               columns; the row max is exchanged through shared memory.  Row max, exp2,
//               row sum, bf16 P back into TMEM, lazy O rescale; at a unit's end they hand
//               the row's (m, l) to the epilogue and go on with the next unit at once.  On
//               partial tiles they evaluate the mask (mask_chunk: once per row and run of keys
//               with the same ids); full tiles skip it; empty tiles are never listed, so never
//               loaded.
//   warps 12..15 epilogue, one thread per row: merge the unit's (O, m, l) into the stored
//               state through a staged TMA store / reduce-add, while the softmax warps and
//               the tensor core work on the next unit in the other O buffer.
// Scores are kept in base-2 units (s * scale * log2 e); the stored m is in the same units
// and always an integer, so that every rescale (lazy, when the max grows past 2^8, within
// a call; and the merge with the stored state) multiplies by an exact power of two.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "score.cuh"
#include "tma_host.h"

namespace marble {
namespace {

constexpr int kThreads = 512;              // 16 warps, roles above
constexpr int kSoftmax = 256;              // softmax threads (warps 4..11)
constexpr int kEpi = 128;                  // epilogue threads (warps 12..15)
constexpr int kWarpSched = 2;
constexpr int kWarpSoft0 = 4;
constexpr int kWarpEpi0 = 12;
// registers per thread: the launch gives every thread 128 (512 x 128 = the SM's 65,536); the
// control warps and the epilogue hand theirs to the two softmax warpgroups, which would spill
// with 128: 128 x 56 + 256 x 168 + 128 x 112 <= 512 x 128
constexpr int kRegsLaunch = 128;
constexpr int kRegsCtl = 56;
constexpr int kRegsSoft = 168;
constexpr int kRegsEpi = 112;
static_assert(128 * kRegsCtl + kSoftmax * kRegsSoft + kEpi * kRegsEpi <= kThreads * kRegsLaunch,
              "register split");
constexpr float kRescaleThreshold = 8.0f;  // base-2 units: rescale O when max grows > 2^8
constexpr int kQueue = 4;                  // work-queue entries

enum {
  B_QFULL0, B_QFULL1, B_QEMPTY0, B_QEMPTY1,  // Q slots (unit & 1): fill / last S of the unit
  B_KFULL0, B_KFULL1, B_KEMPTY0, B_KEMPTY1,  // K ring (slot = tile & 1): fill / S done
  B_VFULL0, B_VFULL1, B_VEMPTY0, B_VEMPTY1,  // V ring: fill / PV done
  B_SFULL0, B_SFULL1,                // S buffer (tile & 1) computed
  B_PFULL0, B_PFULL1,                // P written over S buffer (256 softmax arrivals)
  B_PVDONE,                          // one phase per tile: its PV has completed
  B_OFULL0, B_OFULL1,                // O buffer (unit & 1): the unit's last PV completed
  B_OFREE0, B_OFREE1,                // O buffer read out by the epilogue (128 arrivals)
  B_MX0, B_MX1,                      // per-row max exchanged between the two halves
  B_EPIRDY0, B_EPIRDY1,              // (m, l) of the unit handed over (256 arrivals)
  B_HFREE0, B_HFREE1,                // hand-over slot read by the epilogue (128 arrivals)
  B_EVOTE,                           // per unit: epilogue's merge-mode vote (128 arrivals)
  B_STG,                             // per staging round: rows written (128 arrivals)
  B_STGFREE,                         // per staging round: the TMA has read the staging box
  B_UFULL0,                          // queue entry posted (kQueue barriers)
  B_UEMPTY0 = B_UFULL0 + kQueue,     // queue entry released (kQueue barriers)
  B_DRAIN = B_UEMPTY0 + kQueue,
  B_NUM
};

__host__ __device__ constexpr int arrivals(int b) {
  return (b == B_PFULL0 || b == B_PFULL1 || b == B_MX0 || b == B_MX1 ||
          b == B_EPIRDY0 || b == B_EPIRDY1)
             ? kSoftmax
             : ((b == B_OFREE0 || b == B_OFREE1 || b == B_HFREE0 || b == B_HFREE1 ||
                 b == B_EVOTE || b == B_STG)
                    ? kEpi
                    : 1);
}

struct FwdParams {
  CUtensorMap q_map, k_map, v_map;
  CUtensorMap o_map;  // fp32 O_acc, box 32 x 128 x 1, 128-byte swizzle
  const int64_t* step_ptr;
  const int32_t* step_col;
  const uint8_t* step_tag;
  const int32_t* tracks;  // [4][n] sample, seg, noise, pos in plan order
  const int32_t* order;   // work order of this step: q blocks of the shard, longest first
  unsigned* sched;        // ticket counter pair of this launch
  float* o_acc;
  float* m;
  float* l;
  unsigned* err;
  unsigned long long wait_ns;
  long long n;
  int P, bps, q_shard, kv_shard;
  int hq, group;
  int units;  // bps * hq
  int nwork;  // units with at least one tile: nonempty blocks of the order x hq (x parts)
  int parts;  // scored kernels: pieces of every unit's list, work units of their own (1: whole)
  long long n_out;  // their output's tokens: piece i of a row is row i * n of o_acc, m and l
  int W;
  int first;
  int lse_merge;   // 0 carried state; 1 merge of bf16 partials (standard ring); 2 of fp32 ones
  const int32_t* kiv;       // [2][n] lo, hi of every key's visible-query interval
  const int4* kiv_chunk;    // [nb*4] per 32 keys: min lo, max lo, min hi, max hi
  const int32_t* qidx;      // [n] plan order -> index in the given token order (the plan's perm)
  const uint8_t* iv_block;  // [nb] 1: every key of the block has an exact interval
  float scale_log2;
  ScoreParams score;        // read by the kernels built with a cap or a bias
};

// list range of work unit u = h * bps + i (q block i of the shard, q head h)
__device__ __forceinline__ int unit_tiles(const FwdParams& p, int u, int64_t* e0) {
  const int i = u % p.bps;
  const int64_t nq = (int64_t)p.q_shard * p.bps + i;
  int64_t a, b;
  if (p.kv_shard >= 0) {
    a = p.step_ptr[nq * p.P + p.kv_shard];
    b = p.step_ptr[nq * p.P + p.kv_shard + 1];
  } else {
    a = p.step_ptr[nq * p.P];
    b = p.step_ptr[nq * p.P + p.P];
  }
  *e0 = a;
  return (int)(b - a);
}

// the work queue in shared memory: entry uc of this CTA sits in slot uc % kQueue
struct Queue {
  int unit[kQueue];  // -1: no more work
  int part[kQueue];  // scored kernels: piece of the unit's list
  int T[kQueue];
  long long e0[kQueue];
};

constexpr int kMaxParts = 8;

// tiles of each piece of a list of T tiles (the last may have fewer, or there may be fewer pieces)
__device__ __forceinline__ int part_tiles(int T, int parts) {
  return (int)(((unsigned)T + parts - 1) / (unsigned)parts);
}

// two-slot rings indexed by the tile counter g: slot g & 1, phase parity (g >> 1) & 1
__device__ __forceinline__ uint32_t ring_slot(int g) { return (uint32_t)(g & 1); }
__device__ __forceinline__ uint32_t ring_parity(int g) { return (uint32_t)((g >> 1) & 1); }

// shared memory: Q (2) | K ring (2) | V ring (2) | staging (one 128 x 32 fp32 box) | row-max
// exchange [2][2][128] f32 | hand-over m [2][128] and
// l [2][2][128] f32
template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = 4 * kTile;
  static constexpr int kStg = 6 * kTile;
  static constexpr int kMx = kStg + 16384;
  static constexpr int kHm = kMx + 2 * 2 * 128 * 4;
  static constexpr int kHl = kHm + 2 * 128 * 4;
  static constexpr int kEnd = kHl + 2 * 2 * 128 * 4;
  static constexpr size_t bytes() { return (size_t)kEnd + 1024; }  // + alignment slack
};
static_assert(Smem<128>::bytes() <= 232448, "shared memory budget");

// A row's 64 products of this half, in place, to base-2 scores with the cap and the bias.
// side: +1 or -1 where the tile's keys all come before (after) its queries and positions are
// consecutive, so that the bias is linear in the key; 0 otherwise.  far0: the row's distance to
// the half's first key; pos: the keys' positions.
template <int MOD>
__device__ __forceinline__ void score_row(uint32_t (&v)[2][32], const FwdParams& p, float sl2,
                                          float slope, float side, float far0, int pq,
                                          const int32_t* __restrict__ pos) {
  constexpr bool kCap = (MOD & kScoreCap) != 0, kBias = (MOD & kScoreBias) != 0;
  float top = 0.f;
  if constexpr (kCap) {
    float hi[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 64; ++t)
      hi[t & 3] = fmaxf(hi[t & 3], fabsf(__uint_as_float(v[t >> 5][t & 31])));
    top = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
  }
  // key t of the half is at side (far0 - t): the bias is own + t * step
  const float own = -side * slope * far0, step = side * slope;
  // terms: of the polynomial; 0: the exponential, -1: that or the polynomial, score by score
  auto pairs = [&](auto terms, auto linear) {
    constexpr int kTerms = decltype(terms)::value;
    constexpr bool kLinear = decltype(linear)::value;
    [[maybe_unused]] F2 at[2] = {f2(0.f, 1.f), f2(2.f, 3.f)};
    // four positions at a time, loaded one group ahead: fewer are in flight than the compiler
    // would hoist, and fewer registers spilled (64K pack, cap 50, bias: forward 3280 -> 3150 us)
    [[maybe_unused]] int4 k4, ahead;
    if constexpr (kBias && !kLinear) ahead = __ldg(reinterpret_cast<const int4*>(pos));
#pragma unroll
    for (int t = 0; t < 64; t += 4) {
      if constexpr (kBias && !kLinear) {
        k4 = ahead;
        if (t + 4 < 64) ahead = __ldg(reinterpret_cast<const int4*>(pos + t + 4));
      }
#pragma unroll
      for (int u = 0; u < 4; u += 2) {
        uint32_t &v0 = v[t >> 5][(t & 31) + u], &v1 = v[t >> 5][(t & 31) + u + 1];
        const F2 x = f2(__uint_as_float(v0), __uint_as_float(v1));
        [[maybe_unused]] F2 off;
        if constexpr (kBias && kLinear) {
          // whole numbers counted up, so that the bias is rounded once
          off = fma2(at[u >> 1], f2(step), f2(own));
          at[u >> 1] = add2(at[u >> 1], f2(4.f));
        } else if constexpr (kBias) {
          const float d0 = fabsf((float)(pq - (u == 0 ? k4.x : k4.z)));
          const float d1 = fabsf((float)(pq - (u == 0 ? k4.y : k4.w)));
          off = mul2(f2(d0, d1), f2(-slope));
        }
        F2 s;
        if constexpr (kCap && kTerms <= 0) {
          float r[2], x0, x1;
          split(x, &x0, &x1);
          s = cap_far<(kTerms < 0)>(x0, x1, p.score, r);
          if constexpr (kBias) s = add2(s, off);
        } else {
          F2 factor = f2(sl2);
          if constexpr (kCap) factor = cap_factor<kTerms>(x, p.score);
          if constexpr (kBias)
            s = fma2(x, factor, off);
          else
            s = mul2(x, factor);
        }
        float s0, s1;
        split(s, &s0, &s1);
        v0 = __float_as_uint(s0);
        v1 = __float_as_uint(s1);
      }
    }
  };
  constexpr std::integral_constant<int, -1> kWide{};
  constexpr std::integral_constant<int, 0> kExp{};
  constexpr std::integral_constant<int, 4> kNear{};
  constexpr std::integral_constant<int, 6> kFar{};
  constexpr std::true_type kLin{};
  constexpr std::bool_constant<!kBias> kAny{};
  const bool linear = !kBias || side != 0.f;
  if constexpr (!kCap) {
    if (linear)
      pairs(kFar, kLin);
    else
      pairs(kFar, kAny);
  } else if (linear && __all_sync(0xffffffffu, top <= p.score.lim_n)) {
    pairs(kNear, kLin);
  } else if (__all_sync(0xffffffffu, top <= p.score.lim)) {
    if (linear)
      pairs(kFar, kLin);
    else
      pairs(kFar, kAny);
  } else if (p.score.wide) {
    pairs(kWide, kAny);
  } else {
    pairs(kExp, kAny);
  }
}

// MOD: what happens to the scores (bits kScoreCap, kScoreBias); 0 is the plain softmax.
template <int D, int MOD>
__global__ void __launch_bounds__(kThreads, 1) k_attn_fwd(const __grid_constant__ FwdParams p) {
  using L = Smem<D>;
  constexpr int kTile = L::kTile;
  constexpr int kAtoms = D / 64;  // 128-byte swizzle atoms along d
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem + L::kQ;  // slot b at sQ + b * kTile
  uint8_t* sK = smem + L::kK;
  uint8_t* sV = smem + L::kV;
  uint8_t* sStg = smem + L::kStg;
  float* mxs = reinterpret_cast<float*>(smem + L::kMx);
  float* hm = reinterpret_cast<float*>(smem + L::kHm);
  float* hl = reinterpret_cast<float*>(smem + L::kHl);
  __shared__ __align__(8) uint64_t bar[B_NUM];
  __shared__ Queue queue;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ int epi_mode[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n = p.n;
  WaitCtx w{p.wait_ns, p.err, &abort_flag};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    epi_mode[0] = epi_mode[1] = 0;
    for (int b = 0; b < B_NUM; ++b) mbar_init(&bar[b], arrivals(b));
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = tmem_base;        // S buffers at +0 and +128
  const uint32_t tO = tmem_base + 256;  // O buffers at +0 and +128

  if (warp < kWarpSoft0) {
  // warpgroup 0: scheduler, producer, MMA issuer (and a warp without a role)
  regs_shrink<kRegsCtl>();
  if (warp == kWarpSched) {
    // ------------------------------------------------------------------ scheduler
    if (lane == 0) {
      for (int uc = 0;; ++uc) {
        const int slot = uc % kQueue;
        if (uc >= kQueue && !mbar_wait(&bar[B_UEMPTY0 + slot], ((uc / kQueue) - 1) & 1, w)) break;
        int unit = -1, T = 0;
        int64_t e0 = 0;
        // longest lists first, the q heads of a block one after the other
        unsigned t = atomicAdd(p.sched, 1u);
        if constexpr (MOD == 0) {
          if (t < (unsigned)p.nwork) {
            unit = (int)(t % (unsigned)p.hq) * p.bps + p.order[t / (unsigned)p.hq];
            T = unit_tiles(p, unit, &e0);
          }
        } else {
          int part = 0;
          for (; T == 0 && t < (unsigned)p.nwork; t = T == 0 ? atomicAdd(p.sched, 1u) : t) {
            const unsigned b = t / (unsigned)p.parts;
            part = (int)(t - b * (unsigned)p.parts);
            unit = (int)(b % (unsigned)p.hq) * p.bps + p.order[b / (unsigned)p.hq];
            const int all = unit_tiles(p, unit, &e0), len = part_tiles(all, p.parts);
            T = max(0, min(len, all - part * len));  // 0: the list ends before this piece
            e0 += part * len;
          }
          if (T == 0) unit = -1;
          queue.part[slot] = part;
        }
        queue.unit[slot] = unit;
        queue.T[slot] = T;
        queue.e0[slot] = e0;
        mbar_arrive(&bar[B_UFULL0 + slot]);
        if (unit < 0) break;
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&p.q_map);
      tma_prefetch_desc(&p.k_map);
      tma_prefetch_desc(&p.v_map);
      tma_prefetch_desc(&p.o_map);
    }
    int uc = 0, g = 0;          // units reached, tiles reached
    int q_fills = 0, k_fills = 0, v_fills = 0;  // copies issued (fill t of K/V is tile t)
    bool ok = true;
    while (ok) {
      const int slot = uc % kQueue;
      if (!wait_all(&bar[B_UFULL0 + slot], (uc / kQueue) & 1, w)) break;
      const int unit = queue.unit[slot];
      if (unit < 0) break;
      const int T = queue.T[slot];
      const int64_t e0 = queue.e0[slot];
      const int h = unit / p.bps;
      const int kvh = h / p.group;
      const int64_t nq = (int64_t)p.q_shard * p.bps + unit % p.bps;
      // Q of the unit once the unit two back has finished reading the slot
      const int qb = uc & 1;
      if (uc >= 2 && !wait_all(&bar[B_QEMPTY0 + qb], ((uc >> 1) - 1) & 1, w)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar[B_QFULL0 + qb], kTile);
        for (int a = 0; a < kAtoms; ++a)
          tma_load_3d(sQ + qb * kTile + a * 16384, &p.q_map, &bar[B_QFULL0 + qb], a * 64,
                      (int)(nq * 128), h);
      }
      ++q_fills;
      for (int j = 0; j < T; ++j, ++g) {
        const int nk = p.step_col[e0 + j];
        const uint32_t s = ring_slot(g);
        if (g >= 2 && !wait_all(&bar[B_KEMPTY0 + s], ring_parity(g - 2), w)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[B_KFULL0 + s], kTile);
          for (int a = 0; a < kAtoms; ++a)
            tma_load_3d(sK + s * kTile + a * 16384, &p.k_map, &bar[B_KFULL0 + s], a * 64,
                        nk * 128, kvh);
        }
        ++k_fills;
        if (g >= 2 && !wait_all(&bar[B_VEMPTY0 + s], ring_parity(g - 2), w)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar[B_VFULL0 + s], kTile);
          for (int a = 0; a < kAtoms; ++a)
            tma_load_3d(sV + s * kTile + a * 16384, &p.v_map, &bar[B_VFULL0 + s], a * 64,
                        nk * 128, kvh);
        }
        ++v_fills;
      }
      ++uc;
    }
    // never leave the CTA with a copy still landing in its shared memory: the fills of a
    // slot complete in order, so waiting for the latest fill of each slot suffices (Q fill
    // f went to slot f & 1, K and V fill t to ring slot t & 1)
    if (lane == 0) {
      for (int f = q_fills - 1; f >= 0 && f >= q_fills - 2; --f)
        drain_wait(&bar[B_QFULL0 + (f & 1)], (f >> 1) & 1, p.wait_ns, p.err);
      for (int t = k_fills - 1; t >= 0 && t >= k_fills - 2; --t)
        drain_wait(&bar[B_KFULL0 + ring_slot(t)], ring_parity(t), p.wait_ns, p.err);
      for (int t = v_fills - 1; t >= 0 && t >= v_fills - 2; --t)
        drain_wait(&bar[B_VFULL0 + ring_slot(t)], ring_parity(t), p.wait_ns, p.err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdO = idesc_bf16(128, D, false, true);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV0 = sdesc_sw128(smem_u32(sV), 16384, 1024);
      // Event loop over two cursors into the work queue: issue whichever of the next PV
      // (priority: it feeds the softmax and the epilogue) and the next S (at most two tiles
      // ahead of the next PV) has its inputs ready, polling with non-blocking tests.
      struct Cur {
        int uc, j, g, T, state;  // state: 0 waiting for queue entry uc, 1 in a unit, 2 done
      };
      Cur cs{0, 0, 0, 0, 0}, cp{0, 0, 0, 0, 0};
      auto fetch = [&](Cur& c) {
        if (c.state != 0) return;
        const int slot = c.uc % kQueue;
        if (!mbar_test(&bar[B_UFULL0 + slot], (c.uc / kQueue) & 1)) return;
        c.state = queue.unit[slot] < 0 ? 2 : 1;
        c.T = queue.T[slot];
        c.j = 0;
      };
      auto advance = [](Cur& c) {
        ++c.g;
        if (++c.j == c.T) {
          ++c.uc;
          c.state = 0;
        }
      };
      uint64_t t_idle = 0;
      uint32_t idle = 0;
      while (cs.state != 2 || cp.state != 2) {
        fetch(cs);
        fetch(cp);
        bool progressed = false;
        if (cp.state == 1) {
          const int g = cp.g;
          const uint32_t b = (uint32_t)(g & 1), s = ring_slot(g), ob = (uint32_t)(cp.uc & 1);
          // the first PV of a unit overwrites its O buffer: the unit two back must be read out
          const bool ready =
              mbar_test(&bar[B_PFULL0 + b], (g >> 1) & 1) &&
              mbar_test(&bar[B_VFULL0 + s], ring_parity(g)) &&
              (cp.j != 0 || cp.uc < 2 || mbar_test(&bar[B_OFREE0 + ob], ((cp.uc >> 1) - 1) & 1));
          if (ready) {
            tc_fence_after();
            const uint64_t dV = sdesc_at(dV0, s * kTile);
            // P of half h sits in columns [64 h, 64 h + 32) of the S buffer
            mma_ts(tO + ob * 128, tS + b * 128, dV, kIdO, cp.j > 0 ? 1u : 0u);
#pragma unroll
            for (int k = 1; k < 8; ++k)
              mma_ts(tO + ob * 128, tS + b * 128 + (k >> 2) * 64 + (k & 3) * 8,
                     sdesc_at(dV, k * 2048), kIdO, 1u);
            mma_commit(&bar[B_PVDONE]);
            mma_commit(&bar[B_VEMPTY0 + s]);
            if (cp.j == cp.T - 1) mma_commit(&bar[B_OFULL0 + ob]);
            advance(cp);
            progressed = true;
          }
        }
        if (cs.state == 1 && cs.g < cp.g + 2) {
          const int g = cs.g;
          const uint32_t b = (uint32_t)(g & 1), s = ring_slot(g), qb = (uint32_t)(cs.uc & 1);
          // S(g) overwrites the P of tile g - 2, which PV(g - 2) reads: the PV is issued already
          // (S runs at most two tiles ahead of the next PV), and tcgen05.mma instructions of one
          // thread execute in issue order, so no wait for its completion is needed
          const bool ready = (cs.j != 0 || mbar_test(&bar[B_QFULL0 + qb], (cs.uc >> 1) & 1)) &&
                             mbar_test(&bar[B_KFULL0 + s], ring_parity(g));
          if (ready) {
            tc_fence_after();
            const uint64_t dQ = sdesc_at(dQ0, qb * kTile), dK = sdesc_at(dK0, s * kTile);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
              mma_ss(tS + b * 128, sdesc_at(dQ, off), sdesc_at(dK, off), kIdS, k > 0);
            }
            mma_commit(&bar[B_SFULL0 + b]);
            mma_commit(&bar[B_KEMPTY0 + s]);
            if (cs.j == cs.T - 1) mma_commit(&bar[B_QEMPTY0 + qb]);  // the unit's last read of Q
            advance(cs);
            progressed = true;
          }
        }
        if (progressed) {
          idle = 0;
        } else {
          // the clock is read only while idle, so that it never delays an issue
          __nanosleep(32);
          if ((++idle & 63) == 0) {
            if (*w.abort) break;
            const uint64_t now = globaltimer_ns();
            if (idle == 64) {
              t_idle = now;
            } else if (now - t_idle > p.wait_ns) {
              atomicOr(p.err, kErrTimeout);
              *w.abort = 1;
              break;
            }
          }
        }
      }
      // every MMA issued by this thread has completed before TMEM is released
      mma_commit(&bar[B_DRAIN]);
      drain_wait(&bar[B_DRAIN], 0, p.wait_ns, p.err);
    }
    __syncwarp();
  }
  } else if (warp < kWarpEpi0) {
    // ------------------------------------------------------------------ softmax warps
    regs_grow<kRegsSoft>();
    // two warps per TMEM lane quarter: `half` owns S columns [64 half, 64 half + 64) and O
    // columns [D/2 half, D/2 half + D/2) of its row
    const int quarter = warp & 3;
    const int half = (warp - kWarpSoft0) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lb = (uint32_t)(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    constexpr bool kMayBeFixed = MOD == (kScoreCap | kScoreBias);  // decided unit by unit
    [[maybe_unused]] int exchanges = 0;  // tiles whose row maxima were exchanged
    int uc = 0, g = 0;
    bool ok = true;
    while (ok) {
      const int slot = uc % kQueue;
      if (!wait_all(&bar[B_UFULL0 + slot], (uc / kQueue) & 1, w)) break;
      const int unit = queue.unit[slot];
      if (unit < 0) break;
      const int T = queue.T[slot];
      const int64_t e0 = queue.e0[slot];
      const int64_t tq = ((int64_t)p.q_shard * p.bps + unit % p.bps) * 128 + row;
      const int sq = p.tracks[tq], gq = p.tracks[n + tq], zq = p.tracks[2 * n + tq],
                pq = p.tracks[3 * n + tq];
      const int iq = p.qidx[tq];  // the interval test's coordinate: the query's index
      const uint32_t ob = tO + (uint32_t)(uc & 1) * 128;
      [[maybe_unused]] float slope = 0.f;
      if constexpr ((MOD & kScoreBias) != 0)
        slope = p.score.slopes[unit / p.bps] * 1.4426950408889634f;
      // for a bias the tile's kv block and its first key's position are loaded one tile ahead
      [[maybe_unused]] int kb_n = 0, k0_n = 0;
      if constexpr ((MOD & kScoreBias) != 0) {
        kb_n = p.step_col[e0];
        k0_n = p.tracks[3 * n + (int64_t)kb_n * 128];
      }
      // one stabiliser for every row: with a bias, where it only lowers scores and the launch's
      // lists hold the rows' own keys (see kFixedCap)
      const bool fixed = (MOD & kScoreFixed) != 0 || (kMayBeFixed && p.score.bias_fixed && slope >= 0.f);
      float m_run = -INFINITY, l_h = 0.f;
      for (int j = 0; j < T; ++j, ++g) {
        const uint32_t b = (uint32_t)(g & 1);
        [[maybe_unused]] float far0 = 0.f, side = 0.f;  // see score_row
        [[maybe_unused]] const int32_t* kpos = nullptr;
        if constexpr ((MOD & kScoreBias) != 0) {
          far0 = (float)(pq - k0_n - half * 64);
          if (p.score.consecutive) side = pq - row > k0_n ? 1.f : pq - row < k0_n ? -1.f : 0.f;
          kpos = p.tracks + 3 * n + (int64_t)kb_n * 128 + half * 64;
          if (j + 1 < T) kb_n = p.step_col[e0 + j + 1];
        }
        const bool partial = p.step_tag[e0 + j] == MARBLE_TILE_PARTIAL;
        uint32_t lm[2] = {~0u, ~0u};  // legal-key bits of this row in this half's 64 columns
        const int64_t kb = partial ? p.step_col[e0 + j] : 0;
        // every key of the block has an exact visible-query interval: the test is
        // lo_k <= i_q < hi_k (i_q the query's index in the given token order), with the half's
        // 64 (lo, hi) pairs read straight from global memory (the same addresses for every
        // lane: broadcast loads)
        const bool ivt = partial && p.iv_block[kb] != 0;
        if (ivt) {
          // per 32-key chunk, its keys' (min lo, max lo, min hi, max hi) first: a row inside
          // every interval takes all 32 keys and a row outside all of them none; the keys are
          // tested one by one only when some row of the warp is neither
          const int32_t* klo = p.kiv + kb * 128 + half * 64;
          const int32_t* khi = klo + n;
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int4 cs = __ldg(p.kiv_chunk + kb * 4 + half * 2 + cc);
            const bool all = iq >= cs.y && iq < cs.z;
            const bool none = iq < cs.x || iq >= cs.w;
            uint32_t bits = all ? ~0u : 0u;
            if (__any_sync(0xffffffffu, !(all || none))) {
              bits = 0;
#pragma unroll
              for (int t2 = 0; t2 < 32; t2 += 4) {
                const int4 l4 = __ldg(reinterpret_cast<const int4*>(klo + cc * 32 + t2));
                const int4 h4 = __ldg(reinterpret_cast<const int4*>(khi + cc * 32 + t2));
                bits |= ((iq >= l4.x) & (iq < h4.x) ? 1u : 0u) << t2;
                bits |= ((iq >= l4.y) & (iq < h4.y) ? 1u : 0u) << (t2 + 1);
                bits |= ((iq >= l4.z) & (iq < h4.z) ? 1u : 0u) << (t2 + 2);
                bits |= ((iq >= l4.w) & (iq < h4.w) ? 1u : 0u) << (t2 + 3);
              }
            }
            lm[cc] = bits;
          }
        } else if (partial) {
          // every lane holds the ids of one key of a 32-key chunk
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int32_t* kt = p.tracks + kb * 128 + (2 * half + cc) * 32;
            const int ks = __ldg(kt + lane), kg = __ldg(kt + n + lane), kz = __ldg(kt + 2 * n + lane);
            uint32_t causal = 0;
            if (p.score.consecutive) {
              const int64_t d = (int64_t)pq - __ldg(kt + 3 * n);  // key t is d - t before the row
              causal = bits32(d - p.W + 1, d + 1);
            } else {
#pragma unroll
              for (int t2 = 0; t2 < 32; t2 += 4) {
                const int4 k4 = __ldg(reinterpret_cast<const int4*>(kt + 3 * n + t2));
                causal |= ((unsigned)(pq - k4.x) < (unsigned)p.W ? 1u : 0u) << t2;
                causal |= ((unsigned)(pq - k4.y) < (unsigned)p.W ? 1u : 0u) << (t2 + 1);
                causal |= ((unsigned)(pq - k4.z) < (unsigned)p.W ? 1u : 0u) << (t2 + 2);
                causal |= ((unsigned)(pq - k4.w) < (unsigned)p.W ? 1u : 0u) << (t2 + 3);
              }
            }
            lm[cc] = mask_chunk<true>(sq, gq, zq, ks, kg, kz, causal);
          }
        }
        // a partial tile on which every row of this warp keeps all 64 of its keys takes the
        // full-tile path below
        const bool masked = partial && __any_sync(0xffffffffu, (lm[0] & lm[1]) != ~0u);
        if (!wait_all(&bar[B_SFULL0 + b], (g >> 1) & 1, w)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sb = tS + b * 128;
        uint32_t v[2][32];
        tmem_ld32(sb + lb + (2 * half) * 32, v[0]);
        tmem_ld32(sb + lb + (2 * half + 1) * 32, v[1]);
        tmem_ld_wait();
        // this half's row maximum of the scaled, masked scores; where a key is masked the
        // scaled scores (-inf where masked) replace v, otherwise v keeps the raw scores
        // (scaling by a positive constant commutes with the maximum, and P takes one FMA below)
        [[maybe_unused]] float mx = -INFINITY;
        if constexpr (MOD != 0) {
          score_row<MOD>(v, p, sl2, slope, side, far0, pq, kpos);
          if constexpr ((MOD & kScoreBias) != 0) k0_n = p.tracks[3 * n + (int64_t)kb_n * 128];
          if (masked) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
#pragma unroll
              for (int t = 0; t < 32; ++t)
                if (!((lm[cc] >> t) & 1u)) v[cc][t] = __float_as_uint(-INFINITY);
          }
        }
        if (fixed) {
          m_run = 0.f;
        } else if constexpr (MOD != 0) {
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int t = 0; t < 64; ++t) m4[t & 3] = fmaxf(m4[t & 3], __uint_as_float(v[t >> 5][t & 31]));
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else if (masked) {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
            for (int t = 0; t < 32; ++t) {
              const float s = ((lm[cc] >> t) & 1u) ? __uint_as_float(v[cc][t]) * sl2 : -INFINITY;
              v[cc][t] = __float_as_uint(s);
              mx = fmaxf(mx, s);
            }
          }
        } else {
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int t = 0; t < 32; ++t) mx = fmaxf(mx, __uint_as_float(v[cc][t]));
          mx *= sl2;
        }
        if (!fixed) {
          const int x = kMayBeFixed ? exchanges++ : g;
          float* mxb = mxs + (x & 1) * 256;
          mxb[half * 128 + row] = mx;
          mbar_arrive(&bar[B_MX0 + (x & 1)]);
          if (!wait_all(&bar[B_MX0 + (x & 1)], (x >> 1) & 1, w)) { ok = false; break; }
          mx = fmaxf(mx, mxb[(1 - half) * 128 + row]);
          // the running max is kept integral (base 2): every rescale factor below is then an
          // exact power of two, and bf16 rounding of P does not depend on which keys a step
          // happened to see first
          const float m_new = ceilf(mx);
          const bool grow = m_new > m_run + kRescaleThreshold;
          const bool need = grow && (m_run != -INFINITY);  // earlier tiles of this unit to rescale
          const float alpha = need ? ldexpf(1.f, (int)(m_run - m_new)) : 1.f;
          if (grow) {
            l_h *= alpha;
            m_run = m_new;
          }
          // tcgen05.ld/st are warp-collective: the whole warp rescales when any of its rows
          // must (alpha = 1 on the others).  A row that needs it has a finite max from an
          // earlier tile of this unit, so PV(g-1) is the accumulation to wait for.
          if (__any_sync(0xffffffffu, need)) {
            if (!wait_all(&bar[B_PVDONE], (g - 1) & 1, w)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 64; ++cc) {
              const uint32_t col = half * (D / 2) + cc * 32;
              uint32_t x[32];
              tmem_ld32(ob + lb + col, x);
              tmem_ld_wait();
#pragma unroll
              for (int t = 0; t < 32; ++t) x[t] = __float_as_uint(__uint_as_float(x[t]) * alpha);
              tmem_st32(ob + lb + col, x);
            }
          }
        }
        // P = exp2(s - m_run) as bf16, packed into columns [64 half, 64 half + 32) of the S
        // buffer: inside the fp32 columns this warp has just read.  bf16 because the tensor core
        // wants both operands of one type and V is bf16 (two products for the upper and the lower
        // bits of P would double PV): against 64 bits O is off by 0.0023 of its norm, where its own
        // rounding alone makes 0.0017.  The row sum takes P as it was.
        [[maybe_unused]] const float base = m_run == -INFINITY ? 0.f : m_run;
        // v holds scaled scores where keys were masked, raw ones otherwise
        [[maybe_unused]] const float vs = (MOD != 0 || masked) ? 1.f : sl2;
        auto weight = [&](uint32_t x) {
          const float s = __uint_as_float(x);
          return fast_exp2((MOD & kScoreFixed) != 0 ? s : fmaf(s, vs, -base));
        };
        float rs = 0.f;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            const float p0 = weight(v[cc][t]), p1 = weight(v[cc][t + 1]);
            rs += p0 + p1;
            pk[t >> 1] = pack_bf16(p0, p1);
          }
          tmem_st16(sb + lb + half * 64 + cc * 16, pk);
        }
        tmem_st_wait();
        l_h += rs;
        tc_fence_before();
        mbar_arrive(&bar[B_PFULL0 + b]);
      }
      if (!ok) break;
      // hand the unit's (m, l) to the epilogue once it has read the slot's previous use
      const int ub = uc & 1;
      if (uc >= 2 && !wait_all(&bar[B_HFREE0 + ub], ((uc >> 1) - 1) & 1, w)) break;
      if (half == 0) hm[ub * 128 + row] = m_run;
      hl[(ub * 2 + half) * 128 + row] = l_h;
      mbar_arrive(&bar[B_EPIRDY0 + ub]);
      ++uc;
    }
  }
  else {
    // ------------------------------------------------------------------ epilogue warps
    regs_shrink<kRegsEpi>();
    // one thread per row (warp w owns TMEM lane quarter w & 3)
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lb = (uint32_t)(quarter * 32) << 16;
    if (p.first && (MOD == 0 || p.parts == 1)) {
      // rows of units without a tile in this step start from (O = 0, m = -inf, l = 0)
      for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        int64_t e0;
        if (unit_tiles(p, u, &e0) != 0) continue;
        const int h = u / p.bps;
        const int64_t tq = ((int64_t)p.q_shard * p.bps + u % p.bps) * 128 + row;
        p.m[(int64_t)h * n + tq] = -INFINITY;
        p.l[(int64_t)h * n + tq] = 0.f;
        float4* o = reinterpret_cast<float4*>(p.o_acc + (tq * p.hq + h) * D);
#pragma unroll 8
        for (int t = 0; t < D / 4; ++t) o[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    // Merge each unit's (O, m, l) into the stored state through one staged fp32 box of 32
    // columns at a time:
    //   FIRST         the tile is stored (TMA store);
    //   otherwise     the stored max is kept unless some row's max grew past it by more
    //                 than the lazy threshold, so the update is a pure addition of
    //                 O_call * 2^(m_call - m_stored): a TMA fp32 reduce-add, no load;
    //   some row grew exact merge with the stored tile (loaded by the row threads), then a
    //                 TMA store.
    //   LSE merge     the call's output is normalised into a partial, merged with the
    //                 stored (normalised) output by log-sum-exp weights and stored; m then
    //                 holds the running base-2 LSE and l is 1 (0 for a row that has seen no
    //                 legal key), which the finalize reads unchanged.  Partial and merged
    //                 output are rounded to bf16 (the standard ring merge, kept for
    //                 comparison) or kept in fp32 (merging fp32 partials: exact to fp32).
    int uc = 0, k = 0;  // units merged, staging rounds
    bool ok = true;
    while (ok) {
      const int slot = uc % kQueue;
      if (!wait_all(&bar[B_UFULL0 + slot], (uc / kQueue) & 1, w)) break;
      const int unit = queue.unit[slot];
      if (unit < 0) break;
      const int h = unit / p.bps;
      const int64_t q0 = ((int64_t)p.q_shard * p.bps + unit % p.bps) * 128;
      const int64_t tq = q0 + row;
      const int64_t out0 = MOD == 0 ? 0 : queue.part[slot] * (int64_t)n;
      const int64_t gi = (int64_t)h * (MOD == 0 ? n : p.n_out) + out0 + tq;
      float m_old = -INFINITY, l_old = 0.f;
      if (!p.first) {
        m_old = p.m[gi];
        l_old = p.l[gi];
      }
      const int ub = uc & 1;
      if (!wait_all(&bar[B_EPIRDY0 + ub], (uc >> 1) & 1, w)) break;
      float m_run = hm[ub * 128 + row];
      const float l_run = hl[ub * 256 + row] + hl[ub * 256 + 128 + row];
      // (rows without a legal key have no maximum, but may have got the fixed one)
      if ((MOD & kScoreCap) != 0 && l_run == 0.f) m_run = -INFINITY;
      mbar_arrive(&bar[B_HFREE0 + ub]);
      // the merge mode is one per unit: the four warps vote
      const bool grows = !p.first && m_old != -INFINITY && m_run > m_old + kRescaleThreshold;
      if (__any_sync(0xffffffffu, grows) && lane == 0) atomicOr(&epi_mode[uc & 1], 1);
      mbar_arrive(&bar[B_EVOTE]);
      if (!wait_all(&bar[B_EVOTE], uc & 1, w)) break;
      const int mode = p.lse_merge ? 3 : p.first ? 0 : (epi_mode[uc & 1] ? 2 : 1);
      // every epilogue thread has read the other flag (before this vote), and none can vote
      // on the next unit before row 0 has passed its first staging round of this one
      if (row == 0) epi_mode[(uc + 1) & 1] = 0;
      if (!wait_all(&bar[B_OFULL0 + ub], (uc >> 1) & 1, w)) break;
      tc_fence_after();
      // every role is past queue entry uc: the producer and the S cursor before the last S,
      // the PV cursor before the last PV, the softmax before the hand-over, and this group
      // before the vote
      if (row == 0) mbar_arrive(&bar[B_UEMPTY0 + slot]);
      float a_new = 1.f, a_old = 0.f, m_out = m_run, l_out = l_run;
      if (mode == 1) {
        m_out = (m_old == -INFINITY) ? m_run : m_old;
        a_new = (m_run == -INFINITY) ? 0.f : ldexpf(1.f, (int)fmaxf(m_run - m_out, -1000.f));
        l_out = l_old + l_run * a_new;
      } else if (mode == 2) {
        m_out = fmaxf(m_old, m_run);  // both integral: the factors are exact powers of two
        a_old = (m_old == -INFINITY) ? 0.f : ldexpf(1.f, (int)fmaxf(m_old - m_out, -1000.f));
        a_new = (m_run == -INFINITY) ? 0.f : ldexpf(1.f, (int)fmaxf(m_run - m_out, -1000.f));
        l_out = l_old * a_old + l_run * a_new;
      } else if (mode == 3) {
        // log-sum-exp merge in base 2: b = the call's LSE, m_old = the stored one
        const float b = l_run > 0.f ? m_run + log2f(l_run) : -INFINITY;
        const float hi = fmaxf(m_old, b), lo = fminf(m_old, b);
        m_out = lo == -INFINITY ? hi : hi + log1pf(exp2f(lo - hi)) * 1.4426950408889634f;
        a_old = m_old == -INFINITY ? 0.f : exp2f(m_old - m_out);
        a_new = b == -INFINITY ? 0.f : exp2f(b - m_out);  // weight of the normalised partial
        l_out = m_out == -INFINITY ? 0.f : 1.f;
      }
      p.m[gi] = m_out;
      p.l[gi] = l_out;
      const uint32_t ob = tO + (uint32_t)ub * 128;
      const float4* src = reinterpret_cast<const float4*>(p.o_acc + (tq * p.hq + h) * D);
#pragma unroll 1
      for (int r = 0; r < D / 32; ++r, ++k) {
        if (k > 0 && !wait_all(&bar[B_STGFREE], (k - 1) & 1, w)) { ok = false; break; }
        uint32_t x[32];
        tmem_ld32(ob + lb + r * 32, x);
        tmem_ld_wait();
        if (r == D / 32 - 1) {
          // the O buffer can take unit uc + 2
          tc_fence_before();
          mbar_arrive(&bar[B_OFREE0 + ub]);
        }
        float vals[32];
        if (mode == 3) {
          // rnd(O_old * a_old + rnd(O_call / l_call) * a_new), rnd = bf16 rounding or none
          const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
          const bool rb = p.lse_merge == 1;
#pragma unroll
          for (int t = 0; t < 32; ++t) {
            const float o = __uint_as_float(x[t]) * inv_l;
            vals[t] = (rb ? bf16_round(o) : o) * a_new;
          }
          if (!p.first) {
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const float4 o = src[r * 8 + t];
              vals[4 * t] = fmaf(o.x, a_old, vals[4 * t]);
              vals[4 * t + 1] = fmaf(o.y, a_old, vals[4 * t + 1]);
              vals[4 * t + 2] = fmaf(o.z, a_old, vals[4 * t + 2]);
              vals[4 * t + 3] = fmaf(o.w, a_old, vals[4 * t + 3]);
            }
          }
          if (rb) {
#pragma unroll
            for (int t = 0; t < 32; ++t) vals[t] = bf16_round(vals[t]);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 32; ++t) vals[t] = __uint_as_float(x[t]) * a_new;
        }
        if (mode == 2) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const float4 o = src[r * 8 + t];
            vals[4 * t] += o.x * a_old;
            vals[4 * t + 1] += o.y * a_old;
            vals[4 * t + 2] += o.z * a_old;
            vals[4 * t + 3] += o.w * a_old;
          }
        }
        stage_row32(sStg, row, vals);
        fence_proxy_async_smem();
        mbar_arrive(&bar[B_STG]);
        if (row == 0) {
          if (mbar_wait(&bar[B_STG], k & 1, w)) {
            if (mode == 1)
              tma_reduce_add_3d(&p.o_map, sStg, r * 32, (int)(out0 + q0), h);
            else
              tma_store_3d(&p.o_map, sStg, r * 32, (int)(out0 + q0), h);
            bulk_commit();
            bulk_wait_read_all();
          }
          mbar_arrive(&bar[B_STGFREE]);
        }
      }
      ++uc;
    }
    // the global writes of every TMA store / reduce this thread issued have completed
    if (row == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  if (threadIdx.x == 0) {
    // every CTA of the launch has drawn its last ticket once it gets here: the last one to
    // arrive puts the counter pair back to zero for a later launch
    __threadfence();
    if (atomicAdd(p.sched + 1, 1u) == gridDim.x - 1) {
      atomicExch(p.sched, 0u);
      atomicExch(p.sched + 1, 0u);
    }
  }
}

// everything but the shard pair, the FIRST flag and the work list: encoded once per call
template <int D, int MOD>
marble_status_t prepare(const marble_plan_t* pl, const marble_qkv_t* qkv,
                        const marble_score_t* score, const marble_state_t* st, FwdParams* prm) {
  memset(prm, 0, sizeof(*prm));
  const int64_t n = pl->n;
  if (!make_rows_map(&prm->q_map, qkv->q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, n, qkv->hq, D, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_rows_map(&prm->k_map, qkv->k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, n, qkv->hkv, D, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_rows_map(&prm->v_map, qkv->v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, n, qkv->hkv, D, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_rows_map(&prm->o_map, st->o_acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, n, qkv->hq, D, 32,
                     128, CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(MARBLE_ERR_CUDA, "cuTensorMapEncodeTiled failed for Q/K/V/O_acc");
  prm->step_ptr = pl->step_ptr;
  prm->step_col = pl->step_col;
  prm->step_tag = pl->step_tag;
  prm->tracks = pl->tracks;
  prm->kiv = pl->kiv;
  prm->kiv_chunk = pl->kiv_chunk;
  prm->qidx = pl->perm;
  prm->iv_block = pl->iv_block;
  prm->o_acc = st->o_acc;
  prm->m = st->m;
  prm->l = st->l;
  prm->err = pl->err;
  prm->wait_ns = wait_limit_ns();
  prm->n = prm->n_out = n;
  prm->parts = 1;
  prm->P = pl->P;
  prm->bps = (int)pl->bps;
  prm->hq = qkv->hq;
  prm->group = qkv->hq / qkv->hkv;
  prm->units = (int)(pl->bps * qkv->hq);
  prm->W = pl->W;
  const float scale = qkv->scale > 0.f ? qkv->scale : 1.0f / sqrtf((float)D);
  prm->scale_log2 = scale * 1.4426950408889634f;
  if (MOD & kScoreCap) set_cap(&prm->score, score->cap, scale);
  if (MOD & kScoreBias) prm->score.slopes = score->slopes;
  prm->score.consecutive = pl->pos_is_index;
  if (once_per_device((D == 128 ? 1 : 2) + 4 * MOD)) {
    cudaError_t e = cudaFuncSetAttribute(k_attn_fwd<D, MOD>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Smem<D>::bytes());
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(k_attn_fwd)");
  }
  {
    // the warpgroups' budgets are drawn from the registers that the block is launched with:
    // with fewer the growing warpgroups would wait for ever (checked on every call)
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, k_attn_fwd<D, MOD>);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(k_attn_fwd)");
    if (fa.numRegs < kRegsLaunch)
      return fail(MARBLE_ERR_UNSUPPORTED, "forward kernel built with " + std::to_string(fa.numRegs) +
                                              " registers per thread, fewer than its split needs");
  }
  return MARBLE_OK;
}

template <int D, int MOD>
marble_status_t launch_steps(const marble_plan_t* pl, const marble_qkv_t* qkv,
                             const marble_score_t* score, int n_steps, const int* q_shards, const int* kv_shards, const uint32_t* flags,
                             const marble_state_t* st, cudaStream_t s) {
  FwdParams base;
  marble_status_t rc = prepare<D, MOD>(pl, qkv, score, st, &base);
  if (rc != MARBLE_OK) return rc;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // Steps of different q shards touch disjoint rows of the state: q shard r runs on stream
  // r mod ns (the caller's stream and up to three side streams), so that the tails of
  // launches of different shards overlap.  Steps of one q shard stay in order on one stream.
  constexpr int kFwdSide = 3;
  cudaStream_t st_of[1 + kFwdSide] = {s};
  int ns = 1;
  if (n_steps > 1)
    for (int k = 0; k < kFwdSide; ++k) {
      cudaStream_t x = side_stream(k);
      if (!x) break;
      cudaError_t e = stream_fork(s, x);
      if (e != cudaSuccess) return cuda_fail(e, "fork of the forward streams");
      st_of[ns++] = x;
    }
  int span[1 + kFwdSide], launches[1 + kFwdSide] = {0};
  for (int k = 0; k < ns; ++k) span[k] = timing_begin(st_of[k]);
  for (int i = 0; i < n_steps; ++i) {
    FwdParams prm = base;
    prm.q_shard = q_shards[i];
    prm.kv_shard = kv_shards[i];
    prm.first = (flags[i] & MARBLE_STEP_FIRST) ? 1 : 0;
    prm.lse_merge = (flags[i] & MARBLE_STEP_BF16_MERGE) ? 1 : (flags[i] & MARBLE_STEP_FP32_MERGE) ? 2 : 0;
    // one stabiliser beside a bias needs the rows' own keys among the step's (see kFixedCap)
    if (prm.kv_shard >= 0 && prm.kv_shard != prm.q_shard) prm.score.bias_fixed = 0;
    const int64_t seg = (int64_t)prm.q_shard * (pl->P + 1) + (prm.kv_shard >= 0 ? prm.kv_shard : pl->P);
    prm.order = pl->fwd_order + seg * pl->bps;
    prm.nwork = pl->h_fwd_nwork[seg] * qkv->hq;
    if (prm.nwork == 0 && !prm.first) continue;  // nothing to add to the state
    prm.sched = sched_slot(pl);
    // persistent: one CTA per SM (each takes all 512 TMEM columns); the FIRST call also
    // initialises the units without tiles, spread over the whole grid
    const int want = prm.first ? base.units : prm.nwork;
    // with side streams, a launch takes at most half the SMs: launches of different q shards
    // then share the GPU instead of one waiting for the other's tail
    const int cap = ns > 1 ? (sms + 1) / 2 : sms;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const int k = prm.q_shard % ns;
    k_attn_fwd<D, MOD><<<grid, kThreads, Smem<D>::bytes(), st_of[k]>>>(prm);
    ++launches[k];
  }
  for (int k = 0; k < ns; ++k) timing_end(span[k], st_of[k], kTimeFwd, launches[k]);
  for (int k = 1; k < ns; ++k) {
    cudaError_t e = stream_fork(st_of[k], s);
    if (e != cudaSuccess) return cuda_fail(e, "join of the forward streams");
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "launch k_attn_fwd");
  return MARBLE_OK;
}

// Few and long rows: the fused forward's units are then fewer than the SMs, or the longest of them
// sets the launch's length.  Each row's list is cut into `parts` pieces of one length, units of
// their own that write (O, m, l) to a scratch; this kernel joins a row's pieces.  Their m are
// integers, so that every factor is an exact power of two, and they are added in order.
struct JoinParams {
  const float *o, *m, *l;  // [parts * n][hq][D], [hq][parts * n] twice
  float *o_out, *m_out, *l_out;
  const int64_t* step_ptr;
  long long n;
  int P, hq, parts;
};

template <int D>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ JoinParams p) {
  constexpr unsigned kRow4 = D / 4;
  const unsigned x = blockIdx.x * 256 + threadIdx.x, th = x / kRow4;  // (token, head)
  const unsigned tq = th / (unsigned)p.hq, h = th - tq * (unsigned)p.hq;
  if (tq >= (unsigned)p.n) return;
  const unsigned nq = tq / 128;
  const int T = (int)(p.step_ptr[(size_t)(nq + 1) * p.P] - p.step_ptr[(size_t)nq * p.P]);
  const int len = part_tiles(T, p.parts);
  const size_t one = (size_t)p.n * p.hq;
  const float4* from = reinterpret_cast<const float4*>(p.o) + x;
  float m[kMaxParts], l[kMaxParts], top = -INFINITY;
  float4 v[kMaxParts];
#pragma unroll
  for (int i = 0; i < kMaxParts; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < p.parts && i * len < T) {  // (T 0: no piece)
      const size_t at = ((size_t)h * p.parts + i) * p.n + tq;
      m[i] = p.m[at];
      l[i] = p.l[at];
      v[i] = __ldcs(from + i * one * kRow4);
    }
    top = fmaxf(top, m[i]);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxParts; ++i) {
    // a piece without a legal key has m = -inf and zeros; its factor is 0 (or 1 where all are
    // so), not left out, so that a NaN in it stays one
    const float f = m[i] == top ? 1.f : ldexpf(1.f, (int)fmaxf(m[i] - top, -1000.f));
    sum = fmaf(l[i], f, sum);
    o = make_float4(fmaf(v[i].x, f, o.x), fmaf(v[i].y, f, o.y), fmaf(v[i].z, f, o.z),
                    fmaf(v[i].w, f, o.w));
  }
  reinterpret_cast<float4*>(p.o_out)[x] = o;
  if (x % kRow4 == 0) {
    p.m_out[(size_t)h * p.n + tq] = top;
    p.l_out[(size_t)h * p.n + tq] = sum;
  }
}

// The pieces of a row (1: whole rows), for scored calls: plain calls keep the order in which they
// sum.  A tile takes a lone unit 1.2 us.  Whole rows take the longest one's time; pieces an SM's
// share of all tiles and half a piece more, and then the join: a launch, about 5 tiles, and the
// pieces' bytes, 4 MB a tile (at most 1 GB of them).  Causal rows, d = 128, capped, whole / in
// pieces, with the finalize: 2048 tokens 2 heads 35 / 28 us, 4096 tokens 1 head 53 / 32, 8192
// tokens 1 head 92 / 53, 2 heads 93 / 83, 16384 tokens 1 head 169 / 134.  Where the rule keeps
// whole rows: 2048 tokens 4 heads 35 / 35, 4096 tokens 4 heads 55 / 57.
int row_parts(const marble_plan_t* pl, int64_t hq, int d, int sms) {
  int64_t longest = 0;
  for (int r = 0; r < pl->P; ++r)
    longest = std::max<int64_t>(longest, pl->h_step_max[(size_t)r * (pl->P + 1) + pl->P]);
  const int64_t share = (pl->nnz * hq + sms - 1) / sms;
  const int64_t parts = std::min<int64_t>(kMaxParts, longest / std::max<int64_t>(share, 4));
  if (parts < 2) return 1;
  const int64_t piece = (longest + parts - 1) / parts;
  const int64_t saved = longest - std::max(piece, share + piece / 2);
  const int64_t bytes = (parts + 1) * pl->n * hq * d * 4;
  return bytes <= int64_t(1) << 30 && saved > 5 + (bytes >> 22) ? (int)parts : 1;
}

// The fused forward: one launch over every (q block, q head) of every shard, each row
// walking its tiles in ring order (kv shard (r - s) mod P at step s, the plan's ring-ordered
// copy of its lists) with the fp32 state held on chip from the first step to the last; the
// state is written once, as the FIRST step of the per-step path writes it.
template <int D, int MOD>
marble_status_t launch_fused(const marble_plan_t* pl, const marble_qkv_t* qkv,
                             const marble_score_t* score, const marble_state_t* st,
                             cudaStream_t s) {
  FwdParams prm;
  marble_status_t rc = prepare<D, MOD>(pl, qkv, score, st, &prm);
  if (rc != MARBLE_OK) return rc;
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // every block of the pack as one shard of nb blocks, whole rows, ring-ordered lists
  prm.bps = (int)pl->nb;
  prm.q_shard = 0;
  prm.kv_shard = -1;
  prm.first = 1;
  prm.lse_merge = 0;
  prm.step_col = pl->ring_col;
  prm.step_tag = pl->ring_tag;
  prm.order = pl->order_all;
  prm.units = (int)(pl->nb * qkv->hq);
  prm.nwork = pl->h_nwork_all[0] * qkv->hq;
  prm.sched = sched_slot(pl);
  void* pieces = nullptr;
  if constexpr (MOD != 0) {
    const int parts = row_parts(pl, qkv->hq, D, sms);
    const int64_t rows = parts * pl->n * qkv->hq;
    if (parts > 1 && dev_alloc(&pieces, rows * (D + 2) * sizeof(float), s, true) != cudaSuccess) {
      (void)cudaGetLastError();  // no room for pieces: whole rows
      pieces = nullptr;
    }
    if (pieces) {
      prm.parts = parts;
      prm.n_out = parts * pl->n;
      prm.nwork *= parts;
      prm.units *= parts;
      prm.o_acc = static_cast<float*>(pieces);
      prm.m = prm.o_acc + rows * D;
      prm.l = prm.m + rows;
      if (!make_rows_map(&prm.o_map, prm.o_acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, prm.n_out,
                         qkv->hq, D, 32, 128, CU_TENSOR_MAP_SWIZZLE_128B)) {
        dev_free(pieces, s);
        return fail(MARBLE_ERR_CUDA, "cuTensorMapEncodeTiled failed for the rows' pieces");
      }
    }
  }
  const unsigned grid = (unsigned)(prm.units < sms ? prm.units : sms);
  const int span = timing_begin(s);
  k_attn_fwd<D, MOD><<<grid, kThreads, Smem<D>::bytes(), s>>>(prm);
  if (pieces) {
    const JoinParams j{prm.o_acc, prm.m, prm.l, st->o_acc, st->m, st->l, pl->step_ptr, pl->n,
                       pl->P, qkv->hq, prm.parts};
    const int64_t n4 = pl->n * qkv->hq * (D / 4);
    k_attn_join<D><<<(unsigned)((n4 + 255) / 256), 256, 0, s>>>(j);
  }
  timing_end(span, s, kTimeFwd, pieces ? 2 : 1);
  cudaError_t e = cudaGetLastError();
  if (pieces) dev_free(pieces, s);
  if (e != cudaSuccess) return cuda_fail(e, "launch k_attn_fwd (fused)");
  return MARBLE_OK;
}

// f(d, mod) with the forward's variant of the score
template <class F>
marble_status_t with_fwd_variant(int d, const marble_score_t* score, F f) {
  const int bits = score_bits(score);
  return with_variant(d, bits, [&](auto dd, auto mod) {
    if constexpr (mod() == kScoreCap) {
      if (score->cap * 1.4426950408889634f <= kFixedCap)
        return f(dd, std::integral_constant<int, kScoreCap | kScoreFixed>{});
    }
    return f(dd, mod);
  });
}

}  // namespace

marble_status_t run_attn_fwd_fused(const marble_plan_t* p, const marble_qkv_t* qkv,
                                   const marble_score_t* score, const marble_state_t* st,
                                   cudaStream_t s) {
  if ((int64_t)p->nb * qkv->hq > INT_MAX)
    return fail(MARBLE_ERR_UNSUPPORTED, "too many (block, head) work units");
  return with_fwd_variant(qkv->d, score, [&](auto d, auto mod) {
    return launch_fused<d(), mod()>(p, qkv, score, st, s);
  });
}

marble_status_t run_attn_fwd(const marble_plan_t* p, const marble_qkv_t* qkv,
                             const marble_score_t* score, int n_steps, const int* q_shards,
                             const int* kv_shards, const uint32_t* flags, const marble_state_t* st,
                             cudaStream_t s) {
  return with_fwd_variant(qkv->d, score, [&](auto d, auto mod) {
    return launch_steps<d(), mod()>(p, qkv, score, n_steps, q_shards, kv_shards, flags, st, s);
  });
}

}  // namespace marble
