// Rotary positions with several axes, with the heads' RMS norm and the move between original
// and plan order in the same pass, and the gradient of all three.
//
// For a token at positions pos[0 .. n_axes) and a rotated pair i of a head, (a, b):
//   angle = pos[axis(i)] * freq(i),   a' = a cos - b sin,   b' = a sin + b cos,
// with, before it, x <- x * r * w, r = 1 / sqrt(mean x^2 + eps), where a norm weight w is given.
// Gradient, g = the incoming gradient turned back by the same angle:
//   without a norm dx = g;   with one, xh = x * r:   dw = sum over rows of g * xh,
//   dx = r * (g * w - xh * mean(g * w * xh)).
//
// What bounds both kernels is memory: every element is read once and written once (2 + 2 bytes;
// the gradient 4 + 2, and 2 more for x where there is a norm).  One warp takes a token and walks
// its heads, 32 * 16 / d heads at a time: a thread holds both members of 8 pairs of one head, so
// that the rotation needs no exchange and the norm only a butterfly over d / 16 lanes.  The 8
// cosines and sines of a thread's pairs are computed once per token and serve all of its heads.
// Few tokens are split further, a warp for every few heads.  A pass over 262,144 tokens of 32 + 8
// heads of 128 with values and both norms takes 1002 us forward (6.43 TB/s, 96% of a plain copy's
// rate) and 2001 us for the gradient (6.18 TB/s, 92%).  Loading a
// warp's next heads before storing the present ones was slower (1.14 against 1.07 ms): with 32
// warps on an SM (the gradient with a norm: 16) enough loads are in flight, and the registers
// are better spent on warps.
//
// The angle is a fraction of a turn in 64-bit fixed point: freq / (2 pi) mod 1 scaled by 2^64,
// times the position, modulo 2^64.  The product drops whole turns exactly, so a position of
// 2^31 - 1 has the accuracy of position 1; what is left is rounded to fp32 (2^-25 turns) only
// then, and sincospif does the rest.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace marble {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 64;
constexpr int kPartialCtas = MARBLE_ROPE_WORKSPACE_BYTES / (2 * 128 * 4);

struct HeadPart {
  const void* src;
  void* dst;
  const void* x;                 // gradient: the forward's input (norm only)
  long long src_stride, dst_stride, x_stride;  // elements between tokens
  int heads, groups;             // heads, and warp iterations over them
};

struct RopeParams {
  HeadPart part[3];              // q, k, v
  const int32_t* perm;           // plan index -> original index, or null
  const int32_t* pos;            // [n_axes][n], original order
  const float* weight[2];        // q, k: norm weights or null
  float* partial;                // gradient: [ctas][2][D] partial sums of dw
  unsigned long long turn[kMaxPairs];  // turns per position, * 2^64; 0: not rotated
  uint8_t axis[kMaxPairs];
  long long n;
  int rot_chunks;                // rot_dim / 16: threads of a head whose pairs are rotated
  int split;                     // warps per token
  float eps;
};

// The two 8-channel chunks of thread j of a head.  Halves: the pair of channel c < rot/2 is
// c + rot/2, the channels from rot on are passed through.  Adjacent: pairs (2 i, 2 i + 1).
template <bool kAdjacent>
__device__ __forceinline__ void chunks_of(int j, int rot_chunks, int* ca, int* cb) {
  if (kAdjacent || j >= rot_chunks) {
    *ca = 2 * j;
    *cb = 2 * j + 1;
  } else {
    *ca = j;
    *cb = j + rot_chunks;
  }
}

// element u (0..15) of thread j's registers (a[0..8), b[0..8)) -> channel of the head
template <bool kAdjacent>
__device__ __forceinline__ int channel_of(int j, int u, int rot_chunks) {
  if (kAdjacent) return 16 * j + 2 * (u & 7) + (u >> 3);
  int ca, cb;
  chunks_of<false>(j, rot_chunks, &ca, &cb);
  return (u < 8 ? ca : cb) * 8 + (u & 7);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}
// chunk order (va: chunk ca, vb: chunk cb) <-> pair order (a: first members, b: second ones)
template <bool kAdjacent>
__device__ __forceinline__ void to_pairs(const float (&va)[8], const float (&vb)[8], float (&a)[8],
                                         float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = kAdjacent ? (i < 4 ? va[2 * i] : vb[2 * i - 8]) : va[i];
    b[i] = kAdjacent ? (i < 4 ? va[2 * i + 1] : vb[2 * i - 7]) : vb[i];
  }
}
template <bool kAdjacent>
__device__ __forceinline__ void to_chunks(const float (&a)[8], const float (&b)[8], float (&va)[8],
                                          float (&vb)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    va[i] = kAdjacent ? ((i & 1) ? b[i / 2] : a[i / 2]) : a[i];
    vb[i] = kAdjacent ? ((i & 1) ? b[4 + i / 2] : a[4 + i / 2]) : b[i];
  }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 y = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
  f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}

// The tables a CTA's threads read, in the order they read them: thread j's element u at
// [u][j], so that the threads of a head read consecutive words.
template <int D>
struct Tables {
  static constexpr int kTpr = D / 16;    // threads per head
  unsigned long long turn[8 * kTpr];
  uint8_t axis[8 * kTpr];
  float4 weight[2][4 * kTpr];            // elements 4 u4 .. 4 u4 + 3 of thread j at [u4][j]
};

template <int D, bool kAdjacent>
__device__ __forceinline__ void fill_tables(const RopeParams& p, Tables<D>& t) {
  constexpr int kTpr = D / 16;
  for (int x = threadIdx.x; x < 8 * kTpr; x += kThreads) {
    const int u = x / kTpr, j = x % kTpr;
    t.turn[x] = p.turn[8 * j + u];
    t.axis[x] = p.axis[8 * j + u];
  }
  for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
    const int w = x / D, c = x % D, j = c / 16, u = c % 16;
    if (p.weight[w])
      reinterpret_cast<float*>(&t.weight[w][(u >> 2) * kTpr + j])[u & 3] =
          p.weight[w][channel_of<kAdjacent>(j, u, p.rot_chunks)];
  }
  __syncthreads();
}

template <int D>
__device__ __forceinline__ void angles(const RopeParams& p, const Tables<D>& t, int j, int64_t o,
                                       float (&c)[8], float (&s)[8]) {
  constexpr int kTpr = D / 16;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t at = p.pos[(int64_t)t.axis[u * kTpr + j] * p.n + o];
    const unsigned long long turns = (unsigned long long)at * t.turn[u * kTpr + j];
    // the upper 32 bits as a signed fraction: half turns in [-1, 1)
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s[u], &c[u]);
  }
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int D>
__device__ __forceinline__ void weights_of(const Tables<D>& t, int which, int j, float (&w)[16]) {
#pragma unroll
  for (int u4 = 0; u4 < 4; ++u4) {
    const float4 v = t.weight[which][u4 * (D / 16) + j];
    w[4 * u4] = v.x;
    w[4 * u4 + 1] = v.y;
    w[4 * u4 + 2] = v.z;
    w[4 * u4 + 3] = v.w;
  }
}

template <int D, bool kAdjacent>
__global__ void __launch_bounds__(kThreads, 4) k_rope(const __grid_constant__ RopeParams p) {
  constexpr int kTpr = D / 16, kHpi = 32 / kTpr;
  __shared__ Tables<D> t;
  fill_tables<D, kAdjacent>(p, t);
  const int lane = threadIdx.x & 31, j = lane % kTpr, sub = lane / kTpr;
  const bool rotated = j < p.rot_chunks;
  int ca, cb;
  chunks_of<kAdjacent>(j, p.rot_chunks, &ca, &cb);
  const unsigned items = (unsigned)(p.n * p.split), warps = gridDim.x * kWarps;
  for (unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5); w < items; w += warps) {
    const int64_t i = p.split == 1 ? w : w / (unsigned)p.split;
    const int64_t o = p.perm ? p.perm[i] : i;
    int g = (int)(w - (unsigned)i * p.split);  // the warp's groups: g, g + split, ...
    float c[8], s[8];
    angles<D>(p, t, j, o, c, s);
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const HeadPart& hp = p.part[which];
      const uint4* src =
          static_cast<const uint4*>(hp.src) + (o * hp.src_stride + (g * kHpi + sub) * D) / 8;
      uint4* dst = static_cast<uint4*>(hp.dst) + (i * hp.dst_stride + (g * kHpi + sub) * D) / 8;
      const int step = p.split * (kHpi * D / 8);
      for (; g < hp.groups; g += p.split, src += step, dst += step) {
        const bool live = g * kHpi + sub < hp.heads;
        uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
        if (live) {
          ra = __ldcs(src + ca);
          rb = __ldcs(src + cb);
        }
        // channels that are neither scaled nor turned keep their bits (a NaN's too)
        if (which < 2 && (rotated || p.weight[which & 1])) {
          float va[8], vb[8], a[8], b[8];
          unpack8(ra, va);
          unpack8(rb, vb);
          to_pairs<kAdjacent>(va, vb, a, b);
          if (p.weight[which & 1]) {
            float ss = 0.f, wt[16];
#pragma unroll
            for (int u = 0; u < 8; ++u) ss = fmaf(a[u], a[u], fmaf(b[u], b[u], ss));
            const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + p.eps);
            weights_of<D>(t, which & 1, j, wt);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              a[u] *= r * wt[u];
              b[u] *= r * wt[8 + u];
            }
          }
          if (rotated) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float x = a[u], y = b[u];
              a[u] = x * c[u] - y * s[u];
              b[u] = x * s[u] + y * c[u];
            }
          }
          to_chunks<kAdjacent>(a, b, va, vb);
          ra = pack8(va);
          rb = pack8(vb);
        }
        if (live) {
          dst[ca] = ra;
          dst[cb] = rb;
        }
      }
      g -= hp.groups;
    }
  }
}

// The gradient: rows of fp32 gradients in plan order in, bf16 in original order out.  With a
// norm, a thread sums dw of its 16 channels in registers over one tensor's heads of a token, then
// adds them to its own words of shared memory (registers for q and k both would cost a third of
// the warps in flight; with one loop per tensor and the sums of one at a time 64K tokens of 32 / 8
// heads of 128 take 507 us instead of 614); a CTA's sums go to partial[cta] and k_rope_dw adds those in a fixed
// order, so that dw does not depend on timing.
template <int D, bool kAdjacent, bool kNorm>
__global__ void __launch_bounds__(kThreads, kNorm ? 2 : 4)
    k_rope_bwd(const __grid_constant__ RopeParams p) {
  constexpr int kTpr = D / 16, kHpi = 32 / kTpr;
  __shared__ Tables<D> t;
  __shared__ float4 sums[2][4][kNorm ? kThreads : 1];  // q, k: the 16 sums of every thread
  fill_tables<D, kAdjacent>(p, t);
  const int lane = threadIdx.x & 31, j = lane % kTpr, sub = lane / kTpr;
  const bool rotated = j < p.rot_chunks;
  int ca, cb;
  chunks_of<kAdjacent>(j, p.rot_chunks, &ca, &cb);
  if constexpr (kNorm) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sums[k >> 2][k & 3][threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const unsigned items = (unsigned)(p.n * p.split), warps = gridDim.x * kWarps;
  for (unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5); w < items; w += warps) {
    const int64_t i = p.split == 1 ? w : w / (unsigned)p.split;
    const int64_t o = p.perm ? p.perm[i] : i;
    int g = (int)(w - (unsigned)i * p.split);  // the warp's groups: g, g + split, ...
    float c[8], s[8];
    angles<D>(p, t, j, o, c, s);
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const HeadPart& hp = p.part[which];
      const int at = (g * kHpi + sub) * D, step = p.split * (kHpi * D);
      const float* src = static_cast<const float*>(hp.src) + i * hp.src_stride + at;
      uint4* dst = static_cast<uint4*>(hp.dst) + (o * hp.dst_stride + at) / 8;
      const uint4* x = static_cast<const uint4*>(hp.x) + (o * hp.x_stride + at) / 8;
      const bool norm = kNorm && which < 2 && p.weight[which & 1];
      float dw[16];
      if (norm) {
#pragma unroll
        for (int u = 0; u < 16; ++u) dw[u] = 0.f;
      }
      for (; g < hp.groups; g += p.split, src += step, dst += step / 8, x += step / 8) {
        const bool live = g * kHpi + sub < hp.heads;
        float va[8], vb[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) va[u] = vb[u] = 0.f;
        uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
        if (live) {
          load8(src + ca * 8, va);
          load8(src + cb * 8, vb);
          if (norm) {
            xa = __ldcs(x + ca);
            xb = __ldcs(x + cb);
          }
        }
        if (which < 2) {
          float a[8], b[8];
          to_pairs<kAdjacent>(va, vb, a, b);
          if (rotated) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float y = a[u], z = b[u];
              a[u] = y * c[u] + z * s[u];
              b[u] = z * c[u] - y * s[u];
            }
          }
          if (norm) {
            float x8a[8], x8b[8], x1[8], x2[8], wt[16], ss = 0.f, dot = 0.f;
            unpack8(xa, x8a);
            unpack8(xb, x8b);
            to_pairs<kAdjacent>(x8a, x8b, x1, x2);
#pragma unroll
            for (int u = 0; u < 8; ++u) ss = fmaf(x1[u], x1[u], fmaf(x2[u], x2[u], ss));
            const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + p.eps);
            weights_of<D>(t, which & 1, j, wt);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              x1[u] *= r;
              x2[u] *= r;
              dw[u] = fmaf(a[u], x1[u], dw[u]);
              dw[8 + u] = fmaf(b[u], x2[u], dw[8 + u]);
              a[u] *= wt[u];
              b[u] *= wt[8 + u];
              dot = fmaf(a[u], x1[u], fmaf(b[u], x2[u], dot));
            }
            const float m = row_sum<D>(dot) * (1.f / D);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              a[u] = r * (a[u] - x1[u] * m);
              b[u] = r * (b[u] - x2[u] * m);
            }
          }
          to_chunks<kAdjacent>(a, b, va, vb);
        }
        if (live) {
          dst[ca] = pack8(va);
          dst[cb] = pack8(vb);
        }
      }
      g -= hp.groups;
      if (norm) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4& v = sums[which & 1][k][kNorm ? threadIdx.x : 0];
          v = make_float4(v.x + dw[4 * k], v.y + dw[4 * k + 1], v.z + dw[4 * k + 2],
                          v.w + dw[4 * k + 3]);
        }
      }
    }
  }
  if constexpr (kNorm) {
    // channel x of weight k: thread j's element u, over the CTA's threads with that j in order
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
      const int k = x / D, e = x % D, jj = e / 16, u = e % 16;
      float v = 0.f;
      for (int q = jj; q < kThreads; q += kTpr)
        v += reinterpret_cast<const float*>(&sums[k][u >> 2][q])[u & 3];
      p.partial[(int64_t)blockIdx.x * 2 * D + k * D + channel_of<kAdjacent>(jj, u, p.rot_chunks)] = v;
    }
  }
}

// dw[x] = the CTAs' partial sums of channel x, 32 channels a block, 32 interleaved slices of the
// CTAs each, added in a fixed order
__global__ void __launch_bounds__(1024) k_rope_dw(const float* __restrict__ partial, int ctas,
                                                  int d, float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int x = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int c = slice; c < ctas; c += 32) v += partial[(int64_t)c * 2 * d + x];
  s[slice][lane] = v;
  __syncthreads();
  // warp `slice` adds the slices of channel `slice` of the block's 32
  v = s[lane][slice];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  const int ch = blockIdx.x * 32 + slice;
  float* out = ch < d ? dwq : dwk;
  if (lane == 0 && out) out[ch % d] = v;
}

// freq / (2 pi) modulo 1 as a 64-bit fixed-point fraction.  The quotient is kept as a sum of two
// doubles, so that the last of the 64 bits is still right.
unsigned long long turns_fixed(double freq) {
  constexpr double kHi = 0.15915494309189535;       // 1 / (2 pi), rounded to a double
  constexpr double kLo = -9.839338337591243e-18;    // and what the rounding left
  const double f = std::fabs(freq);
  const double hi = f * kHi;
  const double lo = std::fma(f, kHi, -hi) + f * kLo;
  unsigned long long t = (unsigned long long)std::ldexp(std::fmod(hi, 1.0), 64);
  t += (unsigned long long)(long long)std::ldexp(std::fmod(lo, 0.25), 64);
  return freq < 0 ? 0ull - t : t;
}

void set_part(HeadPart& hp, const void* src, void* dst, const void* x, int64_t ss, int64_t ds,
              int64_t xs, int heads, int d) {
  hp = HeadPart{src, dst, x, ss, ds, xs, src ? heads : 0, 0};
  hp.groups = (hp.heads * (d / 16) + 31) / 32;
}

// everything the two directions share
void set_params(const marble_plan_t* plan, int64_t n, const marble_rope_t* rope, int d,
                RopeParams* out) {
  RopeParams& p = *out;
  p.perm = plan ? plan->perm : nullptr;
  p.pos = rope->pos;
  p.weight[0] = rope->q_weight;
  p.weight[1] = rope->k_weight;
  p.eps = rope->eps;
  p.n = n;
  p.rot_chunks = rope->rot_dim / 16;
  for (int i = 0; i < kMaxPairs; ++i) {
    const bool turn = i < rope->rot_dim / 2;
    p.turn[i] = turn ? turns_fixed(rope->inv_freq[i]) : 0;
    p.axis[i] = turn ? (uint8_t)rope->axis[i] : 0;
  }
}

// CTAs and warps per token.  A warp walks all heads of a token (the angles are then computed
// once) unless that leaves the GPU without work: then a token is split over the fewest warps
// that give every SM 16 of them, a group of heads each at the most.  No more CTAs than run at
// once (per_sm on every SM): each fills its tables once and takes tokens until they run out.
int set_grid(RopeParams* p, int per_sm, int max_ctas) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t groups = p->part[0].groups + p->part[1].groups + p->part[2].groups;
  const int64_t want = (int64_t)sms * 16;
  p->split = (int)std::max<int64_t>(1, std::min<int64_t>(groups, (want + p->n - 1) / p->n));
  const int64_t ctas = (p->n * p->split + kWarps - 1) / kWarps;
  return (int)std::min<int64_t>(ctas, std::min(sms * per_sm, max_ctas));
}

}  // namespace

cudaError_t launch_rope(const marble_plan_t* plan, int64_t n, const marble_rope_t* rope,
                        const marble_heads_t* src, const marble_heads_t* dst, cudaStream_t s) {
  RopeParams p;
  memset(&p, 0, sizeof(p));
  const int d = src->d;
  set_params(plan, n, rope, d, &p);
  set_part(p.part[0], src->q, dst->q, nullptr, src->q_stride, dst->q_stride, 0, src->hq, d);
  set_part(p.part[1], src->k, dst->k, nullptr, src->k_stride, dst->k_stride, 0, src->hkv, d);
  set_part(p.part[2], src->v, dst->v, nullptr, src->v_stride, dst->v_stride, 0, src->hkv, d);
  const int ctas = set_grid(&p, 4, 1 << 20);
  const bool adj = rope->pairing == MARBLE_PAIR_ADJACENT;
  if (d == 128)
    (adj ? k_rope<128, true> : k_rope<128, false>)<<<ctas, kThreads, 0, s>>>(p);
  else
    (adj ? k_rope<64, true> : k_rope<64, false>)<<<ctas, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope_bwd(const marble_plan_t* plan, int64_t n, const marble_rope_t* rope,
                            const marble_heads_t* x, const marble_heads_t* grad,
                            const marble_heads_t* dx, float* dwq, float* dwk, float* workspace,
                            cudaStream_t s) {
  const bool norm = rope->q_weight || rope->k_weight;
  const int d = grad->d;
  int ctas = 0;
  if (n > 0) {
    RopeParams p;
    memset(&p, 0, sizeof(p));
    set_params(plan, n, rope, d, &p);
    p.partial = workspace;
    const marble_heads_t none = {};
    const marble_heads_t& xs = x ? *x : none;
    set_part(p.part[0], grad->q, dx->q, xs.q, grad->q_stride, dx->q_stride, xs.q_stride, grad->hq, d);
    set_part(p.part[1], grad->k, dx->k, xs.k, grad->k_stride, dx->k_stride, xs.k_stride, grad->hkv, d);
    set_part(p.part[2], grad->v, dx->v, nullptr, grad->v_stride, dx->v_stride, 0, grad->hkv, d);
    ctas = set_grid(&p, norm ? 2 : 4, norm ? kPartialCtas : 1 << 20);
    const bool adj = rope->pairing == MARBLE_PAIR_ADJACENT;
    auto kernel = d == 128 ? (adj ? (norm ? k_rope_bwd<128, true, true> : k_rope_bwd<128, true, false>)
                                  : (norm ? k_rope_bwd<128, false, true> : k_rope_bwd<128, false, false>))
                           : (adj ? (norm ? k_rope_bwd<64, true, true> : k_rope_bwd<64, true, false>)
                                  : (norm ? k_rope_bwd<64, false, true> : k_rope_bwd<64, false, false>));
    kernel<<<ctas, kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (norm) k_rope_dw<<<2 * d / 32, 1024, 0, s>>>(workspace, ctas, d, dwq, dwk);
  return cudaGetLastError();
}

}  // namespace marble
