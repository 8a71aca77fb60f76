// The attention over the paged cache (attn_cached.cuh): what a call's kernels get, and the kernels
// for heads of 128.
#include <cstring>
#include <mutex>

#include "attn_cached.cuh"

namespace marble {

marble_status_t launch_d128(cached::AttnParams& p, int type, int nt, bool scored, int grid,
                            int join_rows, cudaStream_t s) {
  return cached::launch_d<128>(p, type, nt, scored, grid, join_rows, s);
}

marble_status_t run_attn_cached(int64_t n, const marble_cache_t* c, const marble_seqs_t* seqs,
                                const marble_attn_cached_t* a, const marble_score_t* score,
                                cudaStream_t s) {
  cached::AttnParams p;
  memset(&p, 0, sizeof(p));
  const bool quant = c->type != MARBLE_CACHE_BF16;
  const int keys = !quant && c->d == 128 ? 32 : 64;
  p.box = 16;
  while (p.box < keys && c->page_tokens % (2 * p.box) == 0) p.box *= 2;
  const auto maps = [&] {
    return cached::pages_map(&p.kmap, c->k, c->type, c->k_stride, *c, p.box) &&
           cached::pages_map(&p.vmap, c->v, c->type, c->v_stride, *c, p.box);
  };
  // (a thread that no call has given the device's context yet gets it from cudaSetDevice)
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  if (!maps() && (cudaSetDevice(dev) != cudaSuccess || !maps()))
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
      p.cap2 = (float)(score->cap * 1.4426950408889634);
      p.inv_cap2 = (float)(1.0 / (score->cap * 1.4426950408889634));
    }
  }
  p.hkv = c->hkv;
  p.group = a->hq / c->hkv;
  p.window = a->window;
  p.span = a->span ? 1 : 0;
  const int64_t rows = std::min<int64_t>(64, (int64_t)p.group * std::max(1, a->new_tokens));
  const int nt = rows <= 8 ? 1 : 2;
  p.row_warps = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  p.rows = 8 * nt * p.row_warps;
  while ((1 << p.rows_log) < p.rows) ++p.rows_log;
  // (the computing warps do four chunks side by side in the time of one; 3 to 9 differ by 2%)
  p.grain = nt == 1 ? 5 : 4 * 5;
  p.limit_ns = wait_limit_ns();
  p.drain_ns = std::max<uint64_t>(p.limit_ns, 1000000000ull);  // copies under way always land
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // workspace: a word for timeouts without a status, the joins, the pieces
  const int64_t piece = p.rows * (int64_t)(c->d + 2) * 4;
  const int64_t most = (MARBLE_ATTN_CACHED_WORKSPACE_BYTES - 65536) / (2 * piece);
  const int grid = (int)std::min<int64_t>(std::min<int64_t>(2 * sms, most), 2000);
  char* ws = static_cast<char*>(a->workspace);
  p.err = seqs->status ? reinterpret_cast<unsigned*>(seqs->status) : reinterpret_cast<unsigned*>(ws);
  p.joins = reinterpret_cast<int4*>(ws + 256);
  p.part_ml = reinterpret_cast<float2*>(ws + 65536);
  p.part_o = reinterpret_cast<float*>(ws + 65536 + 2 * (int64_t)grid * p.rows * 8);
  // The call's two kernels follow each other in the stream: another thread's call with the same
  // workspace, ordered by the stream, must not come between them.
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  return c->d == 128 ? launch_d128(p, c->type, nt, scored, grid, (int)rows, s)
                     : launch_d64(p, c->type, nt, scored, grid, (int)rows, s);
}

}  // namespace marble
