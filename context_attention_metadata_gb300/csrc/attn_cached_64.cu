// The attention over the paged cache for heads of 64 (attn_cached.cuh).
#include "attn_cached.cuh"

namespace marble {

marble_status_t launch_d64(cached::AttnParams& p, int type, int nt, bool scored, int grid,
                           int join_rows, cudaStream_t s) {
  return cached::launch_d<64>(p, type, nt, scored, grid, join_rows, s);
}

}  // namespace marble
