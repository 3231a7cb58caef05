// Internal declarations shared by the host code and the kernels of the 4-bit
// key/value cache and of the log probabilities.  (Apart from internal.h, whose
// code the GEMMs' counter measurements are tied to.)
#ifndef SKINNY_KV4_INTERNAL_H
#define SKINNY_KV4_INTERNAL_H

#include "internal.h"
#include "skinny.h"

namespace skinny {

// The 4-bit key/value cache and the log probabilities (kv4_cache.hip,
// kv4_attention.hip, logprobs.hip).  Arguments are validated.
// Pages that `rows` newest slots can reach.
int kv4_row_pages(int rows);
hipError_t launch_kv4_append(const kv4_cache& c, const kv4_rows& k, const kv4_rows& v, int type, int T,
                             hipStream_t stream);
hipError_t launch_kv4_read(const kv4_cache& c, uint16_t* k, uint16_t* v, int type, int n, hipStream_t stream);
hipError_t launch_kv4_evict(const kv4_cache& c, const float* acc, const kv4_cache& dst, int32_t* kept,
                            int32_t* new_lens, float* new_acc, int keep, int sinks, int recent, hipStream_t stream);
// How an attention call is laid out: query tiles of 16 rows per workgroup and
// groups of them per head, fewest pages of a workgroup, whether segments may be
// split, the grid, and the workspace.
struct AttendPlan {
  int MT, QG, least;
  bool split;
  int64_t grid;
  size_t split_off, stat_off, part_off, total;
};
AttendPlan kv4_attend_plan(int B, int T, int Hq, int Hk, int D, int width);
hipError_t launch_kv4_attention(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale, void* out,
                                float* lse, void* workspace, hipStream_t stream);
hipError_t launch_kv4_weights(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale,
                              const float* lse, const float* acc, float* acc_out, hipStream_t stream);
size_t logprobs_workspace(int R, int V, int k);
hipError_t launch_logprobs(const void* logits, int type, int64_t stride, const int32_t* tokens, float* logprob,
                           float* entropy, int32_t* top_ids, float* top_logprobs, int R, int V, int k,
                           void* workspace, hipStream_t stream);

}  // namespace skinny

#endif
