// Internal declarations shared by the host code and the kernels of the 4-bit
// key/value cache, of what stands around it and of the log probabilities.  (Apart from internal.h, whose
// code the GEMMs' counter measurements are tied to.)
#ifndef SKINNY_KV4_INTERNAL_H
#define SKINNY_KV4_INTERNAL_H

#include "internal.h"
#include "skinny.h"

namespace skinny {

// The 4-bit key/value cache, the norm and rotation before it and the log
// probabilities (kv4_cache.hip, kv4_attention.hip, kv4_chunk.hip, rope.hip,
// logprobs.hip).  Arguments are validated.
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
AttendPlan kv4_attend_plan(int B, int T, int Hq, int Hk, int D, int width, int window, int sinks);  // window 0: none
hipError_t launch_kv4_attention(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale, int window,
                                int sinks, void* out, float* lse, void* workspace, hipStream_t stream);
hipError_t launch_kv4_weights(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale,
                              const float* lse, const float* acc, float* acc_out, hipStream_t stream);
// A chunk call of few rows a sequence: tiles of 16 rows per workgroup, 0 where it is
// not one, the most groups of these that there are, and shares of their pages, per
// key/value head each; a workspace where groups are split.
struct SmallChunk {
  int tiles;
  int64_t groups, shares;
  size_t count_off, segment_off, stat_off, part_off, total;
};
SmallChunk kv4_small_chunk(int N, int B, int G, int Hk, int D, int64_t pages);
hipError_t launch_kv4_small_chunk(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N,
                                  int type, int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                                  const SmallChunk& s, hipStream_t stream);
// How other chunk calls are laid out: the most tiles of rows, workgroups, tiles that are
// cut and parts of them, each per key/value head, and the workspace.
struct ChunkPlan {
  SmallChunk small;
  int64_t tiles, groups, cuts, parts;
  size_t counts_off, begin_off, offset_off, first_off, piece_off, cut_off, stat_off, part_off, total;
};
ChunkPlan kv4_chunk_plan(int N, int B, int Hq, int Hk, int D, int width, int window, int sinks);
hipError_t launch_kv4_chunk(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N,
                            int type, int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                            hipStream_t stream);
struct RopeArgs {
  kv4_rows q, k, q_out, k_out;
  const int32_t* positions;
  const float *inv_freq, *q_weight, *k_weight;
  int tokens, T, Hq, Hk, rot;
  float eps, amplitude;
};
int64_t rope_groups(int tokens, int Hq, int Hk, int D);  // workgroups of a call, at most
hipError_t launch_norm_rope(const RopeArgs& a, int type, int D, bool interleaved, hipStream_t stream);
size_t logprobs_workspace(int R, int V, int k);
hipError_t launch_logprobs(const void* logits, int type, int64_t stride, const int32_t* tokens, float* logprob,
                           float* entropy, int32_t* top_ids, float* top_logprobs, int R, int V, int k,
                           void* workspace, hipStream_t stream);

}  // namespace skinny

#endif
