// Host side of the 4-bit key/value cache and of the log probabilities:
// argument checks before any HIP call.
#include <cmath>

#include "kv4_internal.h"
#include "skinny.h"

using namespace skinny;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status(hipError_t e) { return e == hipSuccess ? SKINNY_OK : SKINNY_EHIP; }
// A grid has fewer than 2^32 threads in a dimension.
bool fits_grid(int64_t groups, int threads = 256) { return groups < (int64_t{1} << 32) / threads; }

int check_shape(int B, int Hk, int D, int width) {
  if (B < 1 || B > 65536 || Hk < 1 || Hk > 1024) return SKINNY_ESHAPE;
  if (D != 64 && D != 128 && D != 256) return SKINNY_ESHAPE;
  if (width < 1 || width >= (1 << 30) / (SKINNY_KV_PAGE / 2)) return SKINNY_ESHAPE;
  return SKINNY_OK;
}

int check_cache(const kv4_cache* c, bool lens) {
  if (!c || !c->data || !c->table || (lens && !c->lens)) return SKINNY_EINVAL;
  const int s = check_shape(c->B, c->Hk, c->D, c->width);
  if (s) return s;
  if (c->pages < 1) return SKINNY_ESHAPE;
  if (!std::isfinite(c->gk) || !std::isfinite(c->gv) || c->gk <= 0.0f || c->gv <= 0.0f) return SKINNY_EINVAL;
  if (!aligned(c->data, 16) || !aligned(c->table, 4) || !aligned(c->lens, 4)) return SKINNY_EALIGN;
  return SKINNY_OK;
}

int check_rows(const kv4_rows* r) {
  if (!r || !r->data || r->sequence < 0 || r->row < 0 || r->head < 0) return SKINNY_EINVAL;
  if (!aligned(r->data, 16) || r->sequence % 8 || r->row % 8 || r->head % 8) return SKINNY_EALIGN;
  return SKINNY_OK;
}

int check_type(int type) { return type == SKINNY_F16 || type == SKINNY_BF16 ? SKINNY_OK : SKINNY_EINVAL; }

int check_heads(int T, int Hq, int Hk) {
  if (T < 1 || T > SKINNY_MAX_M) return SKINNY_ESHAPE;
  if (Hq < 1 || Hq % Hk != 0 || Hq / Hk > SKINNY_KV_MAX_GROUP) return SKINNY_ESHAPE;
  return SKINNY_OK;
}

// The plan of an attention call counts the pages of all sequences, and shares
// of a page at least, one per sequence, in an int.
bool fits_plan(int B, int width) { return static_cast<int64_t>(B) * (width + 1) <= INT32_MAX; }

int check_attend(const kv4_cache* c, const kv4_rows* q, int type, int T, int Hq, float scale) {
  int s = check_cache(c, true);
  if (s) return s;
  s = check_type(type);
  if (s) return s;
  s = check_heads(T, Hq, c->Hk);
  if (s) return s;
  s = check_rows(q);
  if (s) return s;
  return std::isfinite(scale) && scale > 0.0f ? SKINNY_OK : SKINNY_EINVAL;
}

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Whether an output of an eviction lies on one of its inputs or on another
// output.  A workgroup writes its head's outputs while others still read the
// lengths, the weights and the pages.
bool evict_overlaps(const kv4_cache& c, const float* acc, const kv4_cache& d, const int32_t* kept,
                    const int32_t* new_lens, const float* new_acc, int keep) {
  const size_t heads = static_cast<size_t>(c.B) * c.Hk, slot = SKINNY_KV_PAGE * sizeof(float);
  const auto pages = [](const kv4_cache& k) { return Span{k.data, static_cast<size_t>(k.pages) * k.Hk * 72 * k.D}; };
  const auto table = [](const kv4_cache& k) { return Span{k.table, static_cast<size_t>(k.B) * k.width * 4}; };
  const Span in[] = {pages(c), table(c), {c.lens, static_cast<size_t>(c.B) * 4}, {acc, heads * c.width * slot}, table(d)};
  const Span out[] = {pages(d), {kept, heads * keep * 4}, {new_lens, static_cast<size_t>(c.B) * 4}, {new_acc, heads * d.width * slot}};
  for (size_t i = 0; i < 4; ++i) {
    for (const Span& s : in)
      if (overlap(out[i], s)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

}  // namespace

extern "C" {

int kv4_append(const kv4_cache* cache, const kv4_rows* k, const kv4_rows* v, int type, int T, hipStream_t stream) {
  int s = check_cache(cache, true);
  if (s) return s;
  s = check_type(type);
  if (s) return s;
  s = check_rows(k);
  if (s) return s;
  s = check_rows(v);
  if (s) return s;
  if (T < 1 || T > (1 << 30) || !fits_grid(static_cast<int64_t>(cache->B) * kv4_row_pages(T) * cache->Hk))
    return SKINNY_ESHAPE;
  return launch_status(launch_kv4_append(*cache, *k, *v, type, T, stream));
}

int kv4_read(const kv4_cache* cache, void* k, void* v, int type, int n, hipStream_t stream) {
  int s = check_cache(cache, true);
  if (s) return s;
  s = check_type(type);
  if (s) return s;
  if (!k || !v) return SKINNY_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16)) return SKINNY_EALIGN;
  if (n < 1 || n > (1 << 30) || !fits_grid(static_cast<int64_t>(cache->B) * kv4_row_pages(n) * cache->Hk))
    return SKINNY_ESHAPE;
  return launch_status(
      launch_kv4_read(*cache, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), type, n, stream));
}

size_t kv4_attention_workspace_bytes(int B, int T, int Hq, int Hk, int D, int width) {
  if (check_shape(B, Hk, D, width) || check_heads(T, Hq, Hk) || !fits_plan(B, width)) return 0;
  return kv4_attend_plan(B, T, Hq, Hk, D, width).total;
}

int kv4_attention(const kv4_cache* cache, const kv4_rows* q, int type, int T, int Hq, float scale, void* out,
                  float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int s = check_attend(cache, q, type, T, Hq, scale);
  if (s) return s;
  if (!out) return SKINNY_EINVAL;
  if (!aligned(out, 16) || !aligned(lse, 4)) return SKINNY_EALIGN;
  if (!fits_plan(cache->B, cache->width)) return SKINNY_ESHAPE;
  const AttendPlan plan = kv4_attend_plan(cache->B, T, Hq, cache->Hk, cache->D, cache->width);
  if (!fits_grid(plan.grid) || !fits_grid(static_cast<int64_t>(cache->B) * cache->Hk * plan.QG)) return SKINNY_ESHAPE;
  const size_t need = plan.total;
  if (need) {
    if (!workspace) return SKINNY_EINVAL;
    if (!aligned(workspace, 16)) return SKINNY_EALIGN;
    if (workspace_bytes < need) return SKINNY_ESIZE;
  }
  return launch_status(launch_kv4_attention(*cache, *q, type, T, Hq, scale, out, lse, workspace, stream));
}

int kv4_attention_weights(const kv4_cache* cache, const kv4_rows* q, int type, int T, int Hq, float scale,
                          const float* lse, const float* acc, float* acc_out, hipStream_t stream) {
  const int s = check_attend(cache, q, type, T, Hq, scale);
  if (s) return s;
  if (!lse || !acc || !acc_out) return SKINNY_EINVAL;
  if (!aligned(lse, 4) || !aligned(acc, 16) || !aligned(acc_out, 16)) return SKINNY_EALIGN;
  // A workgroup takes 16 pages of a head where there are many.
  if (!fits_grid(static_cast<int64_t>(cache->B) * cache->Hk * ((cache->width + 15) / 16))) return SKINNY_ESHAPE;
  return launch_status(launch_kv4_weights(*cache, *q, type, T, Hq, scale, lse, acc, acc_out, stream));
}

int kv4_evict(const kv4_cache* cache, const float* acc, const kv4_cache* dst, int32_t* kept, int32_t* new_lens,
              float* new_acc, int keep, int sinks, int recent, hipStream_t stream) {
  int s = check_cache(cache, true);
  if (s) return s;
  s = check_cache(dst, false);
  if (s) return s;
  if (!acc || !kept || !new_lens || !new_acc || dst->data == cache->data) return SKINNY_EINVAL;
  if (dst->B != cache->B || dst->Hk != cache->Hk || dst->D != cache->D) return SKINNY_ESHAPE;
  if (keep < 1 || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks) return SKINNY_EINVAL;
  if (keep > static_cast<int64_t>(dst->width) * SKINNY_KV_PAGE) return SKINNY_ESIZE;
  if (!aligned(acc, 16) || !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(new_acc, 16)) return SKINNY_EALIGN;
  if (!fits_grid(static_cast<int64_t>(cache->B) * cache->Hk, 1024)) return SKINNY_ESHAPE;
  if (!fits_grid(static_cast<int64_t>(cache->B) * kv4_row_pages(keep) * cache->Hk)) return SKINNY_ESHAPE;
  if (evict_overlaps(*cache, acc, *dst, kept, new_lens, new_acc, keep)) return SKINNY_EINVAL;
  return launch_status(
      launch_kv4_evict(*cache, acc, *dst, kept, new_lens, new_acc, keep, sinks, recent, stream));
}

size_t lm_head_logprobs_workspace_bytes(int R, int V, int k) {
  if (R < 1 || R >= (1 << 24) || V < 1 || V > (1 << 24) || k < 1 || k > SKINNY_MAX_TOP || k > V) return 0;
  return logprobs_workspace(R, V, k);
}

int lm_head_logprobs(const void* logits, int type, int64_t stride, const int32_t* tokens, float* logprob,
                     float* entropy, int32_t* top_ids, float* top_logprobs, int R, int V, int k, void* workspace,
                     size_t workspace_bytes, hipStream_t stream) {
  if (!logits || !tokens || !logprob || !entropy || !top_ids || !top_logprobs) return SKINNY_EINVAL;
  if (type != SKINNY_F16 && type != SKINNY_BF16 && type != SKINNY_F32) return SKINNY_EINVAL;
  if (R < 1 || R >= (1 << 24) || V < 1 || V > (1 << 24) || k < 1 || k > SKINNY_MAX_TOP || k > V) return SKINNY_ESHAPE;
  if (stride < V) return SKINNY_EINVAL;
  if (!aligned(logits, 16) || !aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) ||
      !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return SKINNY_EALIGN;
  const size_t need = logprobs_workspace(R, V, k);
  if (need) {
    if (!workspace) return SKINNY_EINVAL;
    if (!aligned(workspace, 16)) return SKINNY_EALIGN;
    if (workspace_bytes < need) return SKINNY_ESIZE;
  }
  return launch_status(launch_logprobs(logits, type, stride, tokens, logprob, entropy, top_ids, top_logprobs, R, V, k,
                                       workspace, stream));
}

}  // extern "C"
