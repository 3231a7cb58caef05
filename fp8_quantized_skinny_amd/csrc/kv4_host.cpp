// Host side of the 4-bit key/value cache, of the norm and rotation before it and
// of the log probabilities: argument checks before any HIP call.
#include <algorithm>
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

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (!need) return SKINNY_OK;
  if (!workspace) return SKINNY_EINVAL;
  if (!aligned(workspace, 16)) return SKINNY_EALIGN;
  return bytes < need ? SKINNY_ESIZE : SKINNY_OK;
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

// A window is given, and one that no table's slots outgrow is none.
int check_window(int window, int sinks) { return window >= 0 && sinks >= 0 ? SKINNY_OK : SKINNY_EINVAL; }
int used_window(int window, int width) { return window < static_cast<int64_t>(width) * SKINNY_KV_PAGE ? window : 0; }

int attend(const kv4_cache* cache, const kv4_rows* q, int type, int T, int Hq, float scale, int window, int sinks,
           void* out, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int s = check_attend(cache, q, type, T, Hq, scale);
  if (s) return s;
  s = check_window(window, sinks);
  if (s) return s;
  if (!out) return SKINNY_EINVAL;
  if (!aligned(out, 16) || !aligned(lse, 4)) return SKINNY_EALIGN;
  if (!fits_plan(cache->B, cache->width)) return SKINNY_ESHAPE;
  window = used_window(window, cache->width);
  const AttendPlan plan = kv4_attend_plan(cache->B, T, Hq, cache->Hk, cache->D, cache->width, window, sinks);
  if (!fits_grid(plan.grid) || !fits_grid(static_cast<int64_t>(cache->B) * cache->Hk * plan.QG)) return SKINNY_ESHAPE;
  s = check_workspace(workspace, workspace_bytes, plan.total);
  if (s) return s;
  return launch_status(launch_kv4_attention(*cache, *q, type, T, Hq, scale, window, sinks, out, lse, workspace, stream));
}

int check_chunk(int N, int B, int Hq, int Hk, int D, int width) {
  const int s = check_shape(B, Hk, D, width);
  if (s) return s;
  if (N < 1 || Hq < 1 || Hq % Hk != 0 || Hq / Hk > SKINNY_KV_MAX_GROUP) return SKINNY_ESHAPE;
  return static_cast<int64_t>(N) * (Hq / Hk) <= INT32_MAX ? SKINNY_OK : SKINNY_ESHAPE;
}
bool chunk_fits(const ChunkPlan& p, int Hk) { return p.tiles < (int64_t{1} << 30) && fits_grid(p.groups * Hk, 512); }

// [B][T][H][D] views of 16-bit elements, for qk_norm_rope.
struct Heads {
  const kv4_rows* r;
  int H;
};
// The elements from the first of a token's heads to the last.
int64_t token_extent(const Heads& v, int D) { return (v.H - 1) * (v.H > 1 ? v.r->head : 0) + D; }
int64_t view_extent(const Heads& v, int B, int T, int D) {
  return (B > 1 ? (B - 1) * v.r->sequence : 0) + (T > 1 ? (T - 1) * v.r->row : 0) + token_extent(v, D);
}
// Whether every head of `extent` elements has a place of its own: ordered by
// stride, each dimension steps over all of those before it.
bool apart(const Heads& v, int B, int T, int64_t extent) {
  struct Dim {
    int64_t stride;
    int count;
  } d[3] = {{v.r->sequence, B}, {v.r->row, T}, {v.r->head, v.H}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  for (const Dim& x : d) {
    if (x.count == 1) continue;
    if (x.stride < extent) return false;
    extent += x.stride * (x.count - 1);
  }
  return true;
}
bool same_heads(const Heads& a, const Heads& b, int B, int T) {
  return a.r->data == b.r->data && a.H == b.H && (B == 1 || a.r->sequence == b.r->sequence) &&
         (T == 1 || a.r->row == b.r->row) && (a.H == 1 || a.r->head == b.r->head);
}
// Whether two views share no element, as far as that shows: they lie one behind
// the other; or side by side in the step of a dimension that both take alike, so
// that each has its own part of every step; or both take the sequences' and the
// tokens' steps alike, and either the heads' too, which lie in turn, or no token
// of one comes to lie on one of the other.  (Side by side within the lesser
// step does not do for that: where the greater is no multiple of it, a token may
// lie on one of another sequence.)
bool disjoint(const Heads& a, const Heads& b, int B, int T, int D) {
  const int64_t x = reinterpret_cast<intptr_t>(a.r->data), y = reinterpret_cast<intptr_t>(b.r->data);
  if (x > y) return disjoint(b, a, B, T, D);
  if (x + 2 * view_extent(a, B, T, D) <= y) return true;
  const int64_t at = (y - x) / 2, a_token = token_extent(a, D), b_token = token_extent(b, D);
  const auto beside = [&](int64_t a_extent, int64_t b_extent, int64_t step) { return at >= a_extent && at + b_extent <= step; };
  const bool sequences = B == 1 || a.r->sequence == b.r->sequence, rows = T == 1 || a.r->row == b.r->row;
  if (B > 1 && sequences && beside(view_extent(a, 1, T, D), view_extent(b, 1, T, D), a.r->sequence)) return true;
  if (T > 1 && rows && beside(view_extent(a, B, 1, D), view_extent(b, B, 1, D), a.r->row)) return true;
  if (!sequences || !rows) return false;
  // Heads of the two in turn: those of both together have places of their own.
  const Heads& more = a.H < b.H ? b : a;
  if ((a.H == 1 || b.H == 1 || a.r->head == b.r->head) && at >= D && apart(more, B, T, at + D)) return true;
  const auto nested = [&](int64_t less, int count, int64_t greater) {
    return beside(a_token, b_token, less) && greater >= less * (count - 1) + at + b_token;
  };
  if (B > 1 && T > 1 && (nested(a.r->row, T, a.r->sequence) || nested(a.r->sequence, B, a.r->row))) return true;
  // From a token of a to one of b: at, i steps in the dimension with fewer, and n in the other.
  const bool fewer = B <= T;
  const int few = fewer ? B : T, many = fewer ? T : B;
  const int64_t few_step = fewer ? a.r->sequence : a.r->row, step = fewer ? a.r->row : a.r->sequence;
  if (many == 1) return at >= a_token;
  if (step == 0) return false;
  for (int64_t i = 1 - few; i < few; ++i) {
    const int64_t from = at + i * few_step, before = -b_token - from;
    const int64_t n = before / step - (before % step < 0) + 1;  // the least that ends behind the token of a's beginning
    const int64_t least = n < 1 - many ? 1 - many : n;
    if (least < many && from + least * step < a_token) return false;
  }
  return true;
}

// Whether an output of a chunk call lies on an input or on the other output; out
// on q itself does not: a workgroup reads the values that it or its join writes.
bool chunk_overlaps(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N, int Hq,
                    const void* out, const float* lse, const void* workspace, size_t need) {
  const size_t values = static_cast<size_t>(N) * Hq * c.D * 2;
  const Span o{out, values}, l{lse, lse ? static_cast<size_t>(N) * Hq * 4 : 0},
      x{q, 2 * static_cast<size_t>((N - 1) * row + (Hq - 1) * head + c.D)};
  const bool same = out == q && (N == 1 || row == static_cast<int64_t>(Hq) * c.D) && (Hq == 1 || head == c.D);
  const Span in[] = {{c.data, static_cast<size_t>(c.pages) * c.Hk * 72 * c.D}, {c.table, static_cast<size_t>(c.B) * c.width * 4},
                     {c.lens, static_cast<size_t>(c.B) * 4}, {starts, static_cast<size_t>(c.B + 1) * 4}, {workspace, need}};
  if ((!same && overlap(o, x)) || (lse && (overlap(l, x) || overlap(l, o)))) return true;
  for (const Span& s : in)
    if (overlap(o, s) || (lse && overlap(l, s))) return true;
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
  return kv4_attention_window_workspace_bytes(B, T, Hq, Hk, D, width, 0, 0);
}

int kv4_attention(const kv4_cache* cache, const kv4_rows* q, int type, int T, int Hq, float scale, void* out,
                  float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return attend(cache, q, type, T, Hq, scale, 0, 0, out, lse, workspace, workspace_bytes, stream);
}

size_t kv4_attention_window_workspace_bytes(int B, int T, int Hq, int Hk, int D, int width, int window, int sinks) {
  if (check_shape(B, Hk, D, width) || check_heads(T, Hq, Hk) || !fits_plan(B, width) || check_window(window, sinks)) return 0;
  return kv4_attend_plan(B, T, Hq, Hk, D, width, used_window(window, width), sinks).total;
}

int kv4_attention_window(const kv4_cache* cache, const kv4_rows* q, int type, int T, int Hq, float scale, int window,
                         int sinks, void* out, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return attend(cache, q, type, T, Hq, scale, window, sinks, out, lse, workspace, workspace_bytes, stream);
}

size_t kv4_attention_chunk_workspace_bytes(int N, int B, int Hq, int Hk, int D, int width, int window, int sinks) {
  if (check_chunk(N, B, Hq, Hk, D, width) || check_window(window, sinks)) return 0;
  const ChunkPlan p = kv4_chunk_plan(N, B, Hq, Hk, D, width, used_window(window, width), sinks);
  return chunk_fits(p, Hk) ? p.total : 0;
}

int kv4_attention_chunk(const kv4_cache* cache, const void* q, int64_t row, int64_t head, const int32_t* starts, int N,
                        int type, int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  int s = check_cache(cache, true);
  if (s) return s;
  s = check_type(type);
  if (s) return s;
  s = check_chunk(N, cache->B, Hq, cache->Hk, cache->D, cache->width);
  if (s) return s;
  const kv4_rows rows{q, 0, row, head};
  s = check_rows(&rows);
  if (s) return s;
  s = check_window(window, sinks);
  if (s) return s;
  if (!starts || !out || !std::isfinite(scale) || scale <= 0.0f) return SKINNY_EINVAL;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(starts, 4)) return SKINNY_EALIGN;
  window = used_window(window, cache->width);
  const ChunkPlan p = kv4_chunk_plan(N, cache->B, Hq, cache->Hk, cache->D, cache->width, window, sinks);
  if (!chunk_fits(p, cache->Hk)) return SKINNY_ESHAPE;
  s = check_workspace(workspace, workspace_bytes, p.total);
  if (s) return s;
  if (chunk_overlaps(*cache, q, row, head, starts, N, Hq, out, lse, workspace, p.total)) return SKINNY_EINVAL;
  return launch_status(launch_kv4_chunk(*cache, q, row, head, starts, N, type, Hq, scale, window, sinks, out, lse,
                                        workspace, stream));
}

int qk_norm_rope(const kv4_rows* q, const kv4_rows* k, const int32_t* positions, const float* inv_freq,
                 const float* q_weight, const float* k_weight, int type, int B, int T, int Hq, int Hk, int D, int rot,
                 int interleaved, float eps, float amplitude, const kv4_rows* q_out, const kv4_rows* k_out,
                 hipStream_t stream) {
  int s = check_type(type);
  if (s) return s;
  if (D != 64 && D != 128 && D != 256) return SKINNY_ESHAPE;
  if (B < 1 || T < 1 || Hq < 1 || Hk < 1 || Hq > 65536 || Hk > 65536) return SKINNY_ESHAPE;
  if (static_cast<int64_t>(B) * T > INT32_MAX || !fits_grid(rope_groups(B * T, Hq, Hk, D))) return SKINNY_ESHAPE;
  if (rot < 0 || rot > D || rot % 16 != 0) return SKINNY_ESHAPE;
  for (const kv4_rows* r : {q, k, q_out, k_out}) {
    s = check_rows(r);
    if (s) return s;
  }
  if (!positions || (rot && !inv_freq) || (interleaved != 0 && interleaved != 1)) return SKINNY_EINVAL;
  if (!std::isfinite(eps) || eps < 0.0f || !std::isfinite(amplitude)) return SKINNY_EINVAL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4)) return SKINNY_EALIGN;
  const Heads qi{q, Hq}, ki{k, Hk}, qo{q_out, Hq}, ko{k_out, Hk};
  if (!apart(qo, B, T, D) || !apart(ko, B, T, D) || !disjoint(qo, ko, B, T, D)) return SKINNY_EINVAL;
  if (!disjoint(qo, ki, B, T, D) || !disjoint(ko, qi, B, T, D)) return SKINNY_EINVAL;
  if (!same_heads(qo, qi, B, T) && !disjoint(qo, qi, B, T, D)) return SKINNY_EINVAL;
  if (!same_heads(ko, ki, B, T) && !disjoint(ko, ki, B, T, D)) return SKINNY_EINVAL;
  const Span in[] = {{positions, static_cast<size_t>(B) * T * 4}, {inv_freq, static_cast<size_t>(rot) * 2},
                     {q_weight, q_weight ? D * sizeof(float) : 0}, {k_weight, k_weight ? D * sizeof(float) : 0}};
  for (const Heads* o : {&qo, &ko})
    for (const Span& i : in)
      if (i.bytes && overlap(Span{o->r->data, static_cast<size_t>(view_extent(*o, B, T, D)) * 2}, i)) return SKINNY_EINVAL;
  const RopeArgs a{*q, *k, *q_out, *k_out, positions, inv_freq, q_weight, k_weight, B * T, T, Hq, Hk, rot, eps, amplitude};
  return launch_status(launch_norm_rope(a, type, D, interleaved, stream));
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
