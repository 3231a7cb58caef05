// Log probabilities, entropy and the greatest alternatives of an lm_head's
// logits, in one pass over them.  With m the row's maximum, y = x - m and
// e = exp(y):
//   S = sum e,  log p = y - log S,  H = log S - sum(e y) / S.
//
// Every lane keeps the statistics of the elements it met about its own running
// maximum.  The alternatives: a logit and its index form one 64-bit key that
// orders as wanted (argmax_key), and all keys of a row differ.  The elements of
// a 16-byte load are a group with the key of its greatest logit and its first
// index.  The k greatest elements lie in the k greatest groups, so a wavefront
// collects group keys only: those above a threshold that k groups are known to
// reach go to a list of its own in LDS, which is cut back when it has grown
// long, and the threshold, which the workgroup's wavefronts share, rises.  The
// pass pays one comparison per load for it (and a few operations where a lane
// has something to add); the groups that are left at the end are read again.
//
// Bound by the VALU where there are many rows (12 operations an element, seven
// of them for the sums): 2048 rows of 151936 bf16 logits, 20 alternatives, take
// 115 to 120 us pass after pass, 5.2 to 5.4 TB/s, and 121 from cold caches.
// Collecting every element above the threshold took 240 us; 131 with loads behind
// a branch, each waited for at once.  Eight such rows of fp16 take 11 us, which is
// latency: a load, two cuts, and the meeting of 38 workgroups per row.
#include <hip/hip_runtime.h>

#include "kv4.cuh"
#include "kv4_internal.h"

namespace skinny {
namespace {

typedef unsigned long long Key;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kVectors = 2;                      // 16-byte loads of a lane per step
constexpr int kMost = kVectors * 8;              // elements of a lane per step
constexpr int kSpare = 8;                        // most keys that a cut leaves besides k
constexpr int kKeep = 64;                        // keys at which a list is cut back
constexpr int kList = kKeep + 64 * kVectors;     // a step adds kVectors keys per lane at most
static_assert(SKINNY_MAX_TOP + kSpare < kKeep, "a cut makes room");

struct F32 {
  using T = float;
  static constexpr int kPer = 4;  // elements of a 16-byte load
  static __device__ __forceinline__ float at(const T* p) { return *p; }
  static __device__ __forceinline__ void widen(u32x4 w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
  }
  static constexpr uint32_t kNone = 0xFF800000u;  // -inf
};
template <class E, uint32_t NONE>
struct Half {
  using T = uint16_t;
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float at(const T* p) { return E::load(*p); }
  static __device__ __forceinline__ void widen(u32x4 w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = elem_lo<E>(w[i]);
      x[2 * i + 1] = elem_hi<E>(w[i]);
    }
  }
  static constexpr uint32_t kNone = NONE;
};
using HalfF16 = Half<F16, 0xFC00FC00u>;
using HalfBF16 = Half<BF16, 0xFF80FF80u>;

struct LogprobArgs {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int V, k, splits;
  unsigned* sync;  // arrival counter of each row, zero at rest
  Key* keys;       // [row][split][k]
  Key* stats;      // [row][split][2]: (m, s) and (t, 0)
};

// Running statistics: maximum, sum of exp(x - m), sum of that times (x - m).
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ Stat moved(const Stat& o, float m) {
  // About another maximum m >= o.m: sum f e (y + d), d = o.m - m, f = exp(d).
  if (o.m == -INFINITY || o.m == m) return Stat{m, o.s, o.t};  // nothing yet (a NaN stays), or no move
  const float d = o.m - m, f = __builtin_amdgcn_exp2f(d * kLog2e);
  return Stat{m, o.s * f, f > 0.0f || f != f ? f * (o.t + o.s * d) : o.s * f};
}
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  const Stat x = moved(a, m), y = moved(b, m);
  return Stat{m, x.s + y.s, x.t + y.t};
}

// The logit of a key (-0 became 0).
__device__ __forceinline__ float key_value(Key key) {
  const uint32_t ord = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((ord & 0x80000000u) ? ord ^ 0x80000000u : ~ord);
}
__device__ __forceinline__ int key_index(Key key) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key)); }

// A value that k .. k + kSpare of the wavefront's keys (N per lane, all
// different or 0) reach, by bits from the top; 0 if fewer than k are not 0.
template <int N>
__device__ __forceinline__ Key kth_key(const Key (&key)[N], int k) {
  Key at = 0ull;
  for (int bit = 63; bit >= 0; --bit) {
    const Key next = at | (1ull << bit);
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(key[i] >= next));
    if (n >= k) {
      at = next;
      if (n <= k + kSpare) break;
    }
  }
  return at;
}

// A wavefront's list of keys.
struct List {
  Key* keys;    // LDS, kList of them
  int n;
  int k;
  Key over;     // keys at or below it are not wanted
  float floor;  // logits below it are not
  Key* shared;  // LDS: the greatest `over` of the workgroup's wavefronts

  __device__ __forceinline__ void raise(Key to) {
    if (to > over) {
      over = to;
      floor = key_value(to);
    }
  }
  __device__ __forceinline__ void push(bool want, Key key) {
    const unsigned long long mask = __ballot(want);
    if (want) keys[n + lanes_below(mask)] = key;
    n += __popcll(mask);
  }
  // Cuts the list back to at most k + kSpare keys, the k greatest among them.
  __device__ __forceinline__ void cut() {
    if (n <= 128) cut_held<2>();
    else cut_held<kList / 64>();
  }
  template <int N>
  __device__ __forceinline__ void cut_held() {
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    Key held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) held[i] = i * 64 + lane < n ? keys[i * 64 + lane] : 0ull;
    const Key least = kth_key<N>(held, k);
    n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) push(held[i] >= least && held[i] > 0ull, held[i]);
    if (least - 1ull > over && least > 0ull) {
      raise(least - 1ull);
      if (lane == 0) atomicMax(shared, over);
    }
  }
};

// The groups of one step of a wavefront: U per lane, with their greatest logits
// and first columns; `top` is the greatest of a lane's logits.
template <int U, class At, class Real>
__device__ __forceinline__ void collect(List& list, const float (&most)[U], float top, At at, Real real) {
  if (!__any(top >= list.floor)) return;
  list.raise(__hip_atomic_load(list.shared, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!__any(most[u] >= list.floor)) continue;
    const Key key = argmax_key(most[u], at(u));  // 0 if all are NaN
    list.push(real(u) && key > list.over, key);
  }
  if (list.n > kKeep) list.cut();
}

template <int N>
__device__ __forceinline__ void add(Stat& st, const float (&x)[N], float top) {
  if (top > st.m) st = moved(st, top);
  const float m = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = x[i] - m, e = __builtin_amdgcn_exp2f(y * kLog2e);
    st.s += e;
    st.t += e * fmaxf(y, -1e4f);  // exp(-inf) is 0, and so is its product
  }
}

// Sums and the greatest over the lanes of a wavefront, in lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<0x111, 0xf>(0.0f, v);
  v += dpp<0x112, 0xf>(0.0f, v);
  v += dpp<0x114, 0xf>(0.0f, v);
  v += dpp<0x118, 0xf>(0.0f, v);
  v += dpp<0x142, 0xa>(0.0f, v);
  v += dpp<0x143, 0xc>(0.0f, v);
  return v;
}
__device__ __forceinline__ float lanes_greatest(float v) {
  v = fmaxf(v, dpp<0x111, 0xf>(v, v));
  v = fmaxf(v, dpp<0x112, 0xf>(v, v));
  v = fmaxf(v, dpp<0x114, 0xf>(v, v));
  v = fmaxf(v, dpp<0x118, 0xf>(v, v));
  v = fmaxf(v, dpp<0x142, 0xa>(v, v));
  v = fmaxf(v, dpp<0x143, 0xc>(v, v));
  return v;
}
__device__ __forceinline__ float lane_63(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ Stat wave_join(Stat st) {
  const float m = lane_63(lanes_greatest(st.m));
  st = moved(st, m);
  return Stat{m, lane_63(lanes_sum(st.s)), lane_63(lanes_sum(st.t))};
}

// The workgroup's lists in one: at most k + kSpare keys, the k greatest of all
// among them, in `out`; returns their number.  A barrier comes first and last.
__device__ __forceinline__ int merge_lists(const Key (*lists)[kList], const int* counts, int k, Key* out, int* number) {
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    constexpr int kPer = kKeep / 64, N = kWaves * kPer;
    Key held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = i % kPer * 64 + lane;
      held[i] = j < counts[i / kPer] ? lists[i / kPer][j] : 0ull;
    }
    const Key least = kth_key<N>(held, k);
    List all{out, 0, k, 0ull, 0.0f, nullptr};
#pragma unroll
    for (int i = 0; i < N; ++i) all.push(held[i] >= least && held[i] > 0ull, held[i]);
    if (lane == 0) *number = all.n;
  }
  __syncthreads();
  return *number;
}

// rank(i) < k of the n different keys in LDS goes to put(rank, key), and so do
// the places for which there is no key, as 0.
template <class Put>
__device__ __forceinline__ void ranked(const Key* keys, int n, int k, Put put) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key key = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > key;
    if (rank < k) put(rank, key);
  }
  for (int i = n + threadIdx.x; i < k; i += kThreads) put(i, 0ull);
}

// Results of row r from its statistics and its n candidate keys in LDS.
template <class L>
__device__ __forceinline__ void finish(const LogprobArgs& a, int r, const typename L::T* x, const Stat& st,
                                       const Key* keys, int n) {
  const bool none = st.m == -INFINITY && st.s == 0.0f;
  // Log probabilities are (x - m) - log S: m + log S would swallow log S for a great m.
  const float m = none ? 0.0f : st.m, log = none ? 0.0f : logf(st.s);
  if (threadIdx.x == 0) {
    const int token = a.tokens[r];
    a.logprob[r] = token >= 0 && token < a.V ? L::at(x + token) - m - log : NAN;
    a.entropy[r] = none ? 0.0f : log - st.t / st.s;
  }
  ranked(keys, n, a.k, [&](int rank, Key key) {
    const size_t at = static_cast<size_t>(r) * a.k + rank;
    a.top_ids[at] = key ? key_index(key) : -1;
    a.top_logprobs[at] = key ? key_value(key) - m - log : NAN;
  });
}

__device__ __forceinline__ void put(Key* p, Key v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ Key get(const Key* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ Key two(float a, float b) {
  return static_cast<Key>(__float_as_uint(a)) | (static_cast<Key>(__float_as_uint(b)) << 32);
}
__device__ __forceinline__ float low(Key k) { return __uint_as_float(static_cast<uint32_t>(k)); }
__device__ __forceinline__ float high(Key k) { return __uint_as_float(static_cast<uint32_t>(k >> 32)); }

template <class L>
__global__ __launch_bounds__(kThreads) void logprobs(const LogprobArgs a) {
  using T = typename L::T;
  constexpr int kPer = L::kPer, N = kVectors * kPer;
  __shared__ Key lists[kWaves][kList];
  __shared__ Key groups[kKeep];
  __shared__ Key candidates[kKeep * kPer];
  __shared__ Key shared;
  __shared__ Stat parts[kWaves];
  __shared__ int counts[kWaves];
  __shared__ int number, found;
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  if (threadIdx.x == 0) {
    shared = 0ull;
    found = 0;
  }
  __syncthreads();

  // The row's whole 16-byte vectors are split evenly; the elements before and
  // after them go to the first wavefront, one per lane.
  const int before = static_cast<int>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T));
  const int head = before < a.V ? before : a.V;
  const int vectors = (a.V - head) / kPer, tail = a.V - head - vectors * kPer;
  const int ranges = a.splits * kWaves, range = split * kWaves + wave;
  const int per = (vectors + ranges - 1) / ranges;
  const int v0 = range * per < vectors ? range * per : vectors, v1 = v0 + per < vectors ? v0 + per : vectors;
  const u32x4* vec = reinterpret_cast<const u32x4*>(x + head);
  List list{lists[wave], 0, a.k, 0ull, -INFINITY, &shared};
  Stat st{-INFINITY, 0.0f, 0.0f};

  // Two steps' loads alternate, so that one is in flight while the other is
  // used; both are unconditional (past the range's end the last vector again),
  // since a branch around a load makes the compiler wait for it at once.
  constexpr int kStep = 64 * kVectors;
  const auto fetch = [&](int v, u32x4 (&to)[kVectors]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int i = v + u * 64 + lane;
      to[u] = load16(vec + (i < v1 ? i : v1 - 1));
    }
  };
  const auto use = [&](int v, u32x4 (&from)[kVectors]) __attribute__((always_inline)) {
    if (v + kStep > v1) {
#pragma unroll
      for (int u = 0; u < kVectors; ++u)
        if (v + u * 64 + lane >= v1) from[u] = u32x4{L::kNone, L::kNone, L::kNone, L::kNone};
    }
    float e[N], most[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      L::widen(from[u], e + u * kPer);
      most[u] = e[u * kPer];
#pragma unroll
      for (int i = 1; i < kPer; ++i) most[u] = fmaxf(most[u], e[u * kPer + i]);
    }
    const float top = fmaxf(most[0], most[1]);
    add(st, e, top);
    collect(list, most, top, [&](int u) { return head + (v + u * 64 + lane) * kPer; },
            [&](int u) { return v + u * 64 + lane < v1; });
  };
  if (v0 < v1) {
    u32x4 one[kVectors], two[kVectors];
    fetch(v0, one);
    for (int v = v0; v < v1; v += 2 * kStep) {
      fetch(v + kStep, two);
      use(v, one);
      if (v + kStep >= v1) break;
      fetch(v + 2 * kStep, one);
      use(v + kStep, two);
    }
  }
  if (range == 0 && head + tail > 0) {  // groups of one element
    const int col = lane < head ? lane : a.V - tail + (lane - head);
    const bool real = lane < head + tail;
    const float e[1] = {real ? L::at(x + col) : -INFINITY};
    add(st, e, e[0]);
    collect(list, e, e[0], [&](int) { return col; }, [&](int) { return real; });
  }
  st = wave_join(st);
  if (lane == 0) {
    parts[wave] = st;
    counts[wave] = list.n;
  }
  // Their elements that reach the least of k groups; all, if there are fewer.
  const int ng = merge_lists(lists, counts, a.k, groups, &number);
  st = join(join(parts[0], parts[1]), join(parts[2], parts[3]));
  float floor = lane < ng ? key_value(groups[lane]) : INFINITY;
  floor = ng < a.k ? -INFINITY : -lane_63(lanes_greatest(-floor));
  for (int i0 = 0; i0 < ng * kPer; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int col = i < ng * kPer ? key_index(groups[i / kPer]) + i % kPer : 0;
    const bool whole = col - i % kPer >= head && col - i % kPer < a.V - tail;
    const bool real = i < ng * kPer && (whole || i % kPer == 0);
    const float e = real ? L::at(x + col) : NAN;
    const bool want = e >= floor;
    const unsigned long long mask = __ballot(want);
    int at = 0;
    if (lane == 0 && mask) at = atomicAdd(&found, __popcll(mask));
    at = __builtin_amdgcn_readfirstlane(at) + lanes_below(mask);
    if (want) candidates[at] = argmax_key(e, col);
  }
  __syncthreads();
  if (a.splits == 1) {
    finish<L>(a, r, x, st, candidates, found);
    return;
  }

  // The row's workgroups leave their k greatest keys and statistics (past the
  // XCD's own L2, which the others do not see), and the last to arrive
  // finishes the row.  Nothing waits on another workgroup, and neither the
  // keys' order nor that of the sums depends on the arrivals.
  Key* keys = a.keys + static_cast<size_t>(r) * a.splits * a.k;
  Key* stats = a.stats + static_cast<size_t>(r) * a.splits * 2;
  ranked(candidates, found, a.k, [&](int rank, Key key) { put(keys + split * a.k + rank, key); });
  if (threadIdx.x == 0) {
    put(stats + split * 2, two(st.m, st.s));
    put(stats + split * 2 + 1, two(st.t, 0.0f));
  }
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* count = a.sync + static_cast<size_t>(r) * (kSyncLineBytes / 4);
    const unsigned old = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = old == static_cast<unsigned>(a.splits - 1);
    if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  list.n = 0;
  list.over = 0ull;
  const int n = a.splits * a.k;
  for (int i = wave * 64; i < n; i += kThreads) {
    const Key key = i + lane < n ? get(keys + i + lane) : 0ull;
    list.push(key > list.over, key);
    if (list.n > kKeep) list.cut();
  }
  if (lane == 0) counts[wave] = list.n;
  st = Stat{-INFINITY, 0.0f, 0.0f};
  for (int i = lane; i < a.splits; i += 64) {
    const Key ms = get(stats + i * 2), t = get(stats + i * 2 + 1);
    st = join(st, Stat{low(ms), high(ms), low(t)});
  }
  st = wave_join(st);
  finish<L>(a, r, x, st, groups, merge_lists(lists, counts, a.k, groups, &number));
}

// Workgroups per row: 2048 of all rows, eight per CU, each with one step of its
// wavefronts at least.  Up to 32 rows of 151936 logits the step decides; beyond,
// each workgroup's fixed part (its cuts, its meeting with the others) shows: 128
// rows, 20 alternatives, fp16 / fp32: 24 / 29 us, with 1024 workgroups 21 / 25, 512
// 22 / 26, 256 25 / 34, 4096 37 / 37; 512 rows 44 / 60, 42 / 58, 42 / 58, 42 / 58 and 53 / 67.
int row_splits(int R, int V) {
  constexpr int kStep = kThreads * kMost;
  const int want = 2048 / R, most = (V + kStep - 1) / kStep;
  const int s = want < most ? want : most;
  return s < 1 || R > kMaxSyncGroups ? 1 : s;
}

}  // namespace

size_t logprobs_workspace(int R, int V, int k) {
  const int s = row_splits(R, V);
  return s == 1 ? 0 : kSyncBytes + static_cast<size_t>(R) * s * (k + 2) * sizeof(Key);
}

hipError_t launch_logprobs(const void* logits, int type, int64_t stride, const int32_t* tokens, float* logprob,
                           float* entropy, int32_t* top_ids, float* top_logprobs, int R, int V, int k,
                           void* workspace, hipStream_t stream) {
  const int s = row_splits(R, V);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  LogprobArgs a{logits, stride, tokens, logprob, entropy, top_ids, top_logprobs, V, k, s, nullptr, nullptr, nullptr};
  if (s > 1) {
    a.sync = reinterpret_cast<unsigned*>(ws);
    a.keys = reinterpret_cast<Key*>(ws + kSyncBytes);
    a.stats = a.keys + static_cast<size_t>(R) * s * k;
  }
  const dim3 grid(static_cast<unsigned>(R) * s);
  if (type == SKINNY_F16) logprobs<HalfF16><<<grid, kThreads, 0, stream>>>(a);
  else if (type == SKINNY_BF16) logprobs<HalfBF16><<<grid, kThreads, 0, stream>>>(a);
  else logprobs<F32><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace skinny
