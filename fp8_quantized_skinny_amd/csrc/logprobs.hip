// Log probabilities, entropy and the greatest alternatives of an lm_head's
// logits, in one pass over them.  With m the row's maximum, y = x - m and
// e = exp(y):
//   S = sum e,  log p = y - log S,  H = log S - sum(e y) / S.
//
// Every lane keeps the statistics of the elements it met about its own running
// maximum.  The alternatives: a logit and its index form one 64-bit key that
// orders as wanted (argmax_key), all keys of a row differ, and keys at or
// below a threshold under which k greater ones are known need no further look.
// A wavefront collects the keys above the threshold in a list of its own in
// LDS, cuts the list back to its k greatest when it has grown long, and raises
// the threshold, which the workgroup's wavefronts share, to the least of
// those.  After the first elements few get past it: the pass costs one
// comparison of a lane's maximum per 16 elements.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "kv4.cuh"

namespace skinny {
namespace {

typedef unsigned long long Key;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kVectors = 2;                      // 16-byte loads of a lane per step
constexpr int kMost = kVectors * 8;              // elements of a lane per step
constexpr int kKeep = 128;                       // keys at which a list is cut back
constexpr int kList = SKINNY_MAX_TOP * kMost + kKeep;  // see collect()

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

__device__ __forceinline__ uint32_t key_high(float v) { return static_cast<uint32_t>(argmax_key(v, 0) >> 32); }

// The k-th greatest of the wavefront's keys (N per lane), by bits from the
// top; 0 if there are fewer than k keys other than 0.
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
      if (n == k) {  // the least of exactly k keys
        Key least = ~0ull;
#pragma unroll
        for (int i = 0; i < N; ++i) least = key[i] >= next && key[i] < least ? key[i] : least;
        return ~wave_max_key(~least);
      }
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
  Key* shared;  // LDS: the greatest `over` of the workgroup's wavefronts

  __device__ __forceinline__ void raise(Key to) {
    if (to > over) {
      over = to;
      if ((threadIdx.x & 63) == 0) atomicMax(shared, to);
    }
  }
  __device__ __forceinline__ void push(bool want, Key key) {
    const unsigned long long mask = __ballot(want);
    if (want) keys[n + lanes_below(mask)] = key;
    n += __popcll(mask);
  }
  // Cuts the list back to its k greatest keys (fewer if it has no more).
  __device__ void cut() {
    if (n <= k) return;
    constexpr int kPer = (kList + 63) / 64;
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_wave_barrier();
    if (n <= 192) cut_held<3>(lane);
    else cut_held<kPer>(lane);
  }
  template <int N>
  __device__ __forceinline__ void cut_held(int lane) {
    Key held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) held[i] = i * 64 + lane < n ? keys[i * 64 + lane] : 0ull;
    const Key least = kth_key<N>(held, k);
    n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) push(held[i] >= least && held[i] > 0ull, held[i]);
    raise(least);
  }
};

// One step of a wavefront: N elements per lane, element i of a lane at column
// at(i), real where real(i).  `top` is the greatest of a lane's elements.
template <int N, class At, class Real>
__device__ __forceinline__ void collect(List& list, const float (&x)[N], float top, At at, Real real) {
  const Key shared = *static_cast<volatile Key*>(list.shared);
  if (shared > list.over) list.over = shared;
  const unsigned long long lanes = __ballot(key_high(top) >= static_cast<uint32_t>(list.over >> 32));
  if (lanes == 0ull) return;
  if (list.n + __popcll(lanes) * N > kList) {
    // Room for every lane's elements is not sure: let the lanes' greatest keys
    // decide.  k of them reach the k-th greatest, so nothing below it is
    // wanted, and only the k lanes that reach it hold anything above it: at
    // most k N keys, which the list has room for after a cut.
    list.cut();
    Key best[1] = {0ull};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Key key = real(i) ? argmax_key(x[i], at(i)) : 0ull;
      best[0] = key > best[0] ? key : best[0];
    }
    const Key kth = kth_key<1>(best, list.k);
    if (kth > 0ull) list.raise(kth - 1ull);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const Key key = argmax_key(x[i], at(i));
    const bool want = real(i) && key > list.over;
    if (__any(want)) list.push(want, key);
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

__device__ __forceinline__ Stat wave_join(Stat st) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) st = join(st, Stat{__shfl_xor(st.m, o), __shfl_xor(st.s, o), __shfl_xor(st.t, o)});
  return st;
}

// Results of row r from its statistics and its n candidate keys in LDS (k
// greatest among them, zeros allowed).
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
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Key key = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > key || (keys[j] == key && j < i);
    if (rank < a.k) {
      const int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));  // -1 for no key
      const size_t at = static_cast<size_t>(r) * a.k + rank;
      a.top_ids[at] = id;
      a.top_logprobs[at] = id < 0 ? NAN : L::at(x + id) - m - log;
    }
  }
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
  __shared__ Key final_keys[kWaves * SKINNY_MAX_TOP];
  __shared__ Key shared;
  __shared__ Stat parts[kWaves];
  __shared__ int last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  if (threadIdx.x == 0) shared = 0ull;
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
  List list{lists[wave], 0, a.k, 0ull, &shared};
  Stat st{-INFINITY, 0.0f, 0.0f};

  u32x4 next[kVectors];
  const auto fetch = [&](int v) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int i = v + u * 64 + lane;
      next[u] = i < v1 ? load16(vec + i) : u32x4{L::kNone, L::kNone, L::kNone, L::kNone};
    }
  };
  fetch(v0);
  for (int v = v0; v < v1; v += 64 * kVectors) {
    float e[N];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) L::widen(next[u], e + u * kPer);
    fetch(v + 64 * kVectors);
    float top = e[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, e[i]);
    add(st, e, top);
    collect(list, e, top, [&](int i) { return head + (v + i / kPer * 64 + lane) * kPer + i % kPer; },
            [&](int i) { return v + i / kPer * 64 + lane < v1; });
  }
  if (range == 0 && head + tail > 0) {
    const int col = lane < head ? lane : a.V - tail + (lane - head);
    const bool real = lane < head + tail;
    const float e[1] = {real ? L::at(x + col) : -INFINITY};
    add(st, e, e[0]);
    collect(list, e, e[0], [&](int) { return col; }, [&](int) { return real; });
  }
  list.cut();
  st = wave_join(st);
  if (lane == 0) parts[wave] = st;
  __builtin_amdgcn_wave_barrier();
  if (lane < a.k) final_keys[wave * a.k + lane] = lane < list.n ? list.keys[lane] : 0ull;
  __syncthreads();
  st = join(join(parts[0], parts[1]), join(parts[2], parts[3]));
  if (a.splits == 1) {
    finish<L>(a, r, x, st, final_keys, kWaves * a.k);
    return;
  }

  // The row's workgroups leave their k greatest keys and statistics (past the
  // XCD's own L2, which the others do not see), and the last to arrive
  // finishes the row.  Nothing waits on another workgroup, and neither the
  // keys' order nor that of the sums depends on the arrivals.
  Key* keys = a.keys + static_cast<size_t>(r) * a.splits * a.k;
  Key* stats = a.stats + static_cast<size_t>(r) * a.splits * 2;
  if (wave == 0) {
    Key held[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) held[i] = i * 64 + lane < kWaves * a.k ? final_keys[i * 64 + lane] : 0ull;
    const Key least = kth_key<2>(held, a.k);
    list.n = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) list.push(held[i] >= least && held[i] > 0ull, held[i]);
    __builtin_amdgcn_wave_barrier();
    if (lane < a.k) put(keys + split * a.k + lane, lane < list.n ? list.keys[lane] : 0ull);
    if (lane == 0) {
      put(stats + split * 2, two(st.m, st.s));
      put(stats + split * 2 + 1, two(st.t, 0.0f));
    }
    __builtin_amdgcn_s_waitcnt(0);
    if (lane == 0) {
      unsigned* count = a.sync + static_cast<size_t>(r) * (kSyncLineBytes / 4);
      const unsigned old = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = old == static_cast<unsigned>(a.splits - 1);
      if (last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
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
  list.cut();
  __builtin_amdgcn_wave_barrier();
  if (lane < a.k) final_keys[wave * a.k + lane] = lane < list.n ? list.keys[lane] : 0ull;
  st = Stat{-INFINITY, 0.0f, 0.0f};
  for (int i = lane; i < a.splits; i += 64) {
    const Key ms = get(stats + i * 2), t = get(stats + i * 2 + 1);
    st = join(st, Stat{low(ms), high(ms), low(t)});
  }
  st = wave_join(st);
  __syncthreads();
  finish<L>(a, r, x, st, final_keys, kWaves * a.k);
}

// Workgroups per row: enough of them to fill the chip, each with one step of
// its wavefronts at least.
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
