// Log probabilities, entropy and the greatest alternatives of an lm_head's
// logits.  With m the row's maximum, y = x - m and e = exp(y):
//   S = sum e,  log p = y - log S,  H = log S - sum(e y) / S.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "kv4.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;

struct F32 {
  using T = float;
  static __device__ __forceinline__ float at(const void* p, int i) { return static_cast<const float*>(p)[i]; }
};
template <class E>
struct Half {
  using T = uint16_t;
  static __device__ __forceinline__ float at(const void* p, int i) { return E::load(static_cast<const uint16_t*>(p)[i]); }
};

struct LogprobArgs {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int V, k;
};

// Running softmax statistics: maximum, sum of exp(x - m), sum of that times (x - m).
struct Stat {
  float m, s, t;
};
__device__ __forceinline__ void join(Stat& a, const Stat& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) {  // neither has a finite logit yet; a NaN stays
    a.s += b.s;
    a.t += b.t;
    return;
  }
  // sum e^(x - m) (x - m) from the sums about another maximum: f (t + s d), d = m_old - m.
  const auto moved = [&](const Stat& o) {
    if (o.m == -INFINITY) return Stat{m, o.s, o.t};
    const float d = o.m - m, f = __builtin_amdgcn_exp2f(d * kLog2e);
    return Stat{m, o.s * f, f * (o.t + (o.s > 0.0f && f > 0.0f ? o.s * d : 0.0f))};
  };
  const Stat x = moved(a), y = moved(b);
  a = Stat{m, x.s + y.s, x.t + y.t};
}

template <class L>
__global__ __launch_bounds__(kThreads) void logprobs(const LogprobArgs a) {
  __shared__ Stat parts[kThreads];
  __shared__ unsigned long long best[kThreads / 64];
  const int r = blockIdx.x, tid = threadIdx.x;
  const void* x = static_cast<const typename L::T*>(a.logits) + r * a.stride;
  Stat st{-INFINITY, 0.0f, 0.0f};
  for (int i = tid; i < a.V; i += kThreads) {
    const float v = L::at(x, i);
    if (v != v) st.s = v;
    else if (v > -INFINITY) join(st, Stat{v, 1.0f, 0.0f});
  }
  parts[tid] = st;
  for (int o = kThreads / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (tid < o) join(parts[tid], parts[tid + o]);
  }
  __syncthreads();
  st = parts[0];
  const bool none = st.m == -INFINITY && st.s == 0.0f;
  // Log probabilities are (x - m) - log S: m + log S would swallow log S for a great m.
  const float m = none ? 0.0f : st.m, log = none ? 0.0f : logf(st.s);
  if (tid == 0) {
    const int token = a.tokens[r];
    a.logprob[r] = token >= 0 && token < a.V ? L::at(x, token) - m - log : NAN;
    a.entropy[r] = none ? 0.0f : log - st.t / st.s;
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long key = 0ull;
    for (int i = tid; i < a.V; i += kThreads) {
      const unsigned long long q = argmax_key(L::at(x, i), i);
      if (q < last && q > key) key = q;
    }
    key = wave_max_key(key);
    if ((tid & 63) == 0) best[tid / 64] = key;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) key = best[w] > key ? best[w] : key;
    __syncthreads();
    last = key;
    if (tid == 0) {
      const int id = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(key));
      a.top_ids[static_cast<size_t>(r) * a.k + j] = id;
      a.top_logprobs[static_cast<size_t>(r) * a.k + j] = id < 0 ? NAN : L::at(x, id) - m - log;
    }
  }
}

}  // namespace

size_t logprobs_workspace(int, int, int) { return 0; }

hipError_t launch_logprobs(const void* logits, int type, int64_t stride, const int32_t* tokens, float* logprob,
                           float* entropy, int32_t* top_ids, float* top_logprobs, int R, int V, int k, void*,
                           hipStream_t stream) {
  const LogprobArgs a{logits, stride, tokens, logprob, entropy, top_ids, top_logprobs, V, k};
  if (type == SKINNY_F16) logprobs<Half<F16>><<<dim3(R), kThreads, 0, stream>>>(a);
  else if (type == SKINNY_BF16) logprobs<Half<BF16>><<<dim3(R), kThreads, 0, stream>>>(a);
  else logprobs<F32><<<dim3(R), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace skinny
