// Norm of each query and key head with the rotation of its position, in one pass.
//
//   u = x w / sqrt(mean(x^2) + eps)   (u = x without weights)
//   (c, s)_i = amplitude (cos, sin)(position * inv_freq_i),  i < rot / 2
//   half layout: y_i = u_i c_i - u_{i + rot/2} s_i,  y_{i + rot/2} = u_{i + rot/2} c_i + u_i s_i
//   interleaved: the same of u_{2i} and u_{2i + 1};  y_d = u_d for d >= rot
//
// A wavefront has one token and up to P groups of heads, all queries or all
// keys: a lane holds eight positions of a head, D / 8 lanes a head, so that the
// mean is a sum over neighbouring lanes and the other half of a pair lies in
// the lane itself or rot / 16 lanes away.  The lanes find the token's angles
// together, one or two each, while the heads arrive.
//
// Few tokens are bound by latency (one token, 48 + 4 heads of 128: 2.8 us, four
// loads one behind the other between launch and store), many by memory: 32768
// tokens of these heads, 0.87 GB read and written, 187 us at the 4.68 TB/s of a
// large copy and 174 to 205 here.
#include <hip/hip_runtime.h>

#include "kv4.cuh"
#include "kv4_internal.h"

namespace skinny {
namespace {

constexpr int kWaves = 4;

// Sum over aligned groups of N lanes (8, 16 or 32), in all of them.
template <int N>
__device__ __forceinline__ float group_sum(float v) {
  const auto add = [&](int o) { v += __int_as_float(o); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xf, 0xf, false));  // quad_perm 1 0 3 2
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xf, 0xf, false));  // quad_perm 2 3 0 1
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, false));  // row_half_mirror
  if constexpr (N >= 16) add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, false));  // row_mirror
  if constexpr (N == 32) {
    const uint32_t w = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    v = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  }
  return v;
}

template <int D, class E, int P, bool INTERLEAVED>
__global__ __launch_bounds__(64 * kWaves) void norm_rope(const RopeArgs a) {
  constexpr int kLanes = D / 8, kHeads = 64 / kLanes;  // lanes of a head, heads of a group
  __shared__ __align__(16) float2 turn[kWaves][D / 2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q_parts = (a.Hq + kHeads * P - 1) / (kHeads * P), k_parts = (a.Hk + kHeads * P - 1) / (kHeads * P);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  const int token = static_cast<int>(item / (q_parts + k_parts)), part = static_cast<int>(item % (q_parts + k_parts));
  if (token >= a.tokens) return;
  const bool key = part >= q_parts;
  const int first = (key ? part - q_parts : part) * kHeads * P + lane / kLanes, H = key ? a.Hk : a.Hq;
  const kv4_rows& in = key ? a.k : a.q;
  const kv4_rows& out = key ? a.k_out : a.q_out;
  const float* weight = key ? a.k_weight : a.q_weight;
  const int b = token / a.T, t = token % a.T, piece = lane % kLanes;

  const uint16_t* src = static_cast<const uint16_t*>(in.data) + b * in.sequence + t * in.row + piece * 8;
  u32x4 x[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = first + p * kHeads;
    x[p] = h < H ? *reinterpret_cast<const u32x4*>(src + h * in.head) : u32x4{0u, 0u, 0u, 0u};
  }
  // Angles in turns and in fp64: a far position times a frequency has lost its place in the turn in fp32.  For frequencies up
  // to 1 the product is off by 2^-25.6 of a turn at most, 1 / 2 pi in 53 bits puts 2^-25.5 to it, what is left once the whole
  // turns are off is as good as exact, and its rounding to fp32 is 2^-26: 2^-24.1 together.
  constexpr double kTurn = 0x1.45f306dc9c883p-3;  // 1 / 2 pi
  const int half = a.rot / 2;
  const double position = static_cast<double>(uniform_load(a.positions, token));
  for (int i = lane; i < half; i += 64) {
    const double radians = position * static_cast<double>(a.inv_freq[i]), turns = __builtin_fma(radians, kTurn, -rint(radians * kTurn));
    float c, s;
    sincospif(static_cast<float>(2.0 * turns), &s, &c);
    turn[wave][i] = float2{a.amplitude * c, a.amplitude * s};
  }
  __builtin_amdgcn_wave_barrier();

  const bool rotates = piece * 8 < a.rot;
  const bool upper = piece * 8 >= half;  // of the half layout: the second of its pairs
  const int partner = INTERLEAVED || !rotates ? lane : (upper ? lane - a.rot / 16 : lane + a.rot / 16);
  const int other = partner % kLanes;
  constexpr int kTurns = INTERLEAVED ? 4 : 8;
  float c[kTurns], s[kTurns], w[8], wp[8];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const float2 v = rotates ? turn[wave][INTERLEAVED ? piece * 4 + i : piece * 8 - (upper ? half : 0) + i] : float2{1.0f, 0.0f};
    c[i] = v.x;
    s[i] = INTERLEAVED || upper ? v.y : -v.y;
  }
  if (weight) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = weight[piece * 8 + i];
      wp[i] = weight[other * 8 + i];
    }
  }

  uint16_t* dst = static_cast<uint16_t*>(const_cast<void*>(out.data)) + b * out.sequence + t * out.row + piece * 8;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float u[8], v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = elem_lo<E>(x[p][i]);
      u[2 * i + 1] = elem_hi<E>(x[p][i]);
    }
    if constexpr (!INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t o = __shfl(x[p][i], partner);
        v[2 * i] = elem_lo<E>(o);
        v[2 * i + 1] = elem_hi<E>(o);
      }
    }
    if (weight) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(u[i], u[i], sum);
      const float r = 1.0f / __builtin_sqrtf(group_sum<kLanes>(sum) * (1.0f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] *= r * w[i];
        if constexpr (!INTERLEAVED) v[i] *= r * wp[i];
      }
    }
    float y[8];
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = u[2 * i] * c[i] - u[2 * i + 1] * s[i];
        y[2 * i + 1] = u[2 * i + 1] * c[i] + u[2 * i] * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = u[i] * c[i] + v[i] * s[i];
    }
    const int h = first + p * kHeads;
    if (h < H) {
      u32x4 packed;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // positions that do not turn stay clear of 0 * inf
        packed[i] = rotates ? elem_pack<E>(y[2 * i], y[2 * i + 1]) : elem_pack<E>(u[2 * i], u[2 * i + 1]);
      *reinterpret_cast<u32x4*>(dst + h * out.head) = packed;
    }
  }
}

template <int D, class E, int P>
void launch(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  constexpr int kHeads = 512 / D * P;
  const int64_t waves = static_cast<int64_t>(a.tokens) * ((a.Hq + kHeads - 1) / kHeads + (a.Hk + kHeads - 1) / kHeads);
  const dim3 grid(static_cast<unsigned>((waves + kWaves - 1) / kWaves));
  if (interleaved) norm_rope<D, E, P, true><<<grid, 64 * kWaves, 0, stream>>>(a);
  else norm_rope<D, E, P, false><<<grid, 64 * kWaves, 0, stream>>>(a);
}

}  // namespace

int64_t rope_groups(int tokens, int Hq, int Hk, int D) {
  const int heads = 512 / D;
  return (static_cast<int64_t>(tokens) * ((Hq + heads - 1) / heads + (Hk + heads - 1) / heads) + kWaves - 1) / kWaves;
}

// Four groups of heads per wavefront, which find the angles and weights once, where
// the query heads fill them and there are wavefronts for the CUs even so.  One
// against four groups (us):
//   tokens                          1     64    256    512   1024   4096
//   48 + 4 heads of 128, one     2.81   3.04   4.21   5.83   8.85   28.1
//                        four    3.79   4.04   4.40   5.41   7.90   26.1
//   24 + 4 heads of 256, one     2.99   3.27   4.54   6.41   10.2   32.8
//                        four    3.99   4.37   4.74   5.79   8.60   28.2
//   8 + 1 heads of 128, one      2.58   2.94   2.98   3.16   3.70   8.12
//   (two groups)         four    3.25   3.71   3.78   3.84   4.43   9.83
hipError_t launch_norm_rope(const RopeArgs& a, int type, int D, bool interleaved, hipStream_t stream) {
  const bool fills = a.Hq * D > 3 * 512;  // four groups of query heads at least
  const auto run = [&](auto d, auto e) {
    if (!fills || rope_groups(a.tokens, a.Hq, a.Hk, D) < 1024) launch<d(), decltype(e), 1>(a, interleaved, stream);
    else launch<d(), decltype(e), 4>(a, interleaved, stream);
  };
  const auto by_type = [&](auto d) {
    if (type == SKINNY_F16) run(d, F16());
    else run(d, BF16());
  };
  if (D == 64) by_type(std::integral_constant<int, 64>());
  else if (D == 128) by_type(std::integral_constant<int, 128>());
  else by_type(std::integral_constant<int, 256>());
  return hipGetLastError();
}

}  // namespace skinny
