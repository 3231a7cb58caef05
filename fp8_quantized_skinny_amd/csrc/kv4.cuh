// Device helpers of the 4-bit key/value cache: the places of a token's bytes
// in a page's block (the layout is in skinny.h), element types, page lookup.
#ifndef SKINNY_KV4_CUH
#define SKINNY_KV4_CUH

#include <hip/hip_bf16.h>

#include "common.cuh"
#include "skinny.h"

namespace skinny {

constexpr int kPage = SKINNY_KV_PAGE;

// Offsets of a block's four parts for head size D.
template <int D>
struct KvBlock {
  static constexpr int kKScales = 32 * D;
  static constexpr int kVCodes = 36 * D;
  static constexpr int kVScales = 68 * D;
  static constexpr int kBytes = 72 * D;
  static constexpr int kGroups = D / 16;  // scales per token, also positions per V column block

  // Scale byte of token t's group f (16 positions).
  __host__ __device__ static int k_scale(int t, int f) {
    return kKScales + ((f / (D / 64)) * 16 + t % 16) * (D / 16) + (t / 16) * (D / 64) + f % (D / 64);
  }
  __host__ __device__ static int v_scale(int t, int f) {
    return kVScales + f * 64 + (t % 16 / 4) * 16 + (t / 16) * 4 + t % 4;
  }
  // The eight code bytes of token t's group f of K lie together.
  __host__ __device__ static int k_codes(int t, int f) {
    const int run = (t / 16) * (D / 8) + (f % (D / 64)) * 8;
    return (run / 16) * 1024 + (f / (D / 64)) * 256 + (t % 16) * 16 + run % 16;
  }
  // Of V, 256 / D column blocks of D / 32 bytes each, 16 bytes apart; this is the first.
  __host__ __device__ static int v_codes(int t, int f) {
    const int run = ((t / 16) * 4 + t % 4) * (D / 32);
    return kVCodes + (run / 16) * 1024 + (t % 16 / 4) * 256 + f * (256 / D) * 16 + run % 16;
  }
};

// The eight code bytes of token t's group f, to a block in global memory or LDS.
template <int D>
__device__ __forceinline__ void kv_codes_store(uint8_t* block, int t, int f, bool v, u32x2 c) {
  if (!v) {
    *reinterpret_cast<u32x2*>(block + KvBlock<D>::k_codes(t, f)) = c;
    return;
  }
  uint8_t* p = block + KvBlock<D>::v_codes(t, f);
  if constexpr (D == 256) {
    *reinterpret_cast<u32x2*>(p) = c;
  } else if constexpr (D == 128) {
    *reinterpret_cast<uint32_t*>(p) = c.x;
    *reinterpret_cast<uint32_t*>(p + 16) = c.y;
  } else {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(c.x);
    *reinterpret_cast<uint16_t*>(p + 16) = static_cast<uint16_t>(c.x >> 16);
    *reinterpret_cast<uint16_t*>(p + 32) = static_cast<uint16_t>(c.y);
    *reinterpret_cast<uint16_t*>(p + 48) = static_cast<uint16_t>(c.y >> 16);
  }
}

// Half of a group's, from a block: positions 8 piece .. 8 piece + 7.
template <int D>
__device__ __forceinline__ uint32_t kv_codes_load_half(const uint8_t* block, int t, int piece, bool v) {
  const int f = piece / 2, half = piece % 2;
  if (!v) return *reinterpret_cast<const uint32_t*>(block + KvBlock<D>::k_codes(t, f) + 4 * half);
  const uint8_t* p = block + KvBlock<D>::v_codes(t, f);
  if constexpr (D == 256) {
    return *reinterpret_cast<const uint32_t*>(p + 4 * half);
  } else if constexpr (D == 128) {
    return *reinterpret_cast<const uint32_t*>(p + 16 * half);
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p + 32 * half);
    return static_cast<uint32_t>(q[0]) | (static_cast<uint32_t>(q[8]) << 16);
  }
}

template <int D>
__device__ __forceinline__ int kv_scale_at(int t, int f, bool v) {
  return v ? KvBlock<D>::v_scale(t, f) : KvBlock<D>::k_scale(t, f);
}

// p[i] for an i that is one for the whole wavefront, through the scalar cache:
// no register of the lanes, and no wait for the vector loads in flight.  For
// what nothing writes while the kernel runs (tables and lengths).
__device__ __forceinline__ int uniform_load(const int32_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* Constant;
  return reinterpret_cast<Constant>(reinterpret_cast<uintptr_t>(p))[i];
}

// The slots of sequence b, within what its table holds.
__device__ __forceinline__ int kv_len(const kv4_cache& c, int b) {
  const int n = c.lens[b];
  return n < 0 ? 0 : (n > c.width * kPage ? c.width * kPage : n);
}

__device__ __forceinline__ int kv_len_uniform(const kv4_cache& c, int b) {
  const int n = uniform_load(c.lens, b);
  return n < 0 ? 0 : (n > c.width * kPage ? c.width * kPage : n);
}

// The block of (page id, head), or null where the id names no page.
template <int D>
__device__ __forceinline__ uint8_t* kv_block(const kv4_cache& c, int id, int head) {
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(c.pages)) return nullptr;
  return static_cast<uint8_t*>(c.data) + (static_cast<size_t>(id) * c.Hk + head) * KvBlock<D>::kBytes;
}

// Inclusive sums over the lanes of a wavefront (DPP row shifts and broadcasts).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}

// The greatest of the lanes' values, in lane 63.
__device__ __forceinline__ uint32_t wave_greatest(uint32_t v) {
  const auto with = [&](int o) { v = static_cast<uint32_t>(o) > v ? static_cast<uint32_t>(o) : v; };
  with(__builtin_amdgcn_update_dpp(v, v, 0x111, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(v, v, 0x112, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(v, v, 0x114, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(v, v, 0x118, 0xf, 0xf, false));
  with(__builtin_amdgcn_update_dpp(v, v, 0x142, 0xa, 0xf, false));
  with(__builtin_amdgcn_update_dpp(v, v, 0x143, 0xc, 0xf, false));
  return v;
}

__device__ __forceinline__ int lanes_below(unsigned long long mask) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0u));
}

// 16-bit element types.
struct F16 {
  static constexpr uint32_t kInf = 0x7C00u;
  // v >= 0 rounded towards zero, as bits.
  static __device__ __forceinline__ uint32_t truncated(float v) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(v, 0.0f)) & 0xFFFFu;
  }
  static __device__ __forceinline__ float load(uint32_t bits) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  }
  static __device__ __forceinline__ uint32_t store(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
};
struct BF16 {
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ uint32_t truncated(float v) { return __float_as_uint(v) >> 16; }
  static __device__ __forceinline__ float load(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ uint32_t store(float v) {  // to the nearest, ties to even
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};

// Two elements of a dword, and back.
template <class E>
__device__ __forceinline__ float elem_lo(uint32_t w) { return E::load(w & 0xFFFFu); }
template <class E>
__device__ __forceinline__ float elem_hi(uint32_t w) { return E::load(w >> 16); }
template <class E>
__device__ __forceinline__ uint32_t elem_pack(float lo, float hi) { return E::store(lo) | (E::store(hi) << 16); }

}  // namespace skinny

#endif
