// The 4-bit key/value cache outside attention: writing a step's tokens,
// reading slots back, and eviction by accumulated weight.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "kv4.cuh"
#include "kv4_internal.h"

namespace skinny {
namespace {

constexpr int kThreads = 256;

// 16 values of a head to NVFP4.  The scale is the E4M3 value nearest to
// amax / (6 g); a code is the E2M1 value nearest to x / (scale * g).  Both
// are decided on exact numbers.
//
// The scale: amax has 11 significant bits at most and 6 g 27, so a quotient
// that is not half way between two E4M3 values is 2^-36 of itself from it at
// least.  amax * (1 / 6g) in fp64 is off by 2^-52, and rounding it to a
// multiple of 2^-40 of an E4M3 step first brings those half way back there.
//
// A code: scale * g has at most 28 significant bits, so it and its products
// with the seven borders between codes are exact in fp64, and each border
// becomes the greatest E value that does not pass it (values on a border go
// to the even code).  Magnitudes then compare as 16-bit integers, two to a
// register, and the sign bits of limit - magnitude are the comparisons: c0 ..
// c6 are a thermometer, so code bit 2 is c3, bit 1 is c1 ^ c3 ^ c5 and bit 0
// is the parity of all.  Ten operations a value, against 18 for counting fp32
// comparisons (append of 4 x 8192 tokens, 4 heads of 128: 40 -> 25 us with the
// page's image below, which is 86 MB at 3.6 TB/s).
struct Quantized {
  u32x2 codes;
  uint8_t scale;
};

typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// a where mask is set, b elsewhere; the parity of three.
__device__ __forceinline__ uint32_t bits_of(uint32_t mask, uint32_t a, uint32_t b) {
  return __builtin_amdgcn_bitop3_b32(mask, a, b, 0xCA);
}
__device__ __forceinline__ uint32_t odd(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
}

// Nibbles 0 .. 3 of the low half of v to the even nibbles, of the high half to the odd ones.
__device__ __forceinline__ uint32_t interleave_nibbles(uint32_t v) {
  uint32_t lo = v & 0xFFFFu, hi = v >> 16;
  lo = (lo | (lo << 8)) & 0x00FF00FFu;
  hi = (hi | (hi << 8)) & 0x00FF00FFu;
  lo = (lo | (lo << 4)) & 0x0F0F0F0Fu;
  hi = (hi | (hi << 4)) & 0x0F0F0F0Fu;
  return lo | (hi << 4);
}

template <class E>
__device__ __forceinline__ Quantized quantize16(const u32x4 (&x)[2], double g, double inv6g) {
  u16x2 most{0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, x[i / 4][i % 4] & 0x7FFF7FFFu));
  const uint32_t amax = most.x > most.y ? most.x : most.y;
  const bool nan = amax > E::kInf;
  double ratio = static_cast<double>(E::load(amax)) * inv6g;
  ratio = ratio < 448.0 ? ratio : 448.0;
  // E4M3: steps of 2^(e-3) in the binade of 2^e, e at least -6.
  int e = ratio >= 0x1p-6 ? static_cast<int>((__double_as_longlong(ratio) >> 52) & 0x7FF) - 1023 : -6;
  const int steps = static_cast<int>(__builtin_rint(ldexp(__builtin_rint(ldexp(ratio, 43 - e)), -40)));  // 0 .. 16
  const int byte = (e + 7) * 8 + steps - 8;
  const double unit = ldexp(static_cast<double>(steps), e - 3) * g;
  i16x2 below[7];
  constexpr double kBorder[7] = {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const double b = kBorder[i] * unit;
    // Truncating the nearest float gives the greatest E value up to b or the
    // next one.  Even borders (0.25, 1.25, 2.5, 5) belong to the lower code.
    const uint32_t down = E::truncated(static_cast<float>(b));
    const double value = E::load(down);
    const uint32_t limit = down - ((i % 2 ? value >= b : value > b) ? 1u : 0u);
    below[i] = __builtin_bit_cast(i16x2, limit | (limit << 16));
  }
  u32x2 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t codes = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = x[h][i];
      const i16x2 a = __builtin_bit_cast(i16x2, w & 0x7FFF7FFFu);
      uint32_t c[7];
#pragma unroll
      for (int j = 0; j < 7; ++j) c[j] = __builtin_bit_cast(uint32_t, below[j] - a);
      const uint32_t mid = odd(c[1], c[3], c[5]), low = odd(odd(c[0], c[2], c[4]), c[6], mid);
      constexpr uint32_t kTop = 0x80008000u;
      const uint32_t code = bits_of(kTop, w, bits_of(kTop, c[3], bits_of(kTop, mid, low >> 1) >> 1) >> 1);
      codes = bits_of(0xF000F000u, code, codes >> 4);
    }
    out[h] = interleave_nibbles(codes);
  }
  Quantized q;
  q.scale = nan ? 0x7F : static_cast<uint8_t>(byte);
  q.codes = (nan || steps == 0) ? u32x2{0u, 0u} : out;
  return q;
}

// The places of a workgroup of append: sequence, page of the table and head,
// the pages being those that the newest T slots can reach.
struct Place {
  int b, page, head, len, first;  // first: the oldest slot of the T (may be negative)
};
__host__ __device__ inline int pages_of_rows(int T) { return (T + kPage - 2) / kPage + 1; }
__device__ __forceinline__ bool find_place(const kv4_cache& c, int T, int np, Place& p) {
  int i = blockIdx.x;
  p.head = i % c.Hk;
  i /= c.Hk;
  p.b = i / np;
  p.len = kv_len_uniform(c, p.b);
  p.first = p.len - T;
  p.page = (p.first > 0 ? p.first : 0) / kPage + i % np;
  return p.page * kPage < p.len;
}

// The page's image in LDS leaves as whole 16-byte vectors.
template <int D>
__device__ __forceinline__ void store_image(uint8_t* out, const uint8_t* image) {
  __syncthreads();
  for (int i = threadIdx.x; i < KvBlock<D>::kBytes / 16; i += kThreads)
    reinterpret_cast<u32x4*>(out)[i] = reinterpret_cast<const u32x4*>(image)[i];
}

// One workgroup per sequence, reached page and head; a thread takes 16 values
// of a token's key or value, and all of its loads are in flight before the
// first is used.  A page that the step fills is put together in LDS; of one
// that it shares with older slots only the new tokens' bytes are written.
template <int D, class E>
__global__ __launch_bounds__(kThreads) void append(const kv4_cache c, const kv4_rows k, const kv4_rows v, int T, int np,
                                                   double inv6gk, double inv6gv) {
  __shared__ __align__(16) uint8_t image[KvBlock<D>::kBytes];
  Place p;
  if (!find_place(c, T, np, p)) return;
  uint8_t* block = kv_block<D>(c, uniform_load(c.table, static_cast<int64_t>(p.b) * c.width + p.page), p.head);
  if (!block) return;
  constexpr int G = KvBlock<D>::kGroups, kItems = kPage * G * 2 / kThreads, kBatch = kItems < 4 ? kItems : 4;
  const bool whole = p.page * kPage >= p.first && (p.page + 1) * kPage <= p.len;
#pragma unroll 1
  for (int n0 = 0; n0 < kItems; n0 += kBatch) {
    u32x4 x[kBatch][2];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int i = (n0 + n) * kThreads + threadIdx.x, f = i % G, t = i / G % kPage;
      const int slot = p.page * kPage + t, row = slot - p.first;
      const kv4_rows& r = n0 + n >= kItems / 2 ? v : k;  // kPage * G is a multiple of kThreads
      if (row >= 0 && slot < p.len) {
        const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(r.data) + p.b * r.sequence +
                                                          row * r.row + p.head * r.head + f * 16);
        x[n][0] = load16(src);
        x[n][1] = load16(src + 1);
      } else {
        x[n][0] = x[n][1] = u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int i = (n0 + n) * kThreads + threadIdx.x, f = i % G, t = i / G % kPage;
      const int slot = p.page * kPage + t, row = slot - p.first;
      if (row < 0 || slot >= p.len) continue;
      const bool second = n0 + n >= kItems / 2;
      const Quantized q = quantize16<E>(x[n], second ? c.gv : c.gk, second ? inv6gv : inv6gk);
      if (whole) {
        kv_codes_store<D>(image, t, f, second, q.codes);
        image[kv_scale_at<D>(t, f, second)] = q.scale;
      } else {
        kv_codes_store<D>(block, t, f, second, q.codes);
        block[kv_scale_at<D>(t, f, second)] = q.scale;
      }
    }
  }
  if (whole) store_image<D>(block, image);
}

// Eight held values from their codes and scale.  code * scale is exact; the product
// with g is rounded to fp32 and then to E, so a result next to the middle of two
// of E's values can be the farther one (by 2^-24 of itself).
template <class E>
__device__ __forceinline__ u32x4 held8(uint32_t codes, uint32_t scale, float g) {
  const float s = e4m3f<0>(scale);
  const f16x8 c = e2m1x8(codes);
  u32x4 out;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    out[j] = elem_pack<E>(static_cast<float>(c[2 * j]) * s * g, static_cast<float>(c[2 * j + 1]) * s * g);
  return out;
}

// One workgroup per sequence, head and 64 rows of the output, whose slots lie
// in two pages at most; a thread takes eight values, so that neighbours' loads
// and stores are contiguous.  Bound by memory, its writes above all, which go
// past the caches: 16 x 8192 tokens, four heads of 128, 268 MB written and 75 MB
// read in 55 us after the eviction that wrote the pages (76 with ordinary stores).
template <int D, class E>
__global__ __launch_bounds__(kThreads) void read_rows(const kv4_cache c, uint16_t* k, uint16_t* v, int n, int np) {
  constexpr int P = D / 8, kItems = kPage * P * 2 / kThreads, kBatch = kItems < 8 ? kItems : 8;
  const int h = blockIdx.x % c.Hk;
  const int64_t at = blockIdx.x / c.Hk;
  const int b = static_cast<int>(at / np);
  const int row0 = static_cast<int>(at % np) * kPage;
  const int first = kv_len_uniform(c, b) - n + row0;  // slot of the first row
  const uint8_t* block[2] = {nullptr, nullptr};
  const int p0 = (first > 0 ? first : 0) / kPage;
  const int slots = first + (n - row0 < kPage ? n - row0 : kPage);  // past the last row's slot
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if ((p0 + i) * kPage < slots)
      block[i] = kv_block<D>(c, uniform_load(c.table, static_cast<int64_t>(b) * c.width + p0 + i), h);
#pragma unroll 1
  for (int n0 = 0; n0 < kItems; n0 += kBatch) {
    uint32_t codes[kBatch], scale[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = (n0 + u) * kThreads + threadIdx.x, piece = i % P, r = i / P % kPage;
      const bool isv = n0 + u >= kItems / 2;
      const int slot = first + r;
      const uint8_t* from = slot / kPage == p0 ? block[0] : block[1];
      codes[u] = scale[u] = 0u;
      if (slot >= 0 && row0 + r < n && from) {
        const int t = slot % kPage;
        codes[u] = kv_codes_load_half<D>(from, t, piece, isv);
        scale[u] = from[kv_scale_at<D>(t, piece / 2, isv)];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = (n0 + u) * kThreads + threadIdx.x, piece = i % P, r = i / P % kPage;
      const bool isv = n0 + u >= kItems / 2;
      if (row0 + r >= n) continue;
      uint16_t* dst = (isv ? v : k) + ((static_cast<size_t>(b) * n + row0 + r) * c.Hk + h) * D + piece * 8;
      __builtin_nontemporal_store(held8<E>(codes[u], scale[u], isv ? c.gv : c.gk), reinterpret_cast<u32x4*>(dst));
    }
  }
}

// ---- eviction ---------------------------------------------------------------
constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kRows = 8;                             // most groups of four keys of a thread in LDS
constexpr int kRowSlots = 4 * kSelectThreads;
constexpr int kTileSlots = kRows * kRowSlots;
constexpr int kBins = 2048;
constexpr uint32_t kOutside = 0u, kSure = 0xFFFFFFFFu;

// Orders like the weight, between kOutside and kSure; a NaN is the least.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 1u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive sums over the workgroup's threads; every thread also gets the total.
__device__ __forceinline__ int2 block_scan(int2 v, int2* tmp, int2& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int2 s{wave_scan(v.x), wave_scan(v.y)};
  __syncthreads();
  if (lane == 63) tmp[wave] = s;
  __syncthreads();
  int2 part = lane < kSelectWaves ? tmp[lane] : int2{0, 0};
  part = int2{wave_scan(part.x), wave_scan(part.y)};
  const int w = __builtin_amdgcn_readfirstlane(wave);
  total = int2{__builtin_amdgcn_readlane(part.x, 63), __builtin_amdgcn_readlane(part.y, 63)};
  const int2 before{w ? __builtin_amdgcn_readlane(part.x, w - 1) : 0, w ? __builtin_amdgcn_readlane(part.y, w - 1) : 0};
  return int2{before.x + s.x - v.x, before.y + s.y - v.y};
}

// One workgroup per sequence and head finds the key of the last slot kept by
// narrowing a range of keys: bins of equal width over the range's keys, the
// bin that holds the wanted rank, and again within it until it is one key or
// all of its keys stay (at most three times for 32-bit keys).  Equal-width bins between the least and
// the greatest key spread weights that differ by factors over many bins.
//
// The keys lie in LDS, where a thread finds those that it put there itself,
// four neighbours together: up to 32768 slots are read once, and longer
// sequences again, 32768 at a time, in each of the passes.  The loops stay
// short: with the keys in registers instead, the unrolled passes are 50 KB of
// code that runs once, and fetching it took longer than the work.  16
// sequences x 4 heads of 20000 .. 32768 slots, keeping 8192: 27 us (91 with a
// run of slots per thread, read four times over); one of 4133: 11 us (21).
__global__ __launch_bounds__(kSelectThreads) void select_slots(const kv4_cache c, const float* acc, int dst_width,
                                                               int32_t* kept, int32_t* new_lens, float* new_acc,
                                                               int keep, int sinks, int recent) {
  __shared__ int bins[kBins];
  __shared__ int2 tmp[kSelectWaves];
  __shared__ uint32_t range[2];
  __shared__ int found[2][3];
  __shared__ int2 count[kRows * kSelectWaves];  // of a wavefront's 256 slots: those above the last key, those equal to it
  const unsigned tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;  // slots of a tile may pass 2^31
  const int h = blockIdx.x % c.Hk, b = blockIdx.x / c.Hk;
  const unsigned n = kv_len_uniform(c, b);
  const float* w = acc + (static_cast<size_t>(b) * c.Hk + h) * c.width * kPage;
  int32_t* ids = kept + (static_cast<size_t>(b) * c.Hk + h) * keep;
  float* out = new_acc + (static_cast<size_t>(b) * c.Hk + h) * dst_width * kPage;
  const unsigned most = keep, places = dst_width * kPage, m = n < most ? n : most;
  if (h == 0 && tid == 0) new_lens[b] = m;
  for (unsigned i = m + tid; i < most; i += kSelectThreads) ids[i] = -1;
  for (unsigned i = m + tid; i < places; i += kSelectThreads) out[i] = 0.0f;
  if (n <= most) {
    for (unsigned i = tid; i < n; i += kSelectThreads) {
      ids[i] = i;
      out[i] = w[i];
    }
    return;
  }
  // More slots than stay: those between the sinks and the recent ones compete.
  const unsigned lo_slot = sinks, hi_slot = n - recent;
  int need = keep - sinks - recent;
  extern __shared__ u32x4 keys[];  // [kRows or fewer][kSelectThreads]
  const auto rows = [&](unsigned base) {
    const unsigned left = n - base;
    return left < kTileSlots ? (left + kRowSlots - 1) / kRowSlots : static_cast<unsigned>(kRows);
  };
  const auto load = [&](unsigned base) __attribute__((always_inline)) {
    const unsigned all = rows(base);
#pragma unroll 1
    for (unsigned i0 = 0; i0 < all; i0 += 4) {
      u32x4 held[4];
#pragma unroll
      for (unsigned i = 0; i < 4; ++i) {
        const unsigned s = base + (i0 + i) * kRowSlots + tid * 4;  // acc has whole pages: s + 3 is within it
        held[i] = *reinterpret_cast<const u32x4*>(w + (s < n ? s : 0u));
      }
#pragma unroll
      for (unsigned i = 0; i < 4; ++i) {
        u32x4 k;
#pragma unroll
        for (unsigned e = 0; e < 4; ++e) {
          const unsigned s = base + (i0 + i) * kRowSlots + tid * 4 + e;
          k[e] = s >= n ? kOutside : (s < lo_slot || s >= hi_slot ? kSure : weight_key(__uint_as_float(held[i][e])));
        }
        if (i0 + i < all) keys[(i0 + i) * kSelectThreads + tid] = k;
      }
    }
  };
  // f over the thread's keys of every tile.
  const auto each = [&](auto f) __attribute__((always_inline)) {
    for (unsigned base = 0;; base += kTileSlots) {
      if (n > kTileSlots) load(base);
      const unsigned all = rows(base);
#pragma unroll 4
      for (unsigned i = 0; i < all; ++i) {
        const u32x4 k = keys[i * kSelectThreads + tid];
#pragma unroll
        for (int e = 0; e < 4; ++e) f(k[e]);
      }
      if (n - base <= kTileSlots) break;
    }
  };
  if (n <= kTileSlots) load(0);
  if (tid == 0) {
    range[0] = kSure;
    range[1] = 0u;
  }
  for (unsigned i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
  __syncthreads();
  uint32_t lo = kSure, hi = 0u;
  each([&](uint32_t k) __attribute__((always_inline)) {
    if (k != kOutside && k != kSure) {
      lo = k < lo ? k : lo;
      hi = k > hi ? k : hi;
    }
  });
  lo = ~wave_greatest(~lo);
  hi = wave_greatest(hi);
  if (lane == 63) {
    atomicMin(&range[0], lo);
    atomicMax(&range[1], hi);
  }
  __syncthreads();
  lo = range[0];
  hi = range[1];
  bool whole = false;  // every key from lo on stays
  for (int pass = 0; need > 0 && lo < hi && !whole; ++pass) {
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    each([&](uint32_t k) __attribute__((always_inline)) {
      if (k - lo <= hi - lo) atomicAdd(&bins[(k - lo) >> shift], 1);
    });
    __syncthreads();
    // Bins from the top: thread t has bins kBins-1-2t and kBins-2-2t, and clears them for the next pass.
    const int top = kBins - 1 - 2 * static_cast<int>(tid), a = bins[top], d = bins[top - 1];
    bins[top] = bins[top - 1] = 0;
    int2 total;
    const int above = block_scan(int2{a + d, 0}, tmp, total).x;
    int* at = found[pass % 2];  // the bin, the keys above it, and its own
    if (above < need && need <= above + a + d) {
      const bool first = need <= above + a;
      at[0] = first ? top : top - 1;
      at[1] = first ? above : above + a;
      at[2] = first ? a : d;
    }
    __syncthreads();
    need -= at[1];
    whole = need == at[2];
    const uint32_t base = lo + (static_cast<uint32_t>(at[0]) << shift);
    const uint32_t last = base + ((1u << shift) - 1u);
    lo = base;
    hi = last < base || last > hi ? hi : last;
    if (shift == 0) hi = lo;
  }
  // Every key above the edge stays, and `need` of those equal to it, the lowest
  // slots: a slot's place is the number of slots before it that stay.
  if (whole) need = 0;
  const uint32_t edge = whole ? lo - 1u : (need > 0 ? lo : kSure - 1u);
  int2 before{0, 0};
  for (unsigned base = 0;; base += kTileSlots) {
    if (n > kTileSlots) load(base);
    const unsigned all = rows(base);
#pragma unroll 4
    for (unsigned i = 0; i < all; ++i) {
      const u32x4 k = keys[i * kSelectThreads + tid];
      int above = 0, equal = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        above += __popcll(__ballot(k[e] > edge));
        equal += __popcll(__ballot(k[e] == edge));
      }
      if (lane == 0) count[i * kSelectWaves + wave] = int2{above, equal};
    }
    __syncthreads();
    int2 total;
    const int2 mine = block_scan(tid < all * kSelectWaves ? count[tid] : int2{0, 0}, tmp, total);
    if (tid < all * kSelectWaves) count[tid] = int2{before.x + mine.x, before.y + mine.y};
    __syncthreads();
#pragma unroll 4
    for (unsigned i = 0; i < all; ++i) {
      const u32x4 k = keys[i * kSelectThreads + tid];
      int above = count[i * kSelectWaves + wave].x, equal = count[i * kSelectWaves + wave].y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        above += lanes_below(__ballot(k[e] > edge));
        equal += lanes_below(__ballot(k[e] == edge));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k[e] > edge || (k[e] == edge && equal < need)) {
          const int place = above + (equal < need ? equal : need);
          const unsigned s = base + i * kRowSlots + tid * 4 + e;
          ids[place] = s;
          out[place] = w[s];
        }
        above += k[e] > edge;
        equal += k[e] == edge;
      }
    }
    before.x += total.x;
    before.y += total.y;
    if (n - base <= kTileSlots) break;
    __syncthreads();
  }
}

// One workgroup per page written: its tokens' codes and scales are gathered
// into LDS, all loads in flight at once, and leave as one block.  Neighbours
// among the kept slots share lines of the source, so each load's lanes are
// chosen to meet in them: 64 tokens for one piece of K, and of the scales, and
// four tokens for the whole of V, whose 16 pieces lie in two lines.  Codes of
// the source are loaded non-temporally: they are done with, and what is written
// here is read next.  Bound by memory: keeping a third of the slots touches
// nearly every line of the source, so 16 sequences x 4 heads x 8192 slots kept
// of 20000 .. 32768 read 232 MB and write 75 MB, in 58 to 61 us (94 with the caches'
// own order; 64, and 10 more for the reading that follows, with the stores
// non-temporal too).
template <int D>
__global__ __launch_bounds__(kThreads) void copy_kept(const kv4_cache c, const kv4_cache dst, const int32_t* kept,
                                                      int keep, int np) {
  using Block = KvBlock<D>;
  using KPiece = std::conditional_t<D == 64, u32x2, u32x4>;
  using KScales = std::conditional_t<D == 64, uint8_t, std::conditional_t<D == 128, uint16_t, uint32_t>>;
  using VPiece = std::conditional_t<D == 64, uint16_t, std::conditional_t<D == 128, uint32_t, u32x2>>;
  constexpr int kKPieces = D == 256 ? 2 : 1, kVScales = D / 64, kVPieces = kPage * 16 / kThreads;
  __shared__ __align__(16) uint8_t image[Block::kBytes];
  __shared__ const uint8_t* from[kPage];  // each token's block
  __shared__ int token[kPage];
  const int h = blockIdx.x % c.Hk;
  const int64_t at = blockIdx.x / c.Hk;
  const int b = static_cast<int>(at / np), page = static_cast<int>(at % np);
  const int n = kv_len_uniform(c, b), m = n < keep ? n : keep;
  if (page * kPage >= m) return;
  uint8_t* out = kv_block<D>(dst, uniform_load(dst.table, static_cast<int64_t>(b) * dst.width + page), h);
  if (!out) return;
  if (threadIdx.x < kPage) {
    const int place = page * kPage + threadIdx.x;
    const int slot = place < m ? kept[(static_cast<size_t>(b) * c.Hk + h) * keep + place] : -1;
    from[threadIdx.x] = slot < 0 ? nullptr : kv_block<D>(c, c.table[static_cast<size_t>(b) * c.width + slot / kPage], h);
    token[threadIdx.x] = slot % kPage;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, quarter = threadIdx.x >> 6, column = threadIdx.x % 16;
  const uint8_t* block = from[lane];
  const int t = token[lane];
  KPiece kc[kKPieces]{};
  KScales ks{};
  uint8_t vs[kVScales]{};
  VPiece vc[kVPieces]{};
  if (block) {
#pragma unroll
    for (int i = 0; i < kKPieces; ++i)
      kc[i] = __builtin_nontemporal_load(reinterpret_cast<const KPiece*>(block + Block::k_codes(t, quarter * (D / 64) + 2 * i)));
    ks = *reinterpret_cast<const KScales*>(block + Block::k_scale(t, quarter * (D / 64)));
#pragma unroll
    for (int i = 0; i < kVScales; ++i) vs[i] = block[Block::v_scale(t, quarter * kVScales + i)];
  }
#pragma unroll
  for (int i = 0; i < kVPieces; ++i) {
    const int j = i * (kThreads / 16) + threadIdx.x / 16;
    if (from[j]) vc[i] = __builtin_nontemporal_load(reinterpret_cast<const VPiece*>(from[j] + Block::v_codes(token[j], 0) + column * 16));
  }
#pragma unroll
  for (int i = 0; i < kKPieces; ++i)
    *reinterpret_cast<KPiece*>(image + Block::k_codes(lane, quarter * (D / 64) + 2 * i)) = kc[i];
  *reinterpret_cast<KScales*>(image + Block::k_scale(lane, quarter * (D / 64))) = ks;
#pragma unroll
  for (int i = 0; i < kVScales; ++i) image[Block::v_scale(lane, quarter * kVScales + i)] = vs[i];
#pragma unroll
  for (int i = 0; i < kVPieces; ++i) {
    const int j = i * (kThreads / 16) + threadIdx.x / 16;
    *reinterpret_cast<VPiece*>(image + Block::v_codes(j, 0) + column * 16) = vc[i];
  }
  store_image<D>(out, image);
}

template <class F>
hipError_t by_head_size(int D, F f) {
  if (D == 64) f(std::integral_constant<int, 64>());
  else if (D == 128) f(std::integral_constant<int, 128>());
  else f(std::integral_constant<int, 256>());
  return hipGetLastError();
}

}  // namespace

int kv4_row_pages(int rows) { return pages_of_rows(rows); }

hipError_t launch_kv4_append(const kv4_cache& c, const kv4_rows& k, const kv4_rows& v, int type, int T,
                             hipStream_t stream) {
  const int np = pages_of_rows(T);
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(c.B) * np * c.Hk));
  const double ik = 1.0 / (6.0 * static_cast<double>(c.gk)), iv = 1.0 / (6.0 * static_cast<double>(c.gv));
  return by_head_size(c.D, [&](auto d) {
    if (type == SKINNY_F16) append<d(), F16><<<grid, kThreads, 0, stream>>>(c, k, v, T, np, ik, iv);
    else append<d(), BF16><<<grid, kThreads, 0, stream>>>(c, k, v, T, np, ik, iv);
  });
}

hipError_t launch_kv4_read(const kv4_cache& c, uint16_t* k, uint16_t* v, int type, int n, hipStream_t stream) {
  const int np = (n + kPage - 1) / kPage;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(c.B) * np * c.Hk));
  return by_head_size(c.D, [&](auto d) {
    if (type == SKINNY_F16) read_rows<d(), F16><<<grid, kThreads, 0, stream>>>(c, k, v, n, np);
    else read_rows<d(), BF16><<<grid, kThreads, 0, stream>>>(c, k, v, n, np);
  });
}

hipError_t launch_kv4_evict(const kv4_cache& c, const float* acc, const kv4_cache& dst, int32_t* kept,
                            int32_t* new_lens, float* new_acc, int keep, int sinks, int recent, hipStream_t stream) {
  const int64_t held = (static_cast<int64_t>(c.width) * kPage + kRowSlots - 1) / kRowSlots;
  const size_t lds = static_cast<size_t>(held < kRows ? held : kRows) * kRowSlots * sizeof(uint32_t);
  select_slots<<<dim3(static_cast<unsigned>(c.B * c.Hk)), kSelectThreads, lds, stream>>>(
      c, acc, dst.width, kept, new_lens, new_acc, keep, sinks, recent);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int np = (keep + kPage - 1) / kPage;
  np = np < c.width ? np : c.width;  // no more slots stay than there are
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(c.B) * np * c.Hk));
  return by_head_size(c.D, [&](auto d) { copy_kept<d()><<<grid, kThreads, 0, stream>>>(c, dst, kept, keep, np); });
}

}  // namespace skinny
