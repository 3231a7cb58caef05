// The 4-bit key/value cache outside attention: writing a step's tokens,
// reading slots back, and eviction by accumulated weight.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "kv4.cuh"

namespace skinny {
namespace {

constexpr int kThreads = 256;

// 16 values of a head to NVFP4.  The scale is the E4M3 value nearest to
// amax / (6 g); a code is the E2M1 value nearest to x / (scale * g).  Both
// are decided on exact numbers: scale * g has at most 28 significant bits, so
// it and its products with the seven borders between codes are exact in fp64,
// and each border becomes the least fp32 number on its upper side (values on
// a border go to the even code).  A code is then a count of integer compares.
struct Quantized {
  u32x2 codes;
  uint8_t scale;
};

__device__ __forceinline__ Quantized quantize16(const float (&x)[16], float g) {
  float amax = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax = fmaxf(amax, fabsf(x[i]));
    nan |= x[i] != x[i];
  }
  double ratio = static_cast<double>(amax) / (6.0 * static_cast<double>(g));
  ratio = ratio < 448.0 ? ratio : 448.0;
  // E4M3: steps of 2^(e-3) in the binade of 2^e, e at least -6.
  int e = ratio >= 0x1p-6 ? static_cast<int>((__double_as_longlong(ratio) >> 52) & 0x7FF) - 1023 : -6;
  const int steps = static_cast<int>(__builtin_rint(ldexp(ratio, 3 - e)));  // 0 .. 16
  const int byte = (e + 7) * 8 + steps - 8;
  const double unit = ldexp(static_cast<double>(steps), e - 3) * static_cast<double>(g);
  uint32_t least[7];
  constexpr double kBorder[7] = {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const double b = kBorder[i] * unit;
    const float down = __double2float_rz(b);
    // Even borders (0.25, 1.25, 2.5, 5) belong to the lower code.
    least[i] = __float_as_uint(down) + ((i % 2 == 0 || static_cast<double>(down) < b) ? 1u : 0u);
  }
  u32x2 out{0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    uint32_t code = __float_as_uint(x[i]) >> 31 << 3;
#pragma unroll
    for (int j = 0; j < 7; ++j) code += a >= least[j];
    if (i < 8) out.x |= code << (4 * i);
    else out.y |= code << (4 * (i - 8));
  }
  Quantized q;
  q.scale = nan ? 0x7F : static_cast<uint8_t>(byte);
  q.codes = (nan || steps == 0) ? u32x2{0u, 0u} : out;
  return q;
}

// The places of a workgroup of append and read: sequence, page of the table
// and head, the pages being those that the newest T slots can reach.
struct Place {
  int b, page, head, len, first;  // first: the oldest slot of the T (may be negative)
};
__host__ __device__ inline int pages_of_rows(int T) { return (T + kPage - 2) / kPage + 1; }
__device__ __forceinline__ bool find_place(const kv4_cache& c, int T, int np, Place& p) {
  int i = blockIdx.x;
  p.head = i % c.Hk;
  i /= c.Hk;
  p.b = i / np;
  p.len = kv_len(c, p.b);
  p.first = p.len - T;
  p.page = (p.first > 0 ? p.first : 0) / kPage + i % np;
  return p.page * kPage < p.len;
}

// One workgroup per sequence, reached page and head; a thread takes 16 values
// of a token's key or value.
template <int D, class E>
__global__ __launch_bounds__(kThreads) void append(const kv4_cache c, const kv4_rows k, const kv4_rows v, int T, int np) {
  Place p;
  if (!find_place(c, T, np, p)) return;
  uint8_t* block = kv_block<D>(c, c.table[static_cast<size_t>(p.b) * c.width + p.page], p.head);
  if (!block) return;
  constexpr int G = KvBlock<D>::kGroups;
  for (int i = threadIdx.x; i < kPage * G * 2; i += kThreads) {
    const int f = i % G, t = i / G % kPage;
    const bool isv = i >= kPage * G;
    const int slot = p.page * kPage + t, row = slot - p.first;
    if (row < 0 || slot >= p.len) continue;
    const kv4_rows& r = isv ? v : k;
    const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(r.data) + p.b * r.sequence +
                                                      row * r.row + p.head * r.head + f * 16);
    const u32x4 a = src[0], b = src[1];
    float x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = elem_lo<E>(a[j]);
      x[2 * j + 1] = elem_hi<E>(a[j]);
      x[8 + 2 * j] = elem_lo<E>(b[j]);
      x[8 + 2 * j + 1] = elem_hi<E>(b[j]);
    }
    const Quantized q = quantize16(x, isv ? c.gv : c.gk);
    kv_codes_store<D>(block, t, f, isv, q.codes);
    block[kv_scale_at<D>(t, f, isv)] = q.scale;
  }
}

// 16 held values from their codes and scale, rounded once to E.
template <class E>
__device__ __forceinline__ void held16(u32x2 codes, uint32_t scale, float g, u32x4 (&out)[2]) {
  const float s = e4m3f<0>(scale);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f16x8 c = e2m1x8(codes[h]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[h][j] = elem_pack<E>(static_cast<float>(c[2 * j]) * s * g, static_cast<float>(c[2 * j + 1]) * s * g);
  }
}

// As append, the other way round.  Rows without a slot are zeros: their
// workgroups are those past the sequence's pages, which there are enough of.
template <int D, class E>
__global__ __launch_bounds__(kThreads) void read_rows(const kv4_cache c, uint16_t* k, uint16_t* v, int n, int np) {
  constexpr int G = KvBlock<D>::kGroups;
  const int h = blockIdx.x % c.Hk;
  const int64_t at = blockIdx.x / c.Hk;
  const int b = static_cast<int>(at / np);
  const int row0 = static_cast<int>(at % np) * kPage;  // 64 rows of the output
  const int len = kv_len(c, b);
  for (int i = threadIdx.x; i < kPage * G * 2; i += kThreads) {
    const int f = i % G, row = row0 + i / G % kPage;
    const bool isv = i >= kPage * G;
    if (row >= n) continue;
    const int slot = len - n + row;
    u32x4 out[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
    if (slot >= 0) {
      const uint8_t* block = kv_block<D>(c, c.table[static_cast<size_t>(b) * c.width + slot / kPage], h);
      if (block) {
        const int t = slot % kPage;
        held16<E>(kv_codes_load<D>(block, t, f, isv), block[kv_scale_at<D>(t, f, isv)], isv ? c.gv : c.gk, out);
      }
    }
    u32x4* dst = reinterpret_cast<u32x4*>((isv ? v : k) + ((static_cast<size_t>(b) * n + row) * c.Hk + h) * D + f * 16);
    dst[0] = out[0];
    dst[1] = out[1];
  }
}

// ---- eviction ---------------------------------------------------------------
constexpr int kSelectThreads = 1024;
constexpr int kBins = 2048;

// Orders like the weight; a NaN is the least.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Exclusive sums over the workgroup's threads; every thread also gets the total.
__device__ __forceinline__ int block_scan(int v, int* tmp, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 63) tmp[wave] = s;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kSelectThreads / 64; ++w) {
    if (w < wave) before += tmp[w];
    total += tmp[w];
  }
  return before + s - v;
}

// One workgroup per sequence and head finds the key of the last slot kept by
// narrowing a range of keys: bins of equal width over the range's keys, the
// bin that holds the wanted rank, and again within it until it is one key (at
// most three times for 32-bit keys).  Equal-width bins between the least and
// the greatest key spread weights that differ by factors over many bins.
__global__ __launch_bounds__(kSelectThreads) void select_slots(const kv4_cache c, const float* acc, int dst_width,
                                                               int32_t* kept, int32_t* new_lens, float* new_acc,
                                                               int keep, int sinks, int recent) {
  __shared__ int bins[kBins];
  __shared__ int tmp[kSelectThreads / 64];
  __shared__ uint32_t range[2];
  __shared__ int found[2];
  const int tid = threadIdx.x;
  const int h = blockIdx.x % c.Hk, b = blockIdx.x / c.Hk;
  const int n = kv_len(c, b);
  const float* w = acc + (static_cast<size_t>(b) * c.Hk + h) * c.width * kPage;
  int32_t* ids = kept + (static_cast<size_t>(b) * c.Hk + h) * keep;
  float* out = new_acc + (static_cast<size_t>(b) * c.Hk + h) * dst_width * kPage;
  const int m = n < keep ? n : keep;
  if (h == 0 && tid == 0) new_lens[b] = m;
  for (int i = m + tid; i < keep; i += kSelectThreads) ids[i] = -1;
  for (int i = m + tid; i < dst_width * kPage; i += kSelectThreads) out[i] = 0.0f;
  if (n <= keep) {
    for (int i = tid; i < n; i += kSelectThreads) {
      ids[i] = i;
      out[i] = w[i];
    }
    return;
  }
  // More slots than stay: those between the sinks and the recent ones compete.
  const int lo_slot = sinks, hi_slot = n - recent;
  int need = keep - sinks - recent;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  for (int i = lo_slot + tid; i < hi_slot; i += kSelectThreads) {
    const uint32_t key = weight_key(w[i]);
    lo = key < lo ? key : lo;
    hi = key > hi ? key : hi;
  }
  if (tid == 0) {
    range[0] = 0xFFFFFFFFu;
    range[1] = 0u;
  }
  __syncthreads();
  atomicMin(&range[0], lo);
  atomicMax(&range[1], hi);
  __syncthreads();
  lo = range[0];
  hi = range[1];
  while (need > 0 && lo < hi) {
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
    __syncthreads();
    for (int i = lo_slot + tid; i < hi_slot; i += kSelectThreads) {
      const uint32_t key = weight_key(w[i]);
      if (key >= lo && key <= hi) atomicAdd(&bins[(key - lo) >> shift], 1);
    }
    __syncthreads();
    // Bins from the top: thread t has bins kBins-1-2t and kBins-2-2t.
    const int top = kBins - 1 - 2 * tid, a = bins[top], d = bins[top - 1];
    int total;
    const int above = block_scan(a + d, tmp, total);
    if (above < need && need <= above + a + d) {
      const bool first = need <= above + a;
      found[0] = first ? top : top - 1;
      found[1] = first ? above : above + a;
    }
    __syncthreads();
    need -= found[1];
    const uint32_t base = lo + (static_cast<uint32_t>(found[0]) << shift);
    const uint32_t last = base + ((1u << shift) - 1u);
    lo = base;
    hi = last < base || last > hi ? hi : last;
    __syncthreads();
    if (shift == 0) hi = lo;
  }
  // Every key above lo stays, and `need` of those equal to it, the lowest slots.
  const uint32_t edge = need > 0 ? lo : 0xFFFFFFFFu;
  const int per = (n + kSelectThreads - 1) / kSelectThreads;
  const int s0 = tid * per, s1 = s0 + per < n ? s0 + per : n;
  int above = 0, equal = 0;
  for (int s = s0; s < s1; ++s) {
    const uint32_t key = s < sinks || s >= hi_slot ? 0xFFFFFFFFu : weight_key(w[s]);
    above += s < sinks || s >= hi_slot || (key > edge);
    equal += key == edge && s >= sinks && s < hi_slot;
  }
  int total;
  int left = need - block_scan(equal, tmp, total);
  left = left < 0 ? 0 : left;
  int at = block_scan(above + (equal < left ? equal : left), tmp, total);
  for (int s = s0; s < s1; ++s) {
    const float weight = w[s];
    const bool sure = s < sinks || s >= hi_slot;
    const uint32_t key = weight_key(weight);
    const bool tie = !sure && key == edge && left > 0;
    if (tie) --left;
    if (sure || key > edge || tie) {
      ids[at] = s;
      out[at] = weight;
      ++at;
    }
  }
}

// One workgroup per page written: its tokens' codes and scales are gathered
// into LDS and leave as one block.
template <int D>
__global__ __launch_bounds__(kThreads) void copy_kept(const kv4_cache c, const kv4_cache dst, const int32_t* kept,
                                                      int keep, int np) {
  __shared__ __align__(16) uint8_t image[KvBlock<D>::kBytes];
  constexpr int G = KvBlock<D>::kGroups;
  const int h = blockIdx.x % c.Hk;
  const int64_t at = blockIdx.x / c.Hk;
  const int b = static_cast<int>(at / np), page = static_cast<int>(at % np);
  const int n = kv_len(c, b), m = n < keep ? n : keep;
  if (page * kPage >= m) return;
  uint8_t* out = kv_block<D>(dst, dst.table[static_cast<size_t>(b) * dst.width + page], h);
  if (!out) return;
  const int32_t* ids = kept + (static_cast<size_t>(b) * c.Hk + h) * keep + page * kPage;
  for (int i = threadIdx.x; i < kPage * G * 2; i += kThreads) {
    const int f = i % G, t = i / G % kPage;
    const bool isv = i >= kPage * G;
    u32x2 codes{0u, 0u};
    uint8_t scale = 0;
    if (page * kPage + t < m) {
      const int slot = ids[t];
      const uint8_t* block = kv_block<D>(c, c.table[static_cast<size_t>(b) * c.width + slot / kPage], h);
      if (block) {
        codes = kv_codes_load<D>(block, slot % kPage, f, isv);
        scale = block[kv_scale_at<D>(slot % kPage, f, isv)];
      }
    }
    kv_codes_store<D>(image, t, f, isv, codes);
    image[kv_scale_at<D>(t, f, isv)] = scale;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < KvBlock<D>::kBytes / 16; i += kThreads)
    reinterpret_cast<u32x4*>(out)[i] = reinterpret_cast<const u32x4*>(image)[i];
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
  return by_head_size(c.D, [&](auto d) {
    if (type == SKINNY_F16) append<d(), F16><<<grid, kThreads, 0, stream>>>(c, k, v, T, np);
    else append<d(), BF16><<<grid, kThreads, 0, stream>>>(c, k, v, T, np);
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
  select_slots<<<dim3(static_cast<unsigned>(c.B * c.Hk)), kSelectThreads, 0, stream>>>(
      c, acc, dst.width, kept, new_lens, new_acc, keep, sinks, recent);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int np = (keep + kPage - 1) / kPage;
  np = np < c.width ? np : c.width;  // no more slots stay than there are
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(c.B) * np * c.Hk));
  return by_head_size(c.D, [&](auto d) { copy_kept<d()><<<grid, kThreads, 0, stream>>>(c, dst, kept, keep, np); });
}

}  // namespace skinny
