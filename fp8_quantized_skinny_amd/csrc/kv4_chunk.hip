// Attention of chunks of new tokens over the 4-bit key/value cache.
//
// With S = scale q . K~ over the slots that a row sees:
//   out = sum_j exp(S_j - m) v~_j / sum_j exp(S_j - m),  lse = m + log(sum)
//
// A sequence's T tokens and the G query heads of a key/value head make T * G
// rows (row r: token r / G, head r % G), and a workgroup has a tile of
// kTile = 256 of them: eight wavefronts of 32 rows each.  It widens a page
// (64 tokens) to fp16 in LDS once for all of them, the next one while this one
// is used.  Both products run on v_mfma_f32_32x32x16_f16 in the transposed
// form, as in kv4_attention.hip:
//   S^T[token][row] = K[token][d] Q^T[d][row]
//   O^T[d][row]     = V^T[d][token] P^T[token][row]
// so that a row's scores, weights, maximum and sum stay in the two lanes that
// hold its column.  The first product takes the tokens of a tile of 32 in the
// order that leaves lane 32 h + c with row c's tokens 8 h .. 8 h + 7 of every 16,
// which is the second one's right operand.
#include <hip/hip_runtime.h>

#include "kv4.cuh"
#include "kv4_internal.h"

namespace skinny {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32 * kWaves;
constexpr int kSlots = 256;       // workgroups that the CUs hold at once
constexpr int kLeast = 16;        // fewest pages of a share of a split tile
constexpr int kPlanThreads = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMinNormal = 0x1p-126f;
// Weights go to fp16 relative to a reference that follows the running maximum
// only when that rose by more than 2^kSlack, times 2^kLift (as in
// kv4_attention.hip): below 2^14, and exact to 2^-11 down to 2^-20 of the greatest.
constexpr float kLift = 6.0f, kSlack = 8.0f;

// A tile's share of the pages that its rows see: view pages v0 .. v1.
struct Share {
  int b, first, T, tile;  // sequence, its first row and number of them, tile of it
  int v0, v1;
  int part;               // its place among the parts of split tiles, -1: it is the whole tile
  int pad;
};
struct Split {            // a tile of several shares
  int first, T, tile, part, shares;
};

struct ChunkArgs {
  kv4_cache c;
  const uint16_t* q;
  int64_t row, head;    // strides of q
  const int32_t* starts;
  void* out;
  float* lse;
  int* counts;          // [2]: shares, split tiles
  int* begin;           // [B + 1]: first row of each sequence
  int* offset;          // [B]: tiles before each sequence
  Share* share;
  Split* split;
  float* stat;          // [head][part][kTile][2]: reference maximum (log2) and sum
  float* part;          // [head][part][kTile][D]
  int64_t parts;        // per head
  int N, Hq, G, tiles;  // tiles: most that N rows of B sequences make
  int window, sinks;
  float scale;
};

// The slots that token t of a sequence's T sees, without a window: none where it has no slot itself.
__device__ __forceinline__ int limit_of(int len, int T, int t) {
  const int n = len - (T - 1 - t);
  return n < 0 ? 0 : n;
}

// The pages that the rows of a tile see: the first `low`, which hold the sinks,
// and those from `from` to `end`.
struct View {
  int low, from, end;
  __device__ __forceinline__ int pages() const { return end > from ? low + end - from : 0; }
  __device__ __forceinline__ int page(int v) const { return v < low ? v : v - low + from; }
};
__device__ __forceinline__ View view_of(const ChunkArgs& a, int len, int T, int tile) {
  const int64_t R = static_cast<int64_t>(T) * a.G;
  const int64_t r0 = static_cast<int64_t>(tile) * kTile, r1 = r0 + kTile < R ? r0 + kTile : R;
  const int least = limit_of(len, T, static_cast<int>(r0 / a.G)), most = limit_of(len, T, static_cast<int>((r1 - 1) / a.G));
  View v{0, 0, (most + kPage - 1) / kPage};
  if (a.window) {
    const int from = least - a.window;  // the earliest row's first slot of the window
    v.from = from > 0 ? from / kPage : 0;
    v.low = a.sinks / kPage + (a.sinks % kPage != 0);
    v.low = v.low < v.from ? v.low : v.from;
  }
  return v;
}

// ---- the plan -----------------------------------------------------------------
// One workgroup cuts every tile into shares of about equal numbers of pages, for
// two shares per CU at least where there are pages for that; the longest tiles of
// a sequence, its last, come first.
//
// The rows of a sequence go from its start to the next one's; a start that is not
// in 0 .. N counts as the nearer of these, and one below an earlier start as that:
// no two sequences have a row in common, whatever the starts are.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int sums[kPlanThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int in = wave_scan(v);
  __syncthreads();
  if (lane == 63) sums[wave] = in;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kPlanThreads / 64; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  *total = all;
  return before + in - v;
}

// The greatest of the threads' values up to this one's.
__device__ __forceinline__ int block_running_max(int v) {
  __shared__ int tops[kPlanThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(v, o);
    if (lane >= o && x > v) v = x;
  }
  __syncthreads();
  if (lane == 63) tops[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = tops[w] > v ? tops[w] : v;
  return v;
}

__global__ __launch_bounds__(kPlanThreads) void chunk_plan(const ChunkArgs a) {
  __shared__ unsigned long long pages;
  const int tid = threadIdx.x;
  if (tid == 0) pages = 0ull;
  for (int b0 = 0, top = 0; b0 <= a.c.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int s = b <= a.c.B ? a.starts[b] : 0;
    s = s < top ? top : s;
    s = s > a.N ? a.N : s;
    s = block_running_max(s);
    if (b <= a.c.B) a.begin[b] = s;
    __syncthreads();
    top = a.begin[b0 + kPlanThreads - 1 < a.c.B ? b0 + kPlanThreads - 1 : a.c.B];
  }
  const auto tiles_of = [&](int T) { return static_cast<int>((static_cast<int64_t>(T) * a.G + kTile - 1) / kTile); };
  int tiles = 0;
  for (int b0 = 0; b0 < a.c.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int all;
    const int at = block_scan(b < a.c.B ? tiles_of(a.begin[b + 1] - a.begin[b]) : 0, &all);
    if (b < a.c.B) a.offset[b] = tiles + at;
    tiles += all;
  }
  __syncthreads();
  const auto find = [&](int i, Share* s) {  // the sequence and tile of tile i, and its pages
    int lo = 0, hi = a.c.B - 1;             // the last sequence whose offset is i or less
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (a.offset[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    s->b = lo;
    s->first = a.begin[lo];
    s->T = a.begin[lo + 1] - s->first;
    s->tile = tiles_of(s->T) - 1 - (i - a.offset[lo]);
    return view_of(a, kv_len(a.c, lo), s->T, s->tile).pages();
  };
  Share s;
  unsigned long long mine = 0ull;
  for (int i = tid; i < tiles; i += kPlanThreads) mine += find(i, &s);
  atomicAdd(&pages, mine);
  __syncthreads();
  const unsigned long long even = (pages * a.c.Hk + 2 * kSlots - 1) / (2 * kSlots);
  const int most = static_cast<int>(even < kLeast ? kLeast : (even < 0x7FFFFFFFull ? even : 0x7FFFFFFFull));
  int shares = 0, parts = 0, splits = 0;
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid, n = i < tiles ? find(i, &s) : 0;
    const int k = i < tiles ? (n > most ? (n - 1) / most + 1 : 1) : 0;
    int all, all_parts, all_splits;
    const int at = shares + block_scan(k, &all), part = parts + block_scan(k > 1 ? k : 0, &all_parts);
    const int split = splits + block_scan(k > 1 ? 1 : 0, &all_splits);
    for (int j = 0; j < k; ++j) {
      s.v0 = static_cast<int>(static_cast<int64_t>(n) * j / k);
      s.v1 = static_cast<int>(static_cast<int64_t>(n) * (j + 1) / k);
      s.part = k > 1 ? part + j : -1;
      a.share[at + j] = s;
    }
    if (k > 1) a.split[split] = Split{s.first, s.T, s.tile, part, k};
    shares += all;
    parts += all_parts;
    splits += all_splits;
  }
  if (tid == 0) {
    a.counts[0] = shares;
    a.counts[1] = splits;
  }
}

// ---- the attention ------------------------------------------------------------
__device__ __forceinline__ uint32_t bits_of(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

__device__ __forceinline__ float max_over_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// fp16 of a page: keys by token, values by position (position c * D/16 + j in row 16 j + c).
// Rows are 16 bytes off the banks' period, so that 16 lanes' pieces of 16 neighbouring rows meet all banks.
template <int D>
struct alignas(16) Tile {
  static constexpr int kKeyRow = D + 8, kValueRow = kPage + 8;
  _Float16 k[kPage * kKeyRow];
  _Float16 v[D * kValueRow];
  uint32_t bad[kPage];  // groups of 16 positions of a token that are NaN and were made 0,
  uint32_t any[4];      // where a tile of 16 tokens has one
};

// A thread's part of a page: of tile p of 16 tokens, lane l of the first four
// wavefronts has keys (token l % 16, quarter l / 16 of the positions), of the
// others values (tokens 4 (l / 16) .. + 3, positions (l % 16) D/16 ..).
template <int D>
__device__ __forceinline__ const uint8_t* part_codes(const uint8_t* block, bool value, int p, int lane) {
  return block + (value ? KvBlock<D>::kVCodes : 0) + (p * (D / 8) / 16) * 1024 + lane * 16 + p * (D / 8) % 16;
}
template <int D>
__device__ __forceinline__ const uint8_t* part_scales(const uint8_t* block, bool value, int p, int lane) {
  return block + (value ? KvBlock<D>::kVScales + ((lane & 15) * D / 256) * 64 + (lane >> 4) * 16 + p * 4
                        : KvBlock<D>::kKScales + lane * (D / 16) + p * (D / 64));
}

template <int D>
struct Raw {
  uint32_t w[D / 32];
  uint32_t scale;
  __device__ __forceinline__ void load(const uint8_t* block, bool value, int p, int lane) {
    const uint8_t* s = part_codes<D>(block, value, p, lane);
    if constexpr (D == 64) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(s);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(s + i * 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
    const uint8_t* f = part_scales<D>(block, value, p, lane);
    if (value || D == 256) scale = *reinterpret_cast<const uint32_t*>(f);
    else if (D == 128) scale = *reinterpret_cast<const uint16_t*>(f);
    else scale = *f;
  }
};

// With the widest heads the next page's codes wait in LDS, each wavefront's own
// apart: there are no registers for them beside the sums.
struct Waiting {
  u32x4 codes[kWaves][2][64];
  uint32_t scale[kWaves][64];
  __device__ __forceinline__ void load(const uint8_t* block, int wave, bool value, int p, int lane) {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));  // what was here has been read
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_global_load_lds(part_codes<256>(block, value, p, lane) + i * 1024, &codes[wave][i][0], 16, 0, 0);
    __builtin_amdgcn_global_load_lds(part_scales<256>(block, value, p, lane), &scale[wave][0], 4, 0, 0);
  }
  __device__ __forceinline__ Raw<256> arrived(int wave, int lane) const {
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
    asm volatile("" ::: "memory");
    Raw<256> r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4 v = codes[wave][i][lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) r.w[4 * i + j] = v[j];
    }
    r.scale = scale[wave][lane];
    return r;
  }
};

template <int B>
__device__ __forceinline__ f16x2 e2m1_of(uint32_t w) { return e2m1x2<B>(w); }
__device__ __forceinline__ f16x2 e2m1_byte(uint32_t w, int b) {  // b: a constant after unrolling
  return b == 0 ? e2m1_of<0>(w) : b == 1 ? e2m1_of<1>(w) : b == 2 ? e2m1_of<2>(w) : e2m1_of<3>(w);
}

template <int D>
__device__ __forceinline__ void widen_keys(const Raw<D>& r, Tile<D>* to, int p, int lane) {
  _Float16* row = to->k + (16 * p + (lane & 15)) * Tile<D>::kKeyRow + (lane >> 4) * (D / 4);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const f16x2 pair = i / 4 ? e4m3x2<true>(r.scale) : e4m3x2<false>(r.scale);
    const _Float16 s = pair[i / 2 % 2];
    *reinterpret_cast<f16x8*>(row + 8 * i) = e2m1x8(r.w[i]) * f16x8{s, s, s, s, s, s, s, s};
  }
}

template <int D>
__device__ __forceinline__ void widen_values(const Raw<D>& r, uint32_t scale, Tile<D>* to, int p, int lane) {
  constexpr uint32_t kLow = 0x0F0F0F0Fu;
  _Float16* col = to->v + (lane & 15) * Tile<D>::kValueRow + 16 * p + 4 * (lane >> 4);
  const f16x2 s0 = e4m3x2<false>(scale), s1 = e4m3x2<true>(scale);
#pragma unroll
  for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
    u32x2 pair[2];  // codes of two tokens, one byte per position: even positions in .x, odd ones in .y
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (D == 64) {
        pair[i] = u32x2{bits_of(kLow, r.w[i], r.w[i] >> 12), bits_of(kLow, r.w[i] >> 4, r.w[i] >> 16)};
      } else {
        const uint32_t a = r.w[2 * i * (D / 128) + half], b = r.w[(2 * i + 1) * (D / 128) + half];
        pair[i] = u32x2{bits_of(kLow, a, b << 4), bits_of(kLow, a >> 4, b)};
      }
    }
#pragma unroll
    for (int j = 0; j < (D == 64 ? 4 : 8); ++j) {
      const f16x2 x = e2m1_byte(j % 2 ? pair[0].y : pair[0].x, j / 2) * s0, y = e2m1_byte(j % 2 ? pair[1].y : pair[1].x, j / 2) * s1;
      *reinterpret_cast<f16x4*>(col + (half * 8 + j) * 16 * Tile<D>::kValueRow) = f16x4{x.x, x.y, y.x, y.y};
    }
  }
}

// Of a page that some row does not see whole, or that is none, NaN values become 0
// and are noted: a weight of 0 must not carry them to the rows that do not see them.
template <int D>
__device__ __forceinline__ uint32_t note_bad(uint32_t scale, Tile<D>* to, int p, int lane) {
  const uint32_t wrong = ((scale & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  const bool any = __any(wrong != 0u);
  to->any[p] = any;
  if (any) {
    if (lane < 16) to->bad[16 * p + lane] = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((wrong >> (8 * i + 7)) & 1u) {
        scale &= ~(0xFFu << (8 * i));
        atomicOr(&to->bad[16 * p + 4 * (lane >> 4) + i], 1u << ((lane & 15) * D / 256));
      }
  }
  return scale;
}

// A barrier for what went to LDS; loads of the next page stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(63, 0));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// A wavefront's rows, or its part of them where the tile is split.
template <int D, class E>
__device__ __forceinline__ void store_rows(const ChunkArgs& a, int lane, int wave, int h, int row0, int R, int tile, int part, float m, float l,
                                           f32x16 (&o)[D / 32]) {
  const int half = lane >> 5, local = wave * 32 + (lane & 31), r = tile * kTile + local;
  const float total = sum_over_halves(l);
  const float inv = part >= 0 ? 1.0f : (m == -INFINITY ? 0.0f : a.c.gv / total);
  if (r >= R) return;
  const size_t at_part = (static_cast<size_t>(h) * a.parts + part) * kTile + local;
  const size_t at_row = static_cast<size_t>(row0 + r / a.G) * a.Hq + h * a.G + r % a.G;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // Positions c * D/16 .. of this lane.
      const int c = 8 * g + 4 * half + i;
      float x[D / 16];
#pragma unroll
      for (int j = 0; j < D / 16; ++j) x[j] = o[j / 2][8 * (j % 2) + 4 * g + i] * inv;
      if (part >= 0) {
#pragma unroll
        for (int j = 0; j < D / 16; j += 4)
          *reinterpret_cast<f32x4*>(a.part + at_part * D + c * (D / 16) + j) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]};
      } else {
        uint16_t* dst = static_cast<uint16_t*>(a.out) + at_row * D + c * (D / 16);
#pragma unroll
        for (int j = 0; j < D / 16; j += 4)
          *reinterpret_cast<u32x2*>(dst + j) = u32x2{elem_pack<E>(x[j], x[j + 1]), elem_pack<E>(x[j + 2], x[j + 3])};
      }
    }
  if (half == 0) {
    if (part >= 0) {
      a.stat[at_part * 2] = m;
      a.stat[at_part * 2 + 1] = total;
    } else if (a.lse) {
      a.lse[at_row] = m == -INFINITY && total == 0.0f ? -INFINITY : (m - kLift + __builtin_amdgcn_logf(total)) * kLn2;
    }
  }
}

template <int D>
constexpr int chunk_waves() { return 2; }  // per SIMD

template <int D, class E>
__global__ __launch_bounds__(kThreads, chunk_waves<D>()) void chunk(const ChunkArgs a) {
  constexpr int kSteps = D / 16, DB = D / 32;
  constexpr int kGroup = D == 256 ? 1 : 2;  // tiles of 32 tokens at a time: the widest heads leave registers for one
  constexpr bool kWaits = D == 256;
  constexpr int kProducts = kGroup * (kSteps + 2 * DB), kAhead = D == 256 ? 3 : 6;
  __shared__ __align__(16) std::conditional_t<kWaits, Waiting, int> waiting;
  __shared__ __align__(16) Tile<D> tiles[2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int at = static_cast<int>(blockIdx.x) / a.c.Hk, h = static_cast<int>(blockIdx.x) % a.c.Hk;
  if (at >= uniform_load(a.counts, 0)) return;
  const int32_t* words = reinterpret_cast<const int32_t*>(a.share + at);
  const int b = uniform_load(words, 0), row0 = uniform_load(words, 1), T = uniform_load(words, 2), tile = uniform_load(words, 3),
            v0 = uniform_load(words, 4), v1 = uniform_load(words, 5), part = uniform_load(words, 6);
  const int len = kv_len_uniform(a.c, b), R = T * a.G;  // at most N * G, which an int holds
  const View view = view_of(a, len, T, tile);
  const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.width;

  // This lane's row, and what the tile's, the wavefront's and its own rows see.
  const int wave_row = tile * kTile + wave * 32, r = wave_row + col;
  const auto limit_at = [&](int row) { return limit_of(len, T, row / a.G); };
  const bool busy = wave_row < R;
  const int last = tile * kTile + kTile < R ? tile * kTile + kTile - 1 : R - 1, wave_last = wave_row + 31 < R ? wave_row + 31 : R - 1;
  const int tile_least = limit_at(tile * kTile), tile_most = limit_at(last);
  const int wave_least = busy ? limit_at(wave_row) : 0, wave_most = busy ? limit_at(wave_last) : 0;
  const int limit = r < R ? limit_at(r) : 0;
  // Whether rows with limits from `least` to `most` all see the whole page from slot `first` on.
  const auto whole = [&](int first, int least, int most) {
    return first + kPage <= least && (!a.window || first >= most - a.window || first + kPage <= a.sinks);
  };

  f16x8 q[kSteps];
  float cm;
  {
    const int token = r < R ? r / a.G : 0, hq = r < R ? h * a.G + r % a.G : 0;
    const uint16_t* src = a.q + static_cast<int64_t>(row0 + token) * a.row + hq * a.head + 8 * half;
    u32x4 w[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) w[s] = r < R ? *reinterpret_cast<const u32x4*>(src + 16 * s) : u32x4{0u, 0u, 0u, 0u};
    float factor = 1.0f;
    if constexpr (std::is_same_v<E, BF16>) {
      // To fp16's range by the power of two that brings the row's greatest value to 2^14 .. 2^15:
      // values down to 2^-31 of it keep all their bits, the rest is off by 2^-39 of it at most.
      float amax = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = fabsf(elem_lo<E>(w[s][j])), hi = fabsf(elem_hi<E>(w[s][j]));
          amax = lo < INFINITY ? fmaxf(amax, lo) : amax;
          amax = hi < INFINITY ? fmaxf(amax, hi) : amax;
        }
      amax = max_over_halves(amax);
      int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      ex = ex < -100 ? -100 : ex;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[s][j] = elem_pack<F16>(ldexpf(elem_lo<E>(w[s][j]), 14 - ex), ldexpf(elem_hi<E>(w[s][j]), 14 - ex));
      factor = ldexpf(1.0f, ex - 14);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = __builtin_bit_cast(f16x8, w[s]);
    cm = fmaxf(a.scale * a.c.gk * kLog2e * factor, kMinNormal);
    // The loop must not wait for these again, and with them for the next page.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
  }
  float m = -INFINITY, l = 0.0f;
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};

  // Thread's part of every page; a page that the table does not name is read as page 0 and seen by nobody.
  const bool value = wave >= 4;
  const int p = wave & 3;
  Raw<D> raw;
  // The lane, found again for each page where the addresses made of it would take registers all the while.
  const auto here = [&] {
    int l = lane;
    if constexpr (kWaits) asm volatile("" : "+v"(l));
    return l;
  };
  const auto named = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(a.c.pages); };
  const auto page_id = [&](int v) { return uniform_load(table, view.page(v < v1 ? v : v1 - 1)); };
  const auto load = [&](int id) {
    const uint8_t* block = static_cast<const uint8_t*>(a.c.data) + (static_cast<size_t>(named(id) ? id : 0) * a.c.Hk + h) * KvBlock<D>::kBytes;
    if constexpr (kWaits) waiting.load(block, wave, value, p, here());
    else raw.load(block, value, p, lane);
  };
  const auto widen = [&](Tile<D>* to, int v, int id) {
    const int lane = here();
    if constexpr (kWaits) raw = waiting.arrived(wave, lane);
    if (value) {
      uint32_t s = raw.scale;
      if (!named(id) || !whole(view.page(v) * kPage, tile_least, tile_most)) s = note_bad<D>(s, to, p, lane);
      widen_values<D>(raw, s, to, p, lane);
    } else {
      widen_keys<D>(raw, to, p, lane);
    }
  };
  int id = 0, next_id = 0, after_id = 0;  // of pages v, v + 1, v + 2
  if (v0 < v1) {
    // The first products are of no weights with the values of no page.
    for (int i = threadIdx.x; i < D * Tile<D>::kValueRow / 8; i += kThreads) *reinterpret_cast<u32x4*>(tiles[1].v + 8 * i) = u32x4{0u, 0u, 0u, 0u};
    id = page_id(v0);
    next_id = page_id(v0 + 1);
    load(id);
    widen(&tiles[0], v0, id);
    load(next_id);
    after_id = page_id(v0 + 2);
  }
  lds_barrier();
  if (value) lds_barrier();

  const int key_row = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
  f16x8 w[2 * kGroup];  // weights of the tokens before: none yet
#pragma unroll
  for (int i = 0; i < 2 * kGroup; ++i) w[i] = f16x8{};
  int flagged = -1;      // the first slot of the page before, where it has NaN values that were noted
  const auto add_values = [&](const Tile<D>& of, int u0) {
#pragma unroll
    for (int step = 0; step < 2 * kGroup; ++step)
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const f16x8 x = *reinterpret_cast<const f16x8*>(of.v + (32 * d + col) * Tile<D>::kValueRow + 32 * u0 + 16 * step + 8 * half);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, w[step], o[d], 0, 0, 0);
      }
  };
  const auto add_scores = [&](const Tile<D>& of, int u0, f32x16 (&s)[kGroup]) {
#pragma unroll
    for (int u = 0; u < kGroup; ++u) s[u] = f32x16{};
#pragma unroll
    for (int step = 0; step < kSteps; ++step)
#pragma unroll
      for (int u = 0; u < kGroup; ++u) {
        const f16x8 k = *reinterpret_cast<const f16x8*>(of.k + (32 * (u0 + u) + key_row) * Tile<D>::kKeyRow + 16 * step + 8 * half);
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[step], s[u], 0, 0, 0);
      }
  };
  // The rows that see a NaN value have it by hand.
  const auto add_bad = [&](const Tile<D>& of) {
    for (int t = 0; t < kPage; ++t) {
      const uint32_t groups = of.any[t / 16] ? of.bad[t] : 0u;
      const int slot = flagged + t;
      if (groups && slot < limit && (!a.window || slot >= limit - a.window || slot < a.sinks)) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = 32 * d + 8 * (e / 4) + 4 * half + e % 4, position = (row % 16) * (D / 16) + row / 16;
            if ((groups >> (position / 16)) & 1u) o[d][e] = NAN;
          }
      }
    }
  };
  for (int v = v0; v < v1; ++v) {
    const Tile<D>&now = tiles[(v - v0) & 1], &other = tiles[(v + 1 - v0) & 1];
    const int first = view.page(v) * kPage;
    const bool seen = named(id);
    const bool work = busy && seen && first < wave_most && (!a.window || first + kPage > wave_least - a.window || first < a.sinks);
    const bool partial = work && !whole(first, wave_least, wave_most);
#pragma unroll
    for (int u0 = 0; u0 < 2; u0 += kGroup) {
      f32x16 s[kGroup];
      const Tile<D>& before = u0 ? now : other;
      const int before_u0 = u0 ? u0 - kGroup : 2 - kGroup;
      if (busy) {
        add_values(before, before_u0);
        add_scores(now, u0, s);
        // The operands are read kAhead products before they are used: left to itself the compiler reads two,
        // waits for them, and pays LDS's latency sixteen times.
        __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
        for (int i = 0; i < kProducts - kAhead; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
      }
      if (u0 == 0 && flagged >= 0) add_bad(other);
      lds_barrier();
      if (work) {
        if (partial) {
          const int low = a.window ? limit - a.window : 0;
#pragma unroll
          for (int u = 0; u < kGroup; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int slot = first + 32 * (u0 + u) + 16 * (e / 8) + 8 * half + e % 8;
              const bool out = (slot >= limit) | ((slot < low) & (slot >= a.sinks));
              s[u][e] = out ? -INFINITY : s[u][e];
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, s[u][e]);
        top = max_over_halves(top) * cm;
        const bool up = top > m + kSlack;
        if (__any(up)) {
          const float to = up ? top : m;
          const float alpha = up ? __builtin_amdgcn_exp2f(m - to) : 1.0f;
          m = to;
          l *= alpha;
#pragma unroll
          for (int d = 0; d < DB; ++d) o[d] *= alpha;
        }
        const float lifted = m == -INFINITY ? 0.0f : m - kLift;
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], cm, -lifted));
            l += x;
            w[2 * u + e / 8][e % 8] = static_cast<_Float16>(x);
          }
      } else {
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) w[i] = f16x8{};
      }
      if (u0 == 0 && v + 1 < v1) {
        widen(&tiles[(v + 1 - v0) & 1], v + 1, next_id);
        load(after_id);
      }
      lds_barrier();
    }
    flagged = -1;
    if (seen && !whole(first, tile_least, tile_most) && (now.any[0] | now.any[1] | now.any[2] | now.any[3])) flagged = first;
    id = next_id;
    next_id = after_id;
    after_id = page_id(v + 3);
  }
  if (busy && v0 < v1) add_values(tiles[(v1 - 1 - v0) & 1], 2 - kGroup);
  if (flagged >= 0) add_bad(tiles[(v1 - 1 - v0) & 1]);
  if (!value) lds_barrier();
  store_rows<D, E>(a, here(), wave, h, row0, R, tile, part, m, l, o);
}

// Adds the shares of split tiles: D / 4 threads have a row, eight shares' loads at a time.
template <int D, class E>
__global__ __launch_bounds__(256) void chunk_join(const ChunkArgs a) {
  constexpr int kPer = D / 4, kRows = 256 / kPer, kBatch = 8;
  const int at = static_cast<int>(blockIdx.x) / a.c.Hk, h = static_cast<int>(blockIdx.x) % a.c.Hk;
  if (at >= uniform_load(a.counts, 1)) return;
  const Split sp = a.split[at];
  const int local = blockIdx.y * kRows + threadIdx.x / kPer, r = sp.tile * kTile + local, pos = threadIdx.x % kPer * 4;
  if (r >= sp.T * a.G) return;
  float mm = -INFINITY, total = 0.0f;
  f32x4 x{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < sp.shares; s0 += kBatch) {
    float2 st[kBatch];
    f32x4 v[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int share = s0 + s < sp.shares ? s0 + s : s0;
      const size_t p = (static_cast<size_t>(h) * a.parts + sp.part + share) * kTile + local;
      st[s] = *reinterpret_cast<const float2*>(a.stat + p * 2);
      v[s] = *reinterpret_cast<const f32x4*>(a.part + p * D + pos);
    }
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < sp.shares) {
        // A share without weight is zeros; one with nothing but NaN scores has the same
        // maximum, -inf, but a NaN sum: both are added, times 0.
        const float to = fmaxf(mm, st[s].x), about = to == -INFINITY ? 0.0f : to;
        const float f0 = __builtin_amdgcn_exp2f(mm - about), f = __builtin_amdgcn_exp2f(st[s].x - about);
        mm = to;
        total = total * f0 + f * st[s].y;
        x = x * f0 + f * v[s];
      }
  }
  const size_t at_row = static_cast<size_t>(sp.first + r / a.G) * a.Hq + h * a.G + r % a.G;
  x *= mm == -INFINITY ? 0.0f : a.c.gv / total;
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at_row * D + pos) = u32x2{elem_pack<E>(x[0], x[1]), elem_pack<E>(x[2], x[3])};
  if (pos == 0 && a.lse) a.lse[at_row] = mm == -INFINITY && total == 0.0f ? -INFINITY : (mm - kLift + __builtin_amdgcn_logf(total)) * kLn2;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

ChunkPlan kv4_chunk_plan(int N, int B, int Hq, int Hk, int D, int width, int window, int sinks) {
  ChunkPlan p;
  const int64_t G = Hq / Hk, busy = N < B ? N : B;  // sequences with rows
  p.tiles = (N * G + busy * (kTile - 1)) / kTile;
  // The pages that a tile can see: its rows' tokens, a window before the first of them, and the sinks.
  int64_t pages = width;
  if (window) {
    const int64_t tokens = (kTile - 1) / G + 2 < N ? (kTile - 1) / G + 2 : N;
    const int64_t seen = (window + tokens) / kPage + 2 + (static_cast<int64_t>(sinks) + kPage - 1) / kPage;
    pages = seen < pages ? seen : pages;
  }
  // A tile is split when it has more than `most` pages, of which there are 2 * kSlots / Hk
  // (and a part of one) among the pages of a head's tiles.
  const int64_t most = 2 * kSlots / Hk + 1;
  p.splits = pages > kLeast ? (p.tiles < most ? p.tiles : most) : 0;
  const int64_t each = p.splits * ((pages + kLeast - 1) / kLeast);
  p.parts = p.splits + most < each ? p.splits + most : each;
  p.shares = p.tiles + (p.parts > 0 ? p.parts : 0);
  p.counts_off = kSyncBytes;
  p.begin_off = p.counts_off + 256;
  p.offset_off = p.begin_off + up(static_cast<size_t>(B + 1) * 4);
  p.share_off = p.offset_off + up(static_cast<size_t>(B) * 4);
  p.split_off = p.share_off + up(static_cast<size_t>(p.shares) * sizeof(Share));
  p.stat_off = p.split_off + up(static_cast<size_t>(p.splits) * sizeof(Split));
  p.part_off = p.stat_off + static_cast<size_t>(Hk) * p.parts * kTile * 8;
  p.total = p.part_off + static_cast<size_t>(Hk) * p.parts * kTile * D * 4;
  return p;
}

hipError_t launch_kv4_chunk(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N, int type,
                            int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace, hipStream_t stream) {
  const ChunkPlan p = kv4_chunk_plan(N, c.B, Hq, c.Hk, c.D, c.width, window, sinks);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ChunkArgs a{c, static_cast<const uint16_t*>(q), row, head, starts, out, lse, reinterpret_cast<int*>(ws + p.counts_off),
                    reinterpret_cast<int*>(ws + p.begin_off), reinterpret_cast<int*>(ws + p.offset_off), reinterpret_cast<Share*>(ws + p.share_off),
                    reinterpret_cast<Split*>(ws + p.split_off), reinterpret_cast<float*>(ws + p.stat_off),
                    reinterpret_cast<float*>(ws + p.part_off), p.parts, N, Hq, Hq / c.Hk, static_cast<int>(p.tiles), window, sinks, scale};
  chunk_plan<<<1, kPlanThreads, 0, stream>>>(a);
  const auto run = [&](auto d, auto e) {
    chunk<d(), decltype(e)><<<dim3(static_cast<unsigned>(p.shares * c.Hk)), kThreads, 0, stream>>>(a);
    if (p.splits)
      chunk_join<d(), decltype(e)><<<dim3(static_cast<unsigned>(p.splits * c.Hk), kTile * d() / 1024), 256, 0, stream>>>(a);
  };
  const auto by_type = [&](auto d) {
    if (type == SKINNY_F16) run(d, F16());
    else run(d, BF16());
  };
  if (c.D == 64) by_type(std::integral_constant<int, 64>());
  else if (c.D == 128) by_type(std::integral_constant<int, 128>());
  else by_type(std::integral_constant<int, 256>());
  return hipGetLastError();
}

}  // namespace skinny
