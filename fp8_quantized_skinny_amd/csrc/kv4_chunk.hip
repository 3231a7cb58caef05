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
//
// Two wavefronts share a SIMD, and those of one half of the workgroup run a barrier
// behind the other's: one has the matrix unit for its products, between which it
// widens its part of the next page, while the other has the VALU for its softmax.
// Operands come from LDS, six products ahead of their use.  256 rows are what one
// workgroup a CU holds in registers (D = 128: 64 of sums, 32 of queries, 32 of
// scores a lane), and each row more shares the widening of a page, 42 to 64 VALU
// operations a lane and 36 KB of LDS writes.
//
// Bound by the matrix unit, the VALU and the power that both may draw: 8192 tokens,
// 48 + 4 heads of 128, 811 .. 861 us, 0.96 .. 1.02 PFLOP/s of seen products at
// about 1.8 GHz, where a large fp16 product reaches 1.0 PFLOP/s at first and 1.36
// when nothing else runs for long.  The matrix unit is busy for 53% of the cycles,
// the VALU for 58%, LDS for 37%.  Parts left out of the kernel of 852 us (for
// timing only): softmax 127 us, of which the exponentials 89; widening 92; operand
// reads 58; all but products and widening, 658 us are left.
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
constexpr int kSlots = 256;  // workgroups that the CUs hold at once
constexpr int kLeast = 16;   // fewest pages of a workgroup where tiles are cut
// Both in pages, whatever the head size (see the plan).
constexpr int kCutPages = 6;  // what the cut tiles' parts cost a workgroup: stored by it, and read by the join
constexpr int kBegin = 10;    // what a tile's beginning and end cost (less than kLeast)
constexpr int kPlanThreads = 256;
constexpr int kPlanHeld = 1024;  // sequences whose rows and tiles the plan keeps in LDS
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMinNormal = 0x1p-126f;
// Weights go to fp16 relative to a reference that follows the running maximum
// only when that rose by more than 2^kSlack, times 2^kLift (as in
// kv4_attention.hip): below 2^14, and exact to 2^-11 down to 2^-20 of the greatest.
constexpr float kLift = 6.0f, kSlack = 8.0f;

// A piece of the work: view pages v0 .. v1 of those that a tile's rows see.
struct Piece {
  int b, first, T, tile;  // sequence, its first row and number of them, tile of it
  int v0, v1;
  int part;               // its place among the parts of cut tiles, -1: it is the whole tile
  int pad;
};
struct Cut {              // a tile of several pieces
  int first, T, tile, part, pieces;
};

struct ChunkArgs {
  kv4_cache c;
  const uint16_t* q;
  int64_t row, head;    // strides of q
  const int32_t* starts;
  void* out;
  float* lse;
  int* counts;          // [2]: workgroups per head, cut tiles
  int* begin;           // [B + 1]: first row of each sequence
  int* offset;          // [B]: tiles before each sequence
  int* first;           // [workgroup + 1]: its first piece
  Piece* piece;
  Cut* cut;
  float* stat;          // [head][part][kTile][2]: reference maximum (log2) and sum
  float* part;          // [head][part][kTile * D] (see part_at)
  int64_t parts;        // per head
  int N, Hq, G;
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

// Which pages rows with limits from `least` to `most` see: all of them the whole
// of (each below end, and from begin on or below sinks), some of them something of.
struct Sight {
  int whole_begin, whole_end, whole_sinks, some_begin, some_end, some_sinks;
  __device__ __forceinline__ Sight(const ChunkArgs& a, int least, int most)
      : whole_begin(0), whole_end(least / kPage), whole_sinks(0), some_begin(0), some_end((most + kPage - 1) / kPage), some_sinks(0) {
    if (a.window) {
      const int last = most - a.window, first = least - a.window;  // where the latest and the earliest window begin
      whole_begin = last > 0 ? (last + kPage - 1) / kPage : 0;
      whole_sinks = a.sinks / kPage;
      some_begin = first > 0 ? first / kPage : 0;
      some_sinks = a.sinks / kPage + (a.sinks % kPage != 0);
    }
  }
  __device__ __forceinline__ bool whole(int page) const { return page < whole_end && (page >= whole_begin || page < whole_sinks); }
  __device__ __forceinline__ bool some(int page) const { return page < some_end && (page >= some_begin || page < some_sinks); }
};

// ---- the plan -----------------------------------------------------------------
// One workgroup lists the pieces of a head's work, the same for all heads.  Where
// there are many tiles, none of them long, a workgroup of the attention has a
// whole tile, the longest of a sequence, its last, first.  Otherwise the pages of
// all tiles in a row are dealt out evenly to as many workgroups as the CUs hold:
// each has the end of one tile, whole ones, and the beginning of another, and no
// CU waits for a last long tile (512 tokens over 120000, 24 tiles of 1883 pages a
// head: 1754 us with each tile in six equal shares, 1442 so).  A tile counts kBegin
// pages more than it has, or the workgroup with the shortest tiles, up to eleven of
// them, ends last.  Whole tiles are taken where they end kCutPages or less after the
// even shares.  Three draws each of 16 chunks of 1 .. 640 tokens over up to 9000, and
// of three of 1500 .. 4100 within 1024 (bf16, us); 14 chunks of 1286 take the same with
// all of these:
//   kBegin                0            5           10           14
//   28/4 heads of 64  238 247 272  223 210 222  219 207 208  222 209 213
//   32/8 of 128       365 385 424  337 358 359  329 346 349  336 358 347
//   24/4 of 256       552 573 650  507 531 531  514 536 531  521 556 527
//   kCutPages             0            6           12           24
//   28/4 heads of 64  153 155 158  153 155 158  147 151 151  147 151 152
//   32/8 of 128       243 259 260  243 260 260  242 260 260  244 260 260
//   24/4 of 256       329 339 336  330 337 336  348 371 371  349 372 371
//
// The rows of a sequence go from its start to the next one's; a start that is not
// in 0 .. N counts as the nearer of these, and one below an earlier start as that:
// no two sequences have a row in common, whatever the starts are.
constexpr int kPlanWaves = kPlanThreads / 64;

// Sums over the threads before this one, and over all, of each of N values.
template <class I, int N>
__device__ __forceinline__ void block_scan(I (&v)[N], I (&total)[N]) {
  __shared__ I sums[N][kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  I own[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    own[i] = v[i];
    for (int o = 1; o < 64; o <<= 1) {
      const I x = __shfl_up(v[i], o);
      if (lane >= o) v[i] += x;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 63) sums[i][wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = 0;
    v[i] -= own[i];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      v[i] += w < wave ? sums[i][w] : 0;
      total[i] += sums[i][w];
    }
  }
}

__host__ __device__ constexpr int slots_per_head(int Hk) { return kSlots / Hk > 1 ? kSlots / Hk : 1; }

// The greatest of the threads' values up to this one's, and of all.
__device__ __forceinline__ int block_running_max(int v, int* all) {
  __shared__ int tops[kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(v, o);
    if (lane >= o && x > v) v = x;
  }
  __syncthreads();
  if (lane == 63) tops[wave] = v;
  __syncthreads();
  int top = tops[0];
#pragma unroll
  for (int w = 1; w < kPlanWaves; ++w) top = tops[w] > top ? tops[w] : top;
  for (int w = 0; w < wave; ++w) v = tops[w] > v ? tops[w] : v;
  *all = top;
  return v;
}

__global__ __launch_bounds__(kPlanThreads) void chunk_plan(const ChunkArgs a) {
  __shared__ int held_begin[kPlanHeld + 1], held_offset[kPlanHeld], held_len[kPlanHeld];
  const int tid = threadIdx.x, B = a.c.B;
  const bool held = B <= kPlanHeld;
  for (int b0 = 0, top = 0; b0 <= B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int s = b <= B ? a.starts[b] : 0;
    if (held && b < B) held_len[b] = kv_len(a.c, b);
    s = s < top ? top : s;
    s = s > a.N ? a.N : s;
    s = block_running_max(s, &top);
    if (b <= B) (held ? held_begin[b] : a.begin[b]) = s;
  }
  __syncthreads();
  const auto begin_of = [&](int b) { return held ? held_begin[b] : a.begin[b]; };
  const auto tiles_of = [&](int T) { return static_cast<int>((static_cast<int64_t>(T) * a.G + kTile - 1) / kTile); };
  int tiles = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n[1] = {b < B ? tiles_of(begin_of(b + 1) - begin_of(b)) : 0}, all[1];
    block_scan(n, all);
    if (b < B) (held ? held_offset[b] : a.offset[b]) = tiles + n[0];
    tiles += all[0];
  }
  __syncthreads();
  const auto find = [&](int i, Piece* s) {  // the sequence and tile of tile i, and its pages
    int lo = 0, hi = B - 1;                 // the last sequence whose offset is i or less
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if ((held ? held_offset[mid] : a.offset[mid]) <= i) lo = mid;
      else hi = mid - 1;
    }
    s->b = lo;
    s->first = begin_of(lo);
    s->T = begin_of(lo + 1) - s->first;
    s->tile = tiles_of(s->T) - 1 - (i - (held ? held_offset[lo] : a.offset[lo]));
    return view_of(a, held ? held_len[lo] : kv_len(a.c, lo), s->T, s->tile).pages();
  };
  // A tile whose rows see nothing counts as one page; its beginning and end as kBegin, before its pages.
  Piece s{};
  long long pages = 0, before[1] = {0};  // of all tiles; of those before the thread's last
  int longest = 0, n = 0;
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    n = i < tiles ? find(i, &s) : 0;
    int top;
    block_running_max(n, &top);
    longest = top > longest ? top : longest;
    long long all[1];
    before[0] = i < tiles ? (n ? n : 1) + kBegin : 0;
    block_scan(before, all);
    before[0] += pages;
    pages += all[0];
  }
  const long long slots = slots_per_head(a.c.Hk);
  const long long even = (pages + slots - 1) / slots, each = even < kLeast ? kLeast : even;
  // Whole tiles: in rounds of the longest, or with the longest of them last.
  const long long rounds = (tiles + slots - 1) / slots * (longest + kBegin), last = even + longest / 2;
  const bool whole = slots < 4 || (static_cast<long long>(tiles) >= 4 * slots && longest * 2 * slots <= pages) ||
                     (rounds < last ? rounds : last) <= even + kCutPages;
  int pieces = 0, parts = 0, cuts = 0;
  long long done = 0;
  for (int i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int i = i0 + tid;
    if (whole) {
      if (i < tiles) {
        s.v1 = find(i, &s);
        s.v0 = 0;
        s.part = -1;
        a.piece[i] = s;
        a.first[i] = i;
      }
      continue;
    }
    if (tiles > kPlanThreads) {  // otherwise known from before
      n = i < tiles ? find(i, &s) : 0;
      long long all[1];
      before[0] = i < tiles ? (n ? n : 1) + kBegin : 0;
      block_scan(before, all);
      before[0] += done;
      done += all[0];
    }
    const long long p0 = before[0] + kBegin, p1 = p0 + (n ? n : 1);  // its pages in the row of all
    // Its workgroups; in 32 bits wherever the pages are counted in those, which a division takes a tenth of the time for.
    const bool few = pages <= 0x7FFFFFFF;
    const long long j0 = few ? static_cast<uint32_t>(p0) / static_cast<uint32_t>(each) : p0 / each;
    const long long j1 = few ? static_cast<uint32_t>(p1 - 1) / static_cast<uint32_t>(each) : (p1 - 1) / each;
    const int k = i < tiles ? static_cast<int>(j1 - j0) + 1 : 0;
    int at[3] = {k, k > 1 ? k : 0, k > 1 ? 1 : 0}, all[3];
    block_scan(at, all);
    for (int j = 0; j < k; ++j) {
      const long long from = (j0 + j) * each, to = from + each;
      s.v0 = j ? static_cast<int>(from - p0) : 0;
      s.v1 = j + 1 < k ? static_cast<int>(to - p0) : n;
      s.part = k > 1 ? parts + at[1] + j : -1;
      a.piece[pieces + at[0] + j] = s;
      if (from >= before[0]) a.first[j0 + j] = pieces + at[0] + j;
    }
    if (k > 1) a.cut[cuts + at[2]] = Cut{s.first, s.T, s.tile, parts + at[1], k};
    pieces += all[0];
    parts += all[1];
    cuts += all[2];
  }
  if (tid == 0) {
    const int groups = whole ? tiles : static_cast<int>((pages + each - 1) / each);
    a.first[groups] = whole ? tiles : pieces;
    a.counts[0] = groups;
    a.counts[1] = cuts;
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

// A thread's part of a page.  Wavefront 2 p + half has half of tile p of 16
// tokens: lane l has, of the keys, of token l % 16 a half of quarter l / 16 of the
// positions, D/16 bytes of codes that lie together; of the values, of tokens
// 4 (l / 16) .. + 3 the even or the odd ones of the positions (l % 16) D/16 ..,
// half of D/8 bytes that the other wavefront loads as well: four tokens at a time
// go to LDS in half of the stores that two do.
template <int D>
__device__ __forceinline__ uint32_t key_code_at(int wave, int lane) {
  const int run = wave * (D / 16);  // of the bytes of a lane
  return run / 16 * 1024 + lane * 16 + run % 16;
}
template <int D>
__device__ __forceinline__ uint32_t value_code_at(int wave, int lane) {
  const int run = (wave >> 1) * (D / 8);
  return KvBlock<D>::kVCodes + run / 16 * 1024 + lane * 16 + run % 16;
}
// The four E4M3 scales of the values, and the one or, with the widest heads, two of the keys.
template <int D>
__device__ __forceinline__ uint32_t value_scale_at(int wave, int lane) {
  return KvBlock<D>::kVScales + ((lane & 15) * D / 256) * 64 + (lane >> 4) * 16 + (wave >> 1) * 4;
}
// (Loaded by dwords: of bytes the compiler clears the upper bits as soon as they are there, and waits for that.)
template <int D>
__device__ __forceinline__ uint32_t key_scale_at(int wave, int lane) {
  return KvBlock<D>::kKScales + lane * (D / 16) + (wave * D / 128 & ~3);
}
template <int D>
__device__ __forceinline__ int key_scale_shift(int wave) { return (wave * D / 128 & 3) * 8; }

template <int D>
struct Raw {
  uint32_t k[D / 64], v[D / 32], key_scale, value_scale;
  __device__ __forceinline__ void load_keys(const uint8_t* block, int wave, int lane) {
    const uint8_t* c = block + key_code_at<D>(wave, lane);
    if constexpr (D == 64) {
      k[0] = *reinterpret_cast<const uint32_t*>(c);
    } else {
      const u32x2 x = *reinterpret_cast<const u32x2*>(c);
      k[0] = x.x;
      k[1] = x.y;
    }
    key_scale = *reinterpret_cast<const uint32_t*>(block + key_scale_at<D>(wave, lane));
  }
  __device__ __forceinline__ void load_values(const uint8_t* block, int wave, int lane) {
    const uint8_t* c = block + value_code_at<D>(wave, lane);
    if constexpr (D == 64) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(c);
      v[0] = x.x;
      v[1] = x.y;
    } else {
      const u32x4 x = *reinterpret_cast<const u32x4*>(c);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = x[j];
    }
    value_scale = *reinterpret_cast<const uint32_t*>(block + value_scale_at<D>(wave, lane));
  }
};

// With the widest heads the next codes wait in LDS: there are no registers for
// them beside the sums.  The two wavefronts of a tile load one half of its values
// each, so what they wait for has to lie before a barrier (see the loop).
struct Waiting {
  u32x4 keys[kWaves][64], values[kWaves][64];
  uint32_t key_scale[kWaves][64], value_scale[kWaves / 2][64];
  __device__ __forceinline__ void load(const uint8_t* key_block, const uint8_t* value_block, int wave, int lane) {
    __builtin_amdgcn_global_load_lds(key_block + key_code_at<256>(wave, lane), &keys[wave][0], 16, 0, 0);
    __builtin_amdgcn_global_load_lds(key_block + key_scale_at<256>(wave, lane), &key_scale[wave][0], 4, 0, 0);
    __builtin_amdgcn_global_load_lds(value_block + (value_code_at<256>(wave, lane) + (wave & 1) * 1024), &values[wave][0], 16, 0, 0);
    __builtin_amdgcn_global_load_lds(value_block + value_scale_at<256>(wave, lane), &value_scale[wave >> 1][0], 4, 0, 0);
  }
  __device__ __forceinline__ void arrived(Raw<256>* r, int wave, int lane) const {
    const u32x4 k = keys[wave][lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) r->k[j] = k[j];
    r->key_scale = key_scale[wave][lane];
    r->value_scale = value_scale[wave >> 1][lane];
  }
  // Of the values the words for the first or the second eight positions.
  __device__ __forceinline__ void arrived_values(Raw<256>* r, int half, int wave, int lane) const {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&values[t ? wave | 1 : wave & ~1][lane]);
      r->v[4 * t + half] = w[half];
      r->v[4 * t + 2 + half] = w[2 + half];
    }
  }
};

// Piece i of the widening of a thread's keys: eight positions.
template <int D>
__device__ __forceinline__ void widen_keys(const Raw<D>& r, _Float16* row, int wave, int i) {
  const _Float16 s = e4m3x2<false>(r.key_scale >> key_scale_shift<D>(wave))[i / 2];
  *reinterpret_cast<f16x8*>(row + 8 * i) = e2m1x8(r.k[i]) * f16x8{s, s, s, s, s, s, s, s};
}
template <int D>
__device__ __forceinline__ _Float16* key_row_of(Tile<D>* to, int wave, int lane) {
  return to->k + (16 * (wave >> 1) + (lane & 15)) * Tile<D>::kKeyRow + (lane >> 4) * (D / 4) + (wave & 1) * (D / 8);
}

// Piece i of its values: position 2 i or 2 i + 1 of the D/16, four tokens.
template <int D>
__device__ __forceinline__ void widen_values(const Raw<D>& r, _Float16* column, int wave, int i) {
  const int odd = 4 * (wave & 1);
  f16x2 x[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    // Codes of two tokens, one byte for each of the positions.
    const uint32_t a = r.v[D == 64 ? t : 2 * t * (D / 128) + i / 4];
    const uint32_t b = D == 64 ? a >> 16 : r.v[D == 64 ? 0 : (2 * t + 1) * (D / 128) + i / 4];
    const uint32_t pair = bits_of(0x0F0F0F0Fu, a >> odd, b << (4 - odd));
    const int at = i % 4;
    const f16x2 c = at == 0 ? e2m1x2<0>(pair) : at == 1 ? e2m1x2<1>(pair) : at == 2 ? e2m1x2<2>(pair) : e2m1x2<3>(pair);
    x[t] = c * (t ? e4m3x2<true>(r.value_scale) : e4m3x2<false>(r.value_scale));
  }
  *reinterpret_cast<f16x4*>(column + i * 32 * Tile<D>::kValueRow) = f16x4{x[0].x, x[0].y, x[1].x, x[1].y};
}
template <int D>
__device__ __forceinline__ _Float16* value_column_of(Tile<D>* to, int wave, int lane) {
  return to->v + ((lane & 15) + 16 * (wave & 1)) * Tile<D>::kValueRow + 16 * (wave >> 1) + 4 * (lane >> 4);
}

// Of a page that some row does not see whole, or that is none, NaN values become 0
// and are noted: a weight of 0 must not carry them to the rows that do not see them.
template <int D>
__device__ __forceinline__ void note_bad(Raw<D>* r, Tile<D>* to, int wave, int lane) {
  const uint32_t wrong = ((r->value_scale & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  r->value_scale &= ~(wrong | (wrong - (wrong >> 7)));
  if (wave & 1) return;  // the other wavefront of the tile sees the same
  const int p = wave >> 1;
  const bool any = __any(wrong != 0u);
  to->any[p] = any;
  if (any) {
    if (lane < 16) to->bad[16 * p + lane] = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((wrong >> (8 * i + 7)) & 1u) atomicOr(&to->bad[16 * p + 4 * (lane >> 4) + i], 1u << ((lane & 15) * D / 256));
  }
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

// Where the parts of a cut tile lie: as the wavefronts hold them, so that 64 lanes store and load 1024 bytes in a row.
// Unit wave * 8 + i: the wavefront's lanes have row lane % 32, positions c * D/16 .. for c = first_position(i, lane / 32).
__device__ __forceinline__ int first_position(int i, int half) { return 8 * (i / 4) + 4 * half + i % 4; }
template <int D>
__device__ __forceinline__ size_t part_at(size_t part, int unit, int quarter, int lane) {
  return part * (kTile * D) + static_cast<size_t>(((unit * (D / 64) + quarter) * 64 + lane) * 4);
}
template <int D>
constexpr int kStageRow = 2 * D + 16;  // bytes: rows are 16 off the banks' period

// A wavefront's rows, or its part of them where the tile is split.  Whole rows go through LDS to be stored 1024 bytes at
// a time; from the lanes' own positions every store meets 32 rows (D = 256, 202 tiles a head: 372 against 368 us).
template <int D, class E>
__device__ __forceinline__ void store_rows(const ChunkArgs& a, int lane, int wave, int h, int row0, int R, int tile, int part, float m, float l,
                                           uint32_t nan_groups, f32x16 (&o)[D / 32], uint8_t* stage) {
  const int half = lane >> 5, local = wave * 32 + (lane & 31), r = tile * kTile + local;
  const float total = sum_over_halves(l);
  const float inv = part >= 0 ? 1.0f : (m == -INFINITY ? 0.0f : a.c.gv / total);
  const size_t at_part = static_cast<size_t>(h) * a.parts + part;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = first_position(i, half);
    float x[D / 16];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) x[j] = (nan_groups >> (c * D / 256)) & 1u ? NAN : o[j / 2][8 * (j % 2) + i] * inv;
    if (part >= 0) {
      if (r < R) {
#pragma unroll
        for (int j = 0; j < D / 16; j += 4)
          *reinterpret_cast<f32x4*>(a.part + part_at<D>(at_part, wave * 8 + i, j / 4, lane)) = f32x4{x[j], x[j + 1], x[j + 2], x[j + 3]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < D / 16; j += 4)
        *reinterpret_cast<u32x2*>(stage + (lane & 31) * kStageRow<D> + c * (D / 8) + 2 * j) =
            u32x2{elem_pack<E>(x[j], x[j + 1]), elem_pack<E>(x[j + 2], x[j + 3])};
    }
  }
  const int token = r / a.G;
  if (half == 0 && r < R) {
    if (part >= 0) {
      a.stat[(at_part * kTile + local) * 2] = m;
      a.stat[(at_part * kTile + local) * 2 + 1] = total;
    } else if (a.lse) {
      const size_t at_row = static_cast<size_t>(row0 + token) * a.Hq + h * a.G + r % a.G;
      a.lse[at_row] = m == -INFINITY && total == 0.0f ? -INFINITY : (m - kLift + __builtin_amdgcn_logf(total)) * kLn2;
    }
  }
  if (part >= 0) return;
  constexpr int kLanes = D / 8, kRows = 64 / kLanes;  // lanes of a row, rows of a store
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < 32; i += kRows) {
    const int row = i + lane / kLanes, its = tile * kTile + wave * 32 + row, its_token = __shfl(token, row);
    const u32x4 x = *reinterpret_cast<const u32x4*>(stage + row * kStageRow<D> + lane % kLanes * 16);
    const size_t at_row = static_cast<size_t>(row0 + its_token) * a.Hq + h * a.G + (its - its_token * a.G);
    if (its < R) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + at_row * D + lane % kLanes * 8) = x;
  }
}

// The kernel's arguments, read again: those that are seldom needed would take
// scalar registers from the loop, and these vector registers.
__device__ __forceinline__ const ChunkArgs& arguments() {
  auto p = (const __attribute__((address_space(4))) ChunkArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ChunkArgs*)p;
}

template <int D>
struct Shared {
  Tile<D> tiles[2];
  std::conditional_t<D == 256, Waiting, int> waiting;
  uint32_t nan_groups[kTile];
};

template <int D, class E>
__device__ __forceinline__ void attend_piece(const ChunkArgs& a, int h, int at, Shared<D>& shared) {
  constexpr int kSteps = D / 16, DB = D / 32;
  constexpr int kGroup = D == 256 ? 1 : 2;  // tiles of 32 tokens at a time: the widest heads leave registers for one
  constexpr bool kWaits = D == 256;
  constexpr int kValueProducts = 2 * kGroup * DB, kProducts = kValueProducts + kGroup * kSteps, kAhead = D == 256 ? 3 : 6;
  constexpr int kPieces = D / 64 + D / 32;  // of a thread's widening: keys and values
  constexpr int kDeep = kWaits ? 1 : 2;     // pages whose codes are on the way
  Tile<D>(&tiles)[2] = shared.tiles;
  auto& waiting = shared.waiting;
  auto& nan_groups = shared.nan_groups;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // what is made of it is made for each piece again, or takes registers in between
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5, col = lane & 31;
  const int32_t* words = reinterpret_cast<const int32_t*>(a.piece + at);
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
  // Ids of the next view pages, one a lane: now those of v_ids .., then the 64 after these.  (Loads through the scalar
  // cache would wait for LDS reads and these for them.)
  const auto ids_of = [&](int v) { return v0 < v1 ? table[view.page(v + lane < v1 ? v + lane : v1 - 1)] : 0; };
  int v_ids = v0, ids = ids_of(v0), more_ids = ids_of(v0 + 64);
  // The first ids, the queries and the first page's codes are on the way together (six tiles a workgroup's place one
  // after another: 829 us, and 815 so).
  u32x4 q_words[kSteps];
  {
    const int token = r < R ? r / a.G : 0, hq = r < R ? h * a.G + r % a.G : 0;
    const uint16_t* src = a.q + static_cast<int64_t>(row0 + token) * a.row + hq * a.head + 8 * half;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q_words[s] = r < R ? *reinterpret_cast<const u32x4*>(src + 16 * s) : u32x4{0u, 0u, 0u, 0u};
  }
  __builtin_amdgcn_sched_barrier(0);
  // A page that the table does not name is read as the last one and seen by nobody.
  Raw<D> raws[kDeep];
  // The lane, found again for each page where the addresses made of it would take registers all the while.
  const auto here = [&] {
    int l = lane;
    if constexpr (kWaits) asm volatile("" : "+v"(l));
    return l;
  };
  const auto named = [&](int id) { return static_cast<unsigned>(id) < static_cast<unsigned>(a.c.pages); };
  const auto page_id = [&](int v) { return __builtin_amdgcn_readlane(ids, v - v_ids); };
  const uint8_t* blocks = static_cast<const uint8_t*>(a.c.data) + static_cast<size_t>(h) * KvBlock<D>::kBytes;
  const uint32_t page_bytes = static_cast<uint32_t>(a.c.Hk) * KvBlock<D>::kBytes;
  const uint32_t last_page = static_cast<uint32_t>(a.c.pages) - 1u;
  const auto block = [&](int id) {
    const uint32_t n = static_cast<uint32_t>(id);
    return blocks + static_cast<uint64_t>(page_bytes) * (n < last_page ? n : last_page);
  };
  const auto load = [&](Raw<D>& raw, int key_id, int value_id) {
    const int l = here();
    if constexpr (kWaits) {
      waiting.load(block(key_id), block(value_id), wave, l);
    } else {
      raw.load_keys(block(key_id), wave, l);
      raw.load_values(block(value_id), wave, l);
    }
  };
  if (half == 0) nan_groups[wave * 32 + col] = 0u;
  // A barrier at which what waits in LDS has arrived.
  const auto arrive = [] {
    if constexpr (kWaits) __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
    lds_barrier();
  };
  int id[4] = {0, 0, 0, 0};  // of pages v .. v + 3
  if (v0 < v1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = page_id(v0 + i);
    load(raws[0], id[0], id[0]);
  }
  __builtin_amdgcn_sched_barrier(0);
  f16x8 q[kSteps];
  float cm;
  {
    float factor = 1.0f;
    if constexpr (std::is_same_v<E, BF16>) {
      // To fp16's range by the power of two that brings the row's greatest value to 2^14 .. 2^15:
      // values down to 2^-31 of it keep all their bits, the rest is off by 2^-39 of it at most.
      float amax = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = fabsf(elem_lo<E>(q_words[s][j])), hi = fabsf(elem_hi<E>(q_words[s][j]));
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
          q_words[s][j] = elem_pack<F16>(ldexpf(elem_lo<E>(q_words[s][j]), 14 - ex), ldexpf(elem_hi<E>(q_words[s][j]), 14 - ex));
      factor = ldexpf(1.0f, ex - 14);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      q[s] = __builtin_bit_cast(f16x8, q_words[s]);
      // (Opaque: the loop, otherwise the same, gets other registers, and takes 2% less with bf16, 1% with the widest
      // heads; with fp16 and D = 128 it takes 1.5% more.)
      if constexpr (std::is_same_v<E, BF16> || D == 256) asm volatile("" : "+v"(q[s]));
    }
    cm = fmaxf(a.scale * a.c.gk * kLog2e * factor, kMinNormal);
    // The loop must not wait for these again, and with them for the next page.
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 15));
  }
  float m = -INFINITY, l = 0.0f, l_over = 0.0f;  // l_over: what rounding put into l beyond the weights' sum
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};

  if (v0 < v1) {
    // The first products are of no weights with the values of no page.
    uint32_t zero = 0u;
    asm volatile("" : "+v"(zero));
    for (int i = threadIdx.x; i < D * Tile<D>::kValueRow / 8; i += kThreads) *reinterpret_cast<u32x4*>(tiles[1].v + 8 * i) = u32x4{zero, zero, zero, zero};
    if constexpr (kWaits) {
      arrive();
      waiting.arrived(&raws[0], wave, here());
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) widen_keys<D>(raws[0], key_row_of<D>(&tiles[0], wave, here()), wave, i);
    if constexpr (kWaits) arrive();  // what was waiting has been read
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      load(raws[i], id[i + 1], id[i]);
      asm volatile("" ::: "memory");  // in this order, which the loop's waits count on
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  arrive();
  if (wave >= kWaves / 2) lds_barrier();

  const int key_row = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
  f16x8 w[2 * kGroup];  // weights of the tokens before: none yet
#pragma unroll
  for (int i = 0; i < 2 * kGroup; ++i) w[i] = f16x8{};
  int flagged = -1;  // the first slot of the page before, where NaN values of it may have been noted
  // Operand i of a phase's products: the values of the tokens before, then the keys of these.
  const auto operand = [&](const Tile<D>& before, int before_u0, const Tile<D>& now, int u0, int i) {
    const int step = i / DB, d = i % DB, j = i - kValueProducts;
    return *reinterpret_cast<const f16x8*>(
        i < kValueProducts ? before.v + (32 * d + col) * Tile<D>::kValueRow + 32 * before_u0 + 16 * step + 8 * half
                           : now.k + (32 * (u0 + j % kGroup) + key_row) * Tile<D>::kKeyRow + 16 * (j / kGroup) + 8 * half);
  };
  const auto add_values = [&](f16x8 x, int i) { o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, w[i / DB], o[i % DB], 0, 0, 0); };
  // The groups of positions where this lane's row sees a NaN value of the page before are kept for the end.
  const auto add_bad = [&](const Tile<D>& of) {
    uint32_t any = 0u, groups = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= of.any[i];
    if (!any) return;
    const ChunkArgs& a = arguments();
    for (int t = 0; t < kPage; ++t) {
      const int slot = flagged + t;
      if (of.any[t / 16] && slot < limit && (!a.window || slot >= limit - a.window || slot < a.sinks)) groups |= of.bad[t];
    }
    if (half == 0) nan_groups[wave * 32 + col] |= groups;
  };
  // The pages that all of the tile's rows see whole, most of them: view pages easy .. easy + easy_many.
  const Sight whole_tile(a, tile_least, tile_most);
  const int easy = view.low + whole_tile.whole_begin - view.from;
  const unsigned easy_many = whole_tile.whole_end > whole_tile.whole_begin ? whole_tile.whole_end - whole_tile.whole_begin : 0;

  // A page, whose codes are in raw.
  const auto step = [&](int v, Raw<D>& raw, Tile<D>& now, Tile<D>& other) {
    const bool live = named(id[0]) && (kDeep == 1 || v < v1), whole = static_cast<unsigned>(v - easy) < easy_many && live;
    bool work = busy, partial = false;
    int first = 0;
    if (flagged >= 0) add_bad(other);
    flagged = -1;
    if constexpr (kWaits) waiting.arrived(&raw, wave, here());
    if (!whole) {
      // (Found for each such page, of which there are few: kept, all this takes more scalar registers than there are.)
      int limits[4] = {tile_least, tile_most, wave_least, wave_most};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm volatile("" : "+s"(limits[i]));
      const ChunkArgs& a = arguments();
      const Sight tile_sight(a, limits[0], limits[1]), wave_sight(a, limits[2], limits[3]);
      const int page = view.page(v);
      const bool noted = !live || !tile_sight.whole(page);
      first = page * kPage;
      work = busy && live && wave_sight.some(page);
      partial = work && !wave_sight.whole(page);
      if (noted) note_bad<D>(&raw, &now, wave, here());
      flagged = noted && live ? first : -1;
    }
#pragma unroll
    for (int u0 = 0; u0 < 2; u0 += kGroup) {
      f32x16 s[kGroup];
      // Keys are widened a page ahead; values, which the next phase's products want, of this one.
      _Float16 *row = key_row_of<D>(&other, wave, here()), *column = value_column_of<D>(&now, wave, here());
      const auto widen = [&](int i) {
        if (i < kPieces) {
          if (i < D / 64) widen_keys<D>(raw, row, wave, i);
          else widen_values<D>(raw, column, wave, i - D / 64);
        }
      };
      const auto widen_alone = [&] {
        // (Opaque, or the conversions would be taken out of both branches and done before the products.)
        if constexpr (!kWaits) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) asm volatile("" : "+v"(raw.k[i]), "+v"(raw.v[i]), "+v"(raw.v[D / 64 + i]));
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          if constexpr (kWaits) {
            if (i == D / 64 || i == D / 64 + 4) waiting.arrived_values(&raw, i == D / 64 ? 0 : 1, wave, here());
          }
          widen(i);
          __builtin_amdgcn_sched_barrier(0);  // one piece's registers at a time
        }
      };
      if (u0 == 0 && kWaits) widen_alone();
      if (busy) {
        // The operands are read kAhead products before they are used, and a piece of the widening follows each
        // product: left to itself the compiler reads two operands, waits for them, and pays LDS's latency sixteen times.
        const Tile<D>& before = u0 ? now : other;
        const int before_u0 = u0 ? u0 - kGroup : 2 - kGroup;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) s[u] = f32x16{};
        f16x8 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = operand(before, before_u0, now, u0, i);
        __builtin_amdgcn_s_setprio(3);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kProducts; ++i) {
          const int j = i - kValueProducts;
          if (i < kValueProducts) add_values(x[i % kAhead], i);
          else s[j % kGroup] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[i % kAhead], q[j / kGroup], s[j % kGroup], 0, 0, 0);
          if (i + kAhead < kProducts) x[i % kAhead] = operand(before, before_u0, now, u0, i + kAhead);
          if (u0 == 0 && !kWaits) widen(i);
          __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
      } else if (u0 == 0 && !kWaits) {
        widen_alone();
      }
      lds_barrier();
      if (u0 == 0) {
        load(raw, id[kDeep + 1], id[kDeep]);
        if (v + 4 - v_ids == 64) {
          v_ids += 64;
          ids = more_ids;
          more_ids = ids_of(v_ids + 64);
        }
      }
      if (work) {
        if (partial) {
          const ChunkArgs& a = arguments();
          // Slots counted from the lane's first.  (Opaque, or its differences to the 32 tokens are kept all the while.)
          int until = limit - first - 32 * u0 - 8 * half;
          asm volatile("" : "+v"(until));
          const int from = a.window ? (until > 0 ? until : 0) - a.window : -kPage, sunk = a.sinks - first - 32 * u0 - 8 * half;
#pragma unroll
          for (int u = 0; u < kGroup; ++u)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int slot = 32 * u + 16 * (e / 8) + e % 8;
              const bool out = (slot >= until) | ((slot < from) & (slot >= sunk));
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
          l_over *= alpha;
#pragma unroll
          for (int d = 0; d < DB; ++d) o[d] *= alpha;
        }
        const float lifted = m == -INFINITY ? 0.0f : m - kLift;
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][e], cm, -lifted));
            sum += x;
            w[2 * u + e / 8][e % 8] = static_cast<_Float16>(x);
          }
        // A long sequence's slots may each be too small for a sum of thousands of pages (120000 slots: the log-sum was off
        // by 1e-4): what an addition loses goes into the next one.
        sum -= l_over;
        const float more = l + sum;
        l_over = (more - l) - sum;
        l = more;
      } else {
#pragma unroll
        for (int i = 0; i < 2 * kGroup; ++i) w[i] = f16x8{};
      }
      if (u0 + kGroup == 2) arrive();
      else lds_barrier();
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) id[i] = id[i + 1];
    id[3] = page_id(v + 4);
  };
  // Two pages a turn, whose registers take turns.  (Leaving the loop between them, the compiler waits for both pages'
  // codes at the first one's use.)  An odd last turn ends with a page that nobody sees.
  const int last_odd = kDeep == 2 ? 1 : (v1 - 1 - v0) & 1;
  for (int v = v0; v < v1; v += kDeep) {
    if constexpr (kDeep == 2) {
      step(v, raws[0], tiles[0], tiles[1]);
      step(v + 1, raws[1], tiles[1], tiles[0]);
    } else {
      step(v, raws[0], tiles[(v - v0) & 1], tiles[(v + 1 - v0) & 1]);
    }
  }
  if (busy && v0 < v1) {
#pragma unroll
    for (int i = 0; i < kValueProducts; ++i) add_values(operand(tiles[last_odd], 2 - kGroup, tiles[0], 0, i), i);
  }
  if (flagged >= 0) add_bad(tiles[last_odd]);
  if (wave < kWaves / 2) lds_barrier();
  if (part < 0) lds_barrier();  // all have done with the tiles, where the rows wait to be stored
  static_assert(kWaves * 32 * kStageRow<D> <= sizeof(shared.tiles));
  if (busy)
    store_rows<D, E>(arguments(), here(), wave, h, row0, R, tile, part, m, l, nan_groups[wave * 32 + (here() & 31)], o,
                     reinterpret_cast<uint8_t*>(&tiles[0]) + wave * 32 * kStageRow<D>);
}

template <int D, class E>
__global__ __launch_bounds__(kThreads, 2) void chunk(const ChunkArgs a) {
  __shared__ __align__(16) Shared<D> shared;
  const int at = static_cast<int>(blockIdx.x) / a.c.Hk, h = static_cast<int>(blockIdx.x) % a.c.Hk;
  if (at >= uniform_load(a.counts, 0)) return;
  const int begin = uniform_load(a.first, at), end = uniform_load(a.first, at + 1);
  for (int p = begin; p < end; ++p) {
    if (p > begin) lds_barrier();  // all have done with the tiles of the piece before
    attend_piece<D, E>(arguments(), h, p, shared);
  }
}

// Adds the pieces of cut tiles: a wavefront has a unit of them, kBatch pieces' loads at a time.  Bound by memory: 31 cut
// tiles of 8 heads, 65 MB of parts in 16 us (of rows that lie together, 18).
template <int D, class E>
__global__ __launch_bounds__(256) void chunk_join(const ChunkArgs a) {
  constexpr int kQuarters = D / 64, kBatch = D == 256 ? 4 : 8;
  const int at = static_cast<int>(blockIdx.x) / a.c.Hk, h = static_cast<int>(blockIdx.x) % a.c.Hk;
  if (at >= uniform_load(a.counts, 1)) return;
  const Cut sp = a.cut[at];
  const int lane = threadIdx.x & 63, unit = static_cast<int>(blockIdx.y) * 4 + static_cast<int>(threadIdx.x >> 6);
  const int local = unit / 8 * 32 + (lane & 31), r = sp.tile * kTile + local, c = first_position(unit % 8, lane >> 5);
  if (r >= sp.T * a.G) return;
  float mm = -INFINITY, total = 0.0f;
  f32x4 x[kQuarters];
#pragma unroll
  for (int q = 0; q < kQuarters; ++q) x[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < sp.pieces; s0 += kBatch) {
    float2 st[kBatch];
    f32x4 v[kBatch][kQuarters];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const int piece = s0 + s < sp.pieces ? s0 + s : s0;
      const size_t p = static_cast<size_t>(h) * a.parts + sp.part + piece;
      st[s] = *reinterpret_cast<const float2*>(a.stat + (p * kTile + local) * 2);
#pragma unroll
      for (int q = 0; q < kQuarters; ++q) v[s][q] = *reinterpret_cast<const f32x4*>(a.part + part_at<D>(p, unit, q, lane));
    }
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s < sp.pieces) {
        // A piece without weight is zeros; one with nothing but NaN scores has the same
        // maximum, -inf, but a NaN sum: both are added, times 0.
        const float to = fmaxf(mm, st[s].x), about = to == -INFINITY ? 0.0f : to;
        const float f0 = __builtin_amdgcn_exp2f(mm - about), f = __builtin_amdgcn_exp2f(st[s].x - about);
        mm = to;
        total = total * f0 + f * st[s].y;
#pragma unroll
        for (int q = 0; q < kQuarters; ++q) x[q] = x[q] * f0 + f * v[s][q];
      }
  }
  const size_t at_row = static_cast<size_t>(sp.first + r / a.G) * a.Hq + h * a.G + r % a.G;
  const float inv = mm == -INFINITY ? 0.0f : a.c.gv / total;
#pragma unroll
  for (int q = 0; q < kQuarters; ++q) {
    x[q] *= inv;
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at_row * D + c * (D / 16) + 4 * q) =
        u32x2{elem_pack<E>(x[q][0], x[q][1]), elem_pack<E>(x[q][2], x[q][3])};
  }
  if (c == 0 && a.lse) a.lse[at_row] = mm == -INFINITY && total == 0.0f ? -INFINITY : (mm - kLift + __builtin_amdgcn_logf(total)) * kLn2;
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

ChunkPlan kv4_chunk_plan(int N, int B, int Hq, int Hk, int D, int width, int window, int sinks) {
  ChunkPlan p{};
  const int64_t G = Hq / Hk, busy = N < B ? N : B;  // sequences with rows
  p.tiles = (N * G + busy * (kTile - 1)) / kTile;
  // The pages that a tile can see: its rows' tokens, a window before the first of them, and the sinks.
  int64_t pages = width;
  if (window) {
    const int64_t tokens = (kTile - 1) / G + 2 < N ? (kTile - 1) / G + 2 : N;
    const int64_t seen = (window + tokens) / kPage + 2 + (static_cast<int64_t>(sinks) + kPage - 1) / kPage;
    pages = seen < pages ? seen : pages;
  }
  p.small = kv4_small_chunk(N, B, static_cast<int>(G), Hk, D, pages);
  if (p.small.tiles) {
    p.groups = p.small.shares;
    p.total = p.small.total;
    return p;
  }
  // Of g workgroups in a row at most g - 1 begin inside a tile, and each of these cuts makes one piece more.
  const int64_t slots = slots_per_head(Hk), even = (p.tiles * (pages + kBegin) + kLeast - 1) / kLeast;
  const int64_t inside = slots < 4 ? 0 : (slots < even ? slots : even) - 1;
  p.cuts = p.tiles < inside ? p.tiles : inside;
  p.parts = p.cuts + inside;
  p.groups = p.tiles > inside + 1 ? p.tiles : inside + 1;
  p.counts_off = kSyncBytes;
  p.begin_off = p.counts_off + 256;
  p.offset_off = p.begin_off + up(static_cast<size_t>(B + 1) * 4);
  p.first_off = p.offset_off + up(static_cast<size_t>(B) * 4);
  p.piece_off = p.first_off + up(static_cast<size_t>(p.groups + 1) * 4);
  p.cut_off = p.piece_off + up(static_cast<size_t>(p.tiles + inside) * sizeof(Piece));
  p.stat_off = p.cut_off + up(static_cast<size_t>(p.cuts) * sizeof(Cut));
  p.part_off = p.stat_off + static_cast<size_t>(Hk) * p.parts * kTile * 8;
  p.total = p.part_off + static_cast<size_t>(Hk) * p.parts * kTile * D * 4;
  return p;
}

hipError_t launch_kv4_chunk(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N, int type,
                            int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace, hipStream_t stream) {
  const ChunkPlan p = kv4_chunk_plan(N, c.B, Hq, c.Hk, c.D, c.width, window, sinks);
  if (p.small.tiles)
    return launch_kv4_small_chunk(c, q, row, head, starts, N, type, Hq, scale, window, sinks, out, lse, workspace, p.small, stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ChunkArgs a{c, static_cast<const uint16_t*>(q), row, head, starts, out, lse, reinterpret_cast<int*>(ws + p.counts_off),
                    reinterpret_cast<int*>(ws + p.begin_off), reinterpret_cast<int*>(ws + p.offset_off), reinterpret_cast<int*>(ws + p.first_off),
                    reinterpret_cast<Piece*>(ws + p.piece_off), reinterpret_cast<Cut*>(ws + p.cut_off),
                    reinterpret_cast<float*>(ws + p.stat_off), reinterpret_cast<float*>(ws + p.part_off), p.parts, N, Hq, Hq / c.Hk,
                    window, sinks, scale};
  chunk_plan<<<1, kPlanThreads, 0, stream>>>(a);
  const auto run = [&](auto d, auto e) {
    chunk<d(), decltype(e)><<<dim3(static_cast<unsigned>(p.groups * c.Hk)), kThreads, 0, stream>>>(a);
    if (p.cuts)
      chunk_join<d(), decltype(e)><<<dim3(static_cast<unsigned>(p.cuts * c.Hk), kTile / 16), 256, 0, stream>>>(a);
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
