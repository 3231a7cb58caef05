// Attention over the 4-bit key/value cache, and the attention weights it adds
// to the slots.
//
// With S = scale q . K~ over the slots that a row sees:
//   out = sum_j exp(S_j - m) v~_j / sum_j exp(S_j - m),  lse = m + log(sum)
//   weight_j = sum over rows of exp(S_j - lse)
//
// A wavefront takes a page (64 tokens) of one key/value head for up to MT * 16
// of the head's T * G query rows, so that codes are widened once for all of
// them.  Both products run on v_mfma_f32_16x16x32_f16 in the transposed form:
//   S^T[token][query] = K[token][d] Q^T[d][query]
//   O^T[d][query]     = V^T[d][token] P^T[token][query]
// The first leaves lane 16 g + c with query c's scores of tokens 4 g .. 4 g + 3
// of a 16-token tile, which is how the second wants its right operand (any
// order of the summed tokens serves as long as both operands have it), so P
// never leaves its lanes, and the running maximum and sum of a query are values
// of its own lanes.  The cache's byte order gives lane 16 g + c of every load
// the K codes of token c's quarter g, and the V codes of tokens 4 g .. 4 g + 3
// at positions c * D/16 ...
#include <hip/hip_runtime.h>

#include "kv4.cuh"
#include "kv4_internal.h"

namespace skinny {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kMinNormal = 0x1p-126f;
// Weights go to fp16 times 2^kLift relative to the reference maximum, which
// follows the running one only when that rose by more than 2^kSlack: weights
// then stay below 2^(kLift + kSlack) = 2^14 and keep fp16's full precision
// down to 2^-20 of the greatest, and a row's sums are rescaled rarely.
constexpr float kLift = 6.0f, kSlack = 8.0f;

struct ChunkSegment {  // a group of rows of a sequence, for the join of its shares
  int first, splits;   // its first share and their number; the next is Hk further
  int row0, r0, R;     // the sequence's first token among all, the group's first row in it, and the sequence's rows
  int pad[3];
};

struct AttendArgs {
  kv4_cache c;
  kv4_rows q;
  void* out;
  float* lse;
  float* part;   // [share][MT * 16][D]: sums of a split segment's shares
  float* stat;   // [share][MT * 16][2]: their reference maximum (log2) and sum
  int2* split;   // [segment]: its first share and their number
  int T, Hq, G, QG;
  int least;     // fewest pages of a share
  float scale;
  int window, sinks;  // windowed calls: a row with limit L sees the slots from L - window on, and those below sinks
  const int32_t* starts;  // chunks of another length for each sequence: their rows (see kv4_attention_chunk), of N
  int N;
  ChunkSegment* segments;  // [group][Hk] where chunks are split, and the number of groups; otherwise null
  int* count;
};

// The pages that rows with limits from `least` to `most` see: all up to the
// latter, or with a window the first `low`, which hold the sinks, and those from
// `from` on, where the earliest row's window begins.
template <bool WINDOW>
struct View {
  int low, from, end;
  __device__ __forceinline__ View(const AttendArgs& a, int least, int most) : low(0), from(0), end((most + kPage - 1) / kPage) {
    if constexpr (WINDOW) {
      least -= a.window;
      from = least > 0 ? least / kPage : 0;
      low = a.sinks / kPage + (a.sinks % kPage != 0);
      low = low < from ? low : from;
    }
  }
  __device__ __forceinline__ int pages() const { return WINDOW ? low + end - from : end; }
  __device__ __forceinline__ int page(int v) const { return !WINDOW || v < low ? v : v - low + from; }
};

// Whether a row with this limit does not see the slot.
template <bool WINDOW>
__device__ __forceinline__ bool hidden(const AttendArgs& a, int slot, int limit) {
  return slot >= limit || (WINDOW && slot < limit - a.window && slot >= a.sinks);
}

// A row's log-sum, of its reference maximum (log2) and its sum: -inf for a row
// without weight, and NaN for one with a NaN among its scores.  Maxima pass over
// NaN, so that a row of nothing else keeps the -inf that it began with; the sum tells.
__device__ __forceinline__ float log_sum(float m, float total) {
  return m == -INFINITY && total == 0.0f ? -INFINITY : (m - kLift + __builtin_amdgcn_logf(total)) * kLn2;
}

// As sum_over_rows, for the greatest.
__device__ __forceinline__ float max_over_rows(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  const uint32_t w = __float_as_uint(v);
  const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// A workgroup's query rows: loaded before its keys, since loads arrive in
// order, then put into LDS as fp16 with a row stride of D + 8 halves (16 bytes
// off the banks' period).  bf16 rows are scaled by the power of two that brings
// their greatest value to 2^14 .. 2^15; `factor` undoes it.  A bf16 value has
// eight bits and fp16's least step is 2^-24: what is scaled to 2^-17 or more,
// 2^-31 of the greatest, keeps them all, and the rest is off by 2^-39 of the
// greatest at most.
template <int D, int MT>
struct Queries {
  static constexpr int kPer = D / 8;  // threads per row
  static constexpr int kItems = (MT * 16 * kPer + kThreads - 1) / kThreads;
  static_assert(MT * 16 * kPer % 64 == 0, "whole wavefronts take part in the shuffles");
  u32x4 loaded[kItems];

  __device__ __forceinline__ void load(const kv4_rows& q, int b, int h, int qg, int G, int R) {
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int i = n * kThreads + threadIdx.x, r = qg * MT * 16 + i / kPer;
      loaded[n] = u32x4{0u, 0u, 0u, 0u};
      if (i < MT * 16 * kPer && r < R)
        loaded[n] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(q.data) + b * q.sequence + (r / G) * q.row +
                                                    (h * G + r % G) * q.head + i % kPer * 8);
    }
  }
  template <class E>
  __device__ __forceinline__ void put(_Float16* qs, float* factor) const {
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      const int i = n * kThreads + threadIdx.x;
      if (i < MT * 16 * kPer) put_piece<E>(i / kPer, i % kPer, loaded[n], qs, factor);
    }
  }
  template <class E>
  static __device__ __forceinline__ void put_piece(int row, int piece, u32x4 w, _Float16* qs, float* factor) {
    if constexpr (std::is_same_v<E, BF16>) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = fabsf(elem_lo<E>(w[j])), hi = fabsf(elem_hi<E>(w[j]));
        amax = lo < INFINITY ? fmaxf(amax, lo) : amax;
        amax = hi < INFINITY ? fmaxf(amax, hi) : amax;
      }
#pragma unroll
      for (int o = 1; o < kPer; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o));
      int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      ex = ex < -100 ? -100 : ex;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = elem_pack<F16>(ldexpf(elem_lo<E>(w[j]), 14 - ex), ldexpf(elem_hi<E>(w[j]), 14 - ex));
      if (piece == 0) factor[row] = ldexpf(1.0f, ex - 14);
    } else if (piece == 0) {
      factor[row] = 1.0f;
    }
    *reinterpret_cast<u32x4*>(qs + row * (D + 8) + piece * 8) = w;
  }
};

// A lane's part of a block: K and V codes and scales.  All are loaded
// non-temporally: a layer's cache is not read again before the rest of the model
// has passed through the caches.  With the scales alone loaded in the ordinary way
// 290 MB from cold caches take 67 us instead of 52, with the keys too 89; where
// all of it stays in the last-level cache between calls, ordinary loads gain 1 or 2%.
template <int D>
struct KRegs {
  u32x4 codes[D / 32];
  uint32_t scales[D / 64];
  __device__ __forceinline__ void load(const uint8_t* block, int lane) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) codes[i] = load16(block + i * 1024 + lane * 16);
    const uint8_t* s = block + KvBlock<D>::kKScales + lane * (D / 16);
    if constexpr (D == 64) {
      scales[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(s));
    } else if constexpr (D == 128) {
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(s));
      scales[0] = v.x;
      scales[1] = v.y;
    } else {
      const u32x4 v = load16(s);
#pragma unroll
      for (int i = 0; i < 4; ++i) scales[i] = v[i];
    }
  }
  // Keys of tile j (tokens 16 j ..), the eight positions 8 step .. of the lane's quarter.
  __device__ __forceinline__ f16x8 frag(int j, int step) const {
    const int w = j * (D / 32) + step, b = j * (D / 64) + step / 2;
    const uint32_t sw = scales[b / 4];
    const f16x2 pair = (b % 4) / 2 ? e4m3x2<true>(sw) : e4m3x2<false>(sw);
    const _Float16 s = pair[b % 2];
    return e2m1x8(codes[w / 4][w % 4]) * f16x8{s, s, s, s, s, s, s, s};
  }
};

__device__ __forceinline__ uint32_t bits_of(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

template <int D>
struct VRegs {
  u32x4 codes[D / 32];
  uint32_t scales[4];  // byte i of scales[j]: token 16 j + 4 g + i
  __device__ __forceinline__ void load(const uint8_t* block, int lane) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) codes[i] = load16(block + KvBlock<D>::kVCodes + i * 1024 + lane * 16);
    const int g = lane >> 4, c = lane & 15;
    const u32x4 v = load16(block + KvBlock<D>::kVScales + (c * (D / 16) / 16) * 64 + g * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) scales[i] = v[i];
  }
  // Codes of a pair of tokens (2 p, 2 p + 1 of the lane's four of tile j) at
  // eight positions (D == 64: four), one byte per position with the first
  // token's code in its low nibble: even positions in .x, odd ones in .y.
  __device__ __forceinline__ u32x2 pair(int j, int p, int half) const {
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
    if constexpr (D == 64) {
      const uint32_t w = codes[(j * 2 + p) / 4][(j * 2 + p) % 4];
      return u32x2{bits_of(kLow, w, w >> 12), bits_of(kLow, w >> 4, w >> 16)};
    } else {
      const int i = (j * 4 + p * 2) * (D / 128) + half, i2 = i + D / 128;
      const uint32_t a = codes[i / 4][i % 4], b = codes[i2 / 4][i2 % 4];
      return u32x2{bits_of(kLow, a, b << 4), bits_of(kLow, a >> 4, b)};
    }
  }
};

template <int B>
__device__ __forceinline__ f16x2 e2m1_at(u32x2 pair, int odd) {
  return e2m1x2<B>(odd ? pair.y : pair.x);
}
__device__ __forceinline__ f16x2 e2m1_pos(u32x2 pair, int s) {  // position s (0 .. 7), a constant after unrolling
  switch (s / 2) {
    case 0: return e2m1_at<0>(pair, s & 1);
    case 1: return e2m1_at<1>(pair, s & 1);
    case 2: return e2m1_at<2>(pair, s & 1);
    default: return e2m1_at<3>(pair, s & 1);
  }
}

// Slots past the sequence's length hold anything: their V scales become 0, so
// that the codes stand for 0 and not for NaN.  A NaN in a slot that only later
// rows see must not reach the others through a weight of 0: such scales become
// 0 too, and the sums of the rows that do see the slot are made NaN by hand, where
// the scale is theirs.
template <bool WINDOW, int D, int MT>
__device__ __forceinline__ void clean_values(const AttendArgs& a, VRegs<D>& v, int first, int len, int lane,
                                             const int (&limit)[MT], f32x4 (&o)[MT][D / 16]) {
  const int g = lane >> 4;
  uint32_t bad = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int left = len - (first + 16 * j + 4 * g);
    left = left < 0 ? 0 : left;
    if (left < 4) v.scales[j] &= (1u << (8 * left)) - 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((v.scales[j] >> (8 * i)) & 0x7Fu) == 0x7Fu) {
        bad |= 1u << (4 * j + i);
        v.scales[j] &= ~(0xFFu << (8 * i));
      }
  }
  if (!__any(bad != 0u)) return;
  // Row r of the sums is of the values that lanes r, 16 + r, .. hold: these rows, and no others of the query, are
  // made NaN where it sees the token.
  for (int rg = 0; rg < 4; ++rg)
    for (int tg = 0; tg < 4; ++tg)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t of = __builtin_amdgcn_readlane(bad, 16 * tg + 4 * rg + e);
        if (!of) continue;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          bool seen = false;
          for (int i = 0; i < 16; ++i) seen |= ((of >> i) & 1u) && !hidden<WINDOW>(a, first + 16 * (i / 4) + 4 * tg + i % 4, limit[mt]);
          if (seen && g == rg) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) o[mt][s][e] = NAN;
          }
        }
      }
}

// A workgroup's share of the work: pages p0 .. p1 of one segment (sequence b,
// head h, query group qg).  The lengths are known to the device only, so every
// wavefront works the same plan out of them: the least number of pages per
// share for which the shares of all segments, each cut into equal ones, fit
// the grid.  A long sequence among short ones then has more workgroups, and no
// share is much longer than the mean.
struct Share {
  int b, h, qg, len, p0, p1, splits, first;  // first: the segment's first share; the next is Hk * QG further
  bool any;
};
template <bool WINDOW>
__device__ __forceinline__ Share plan_share(const AttendArgs& a, int lane) {
  const kv4_cache& c = a.c;
  const int QG = a.QG, least = a.least;
  const auto seen = [&](int len) { return View<WINDOW>(a, len - (a.T - 1), len).pages(); };
  const int per = c.Hk * QG;                      // segments of a sequence
  const int room = static_cast<int>(gridDim.x) / per;  // shares per head and query group; at least B
  const int at = static_cast<int>(blockIdx.x) / per;
  Share s;
  s.any = false;
  s.b = s.len = s.p0 = s.p1 = s.splits = s.first = 0;
  const int hq = static_cast<int>(blockIdx.x) % per;
  s.h = hq / QG;
  s.qg = hq % QG;
  if (room == c.B) {  // one share per segment
    s.any = true;
    s.b = at;
    s.len = kv_len_uniform(c, at);
    s.p1 = seen(s.len);
    s.splits = 1;
    s.first = static_cast<int>(blockIdx.x);
    return s;
  }
  const auto pages = [&](int b) { return b < c.B ? seen(kv_len(c, b)) : 0; };
  const int held = lane < c.B ? kv_len(c, lane) : 0;  // of the first 64 sequences
  int mine = seen(held), total = 0;
  for (int b0 = 0; b0 < c.B; b0 += 64)
    total += __builtin_amdgcn_readlane(wave_scan(b0 ? pages(b0 + lane) : mine), 63);
  int chunk = total / (room - (c.B >> 1)) + 1;
  chunk = chunk < least ? least : chunk;
  const auto shares = [&](int b0) {
    const int n = ((b0 ? pages(b0 + lane) : mine) + chunk - 1) / chunk;
    return b0 + lane < c.B ? (n < 1 ? 1 : n) : 0;
  };
  for (;;) {
    int all = 0;
    for (int b0 = 0; b0 < c.B; b0 += 64) all += __builtin_amdgcn_readlane(wave_scan(shares(b0)), 63);
    if (all <= room) break;
    chunk += (chunk >> 4) + 1;
  }
  int before = 0;
  for (int b0 = 0; b0 < c.B; b0 += 64) {
    const int n = shares(b0), upto = before + wave_scan(n);
    const int last = __builtin_amdgcn_readlane(upto, 63);
    if (at < last) {
      const int l = __popcll(__ballot(upto <= at));  // the lane of the sequence
      s.any = true;
      s.b = b0 + l;
      s.splits = __builtin_amdgcn_readlane(n, l);
      const int first = __builtin_amdgcn_readlane(upto, l) - s.splits;
      s.first = first * per + hq;
      s.len = b0 ? kv_len_uniform(c, s.b) : __builtin_amdgcn_readlane(held, l);
      const int np = seen(s.len), each = (np + s.splits - 1) / s.splits;
      s.p0 = (at - first) * each;
      s.p1 = s.p0 + each < np ? s.p0 + each : np;
      break;
    }
    before = last;
  }
  // The compiler does not see that all lanes agree.
  for (int* f : {&s.b, &s.h, &s.qg, &s.len, &s.p0, &s.p1, &s.splits, &s.first}) *f = __builtin_amdgcn_readfirstlane(*f);
  return s;
}

// Chunks: a workgroup has a group of `rows` rows of a head and the pages that they
// see, or a share of these.  The rows of a sequence go from its start to the next
// one's, as in kv4_chunk.hip: starts are held to 0 .. N and to what came before
// them.  Shares are found as above, but for a sequence's groups alike: as many as
// the pages of its last group want, of which no other has more.  Of a group of rows
// that see fewer the last shares may be left without a page, and add nothing.
struct ChunkRows {
  int T, row0;      // the sequence's tokens, and its first row
  int end, group;   // where the share's pages end, and the group among all sequences'
};
__device__ __forceinline__ Share chunk_share(const AttendArgs& a, int rows, int lane, ChunkRows* of) {
  const int at = static_cast<int>(blockIdx.x) / a.c.Hk, B = a.c.B;
  const auto held = [&](int s, int least) { return s < least ? least : (s > a.N ? a.N : s); };
  struct Sequence {
    int begin, end, n, pages, len;  // its rows, groups of these, and the pages that they see
  };
  // Of sequence b0 + lane; `start` goes from the first one's to the next ones'.
  const auto sequence = [&](int b0, int& start) {
    const int b = b0 + lane;
    Sequence s{0, 0, 0, 0, 0};
    s.end = held(b < B ? a.starts[b + 1] : 0, start);
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(s.end, o);
      if (lane >= o && x > s.end) s.end = x;
    }
    const int up = __shfl_up(s.end, 1);
    s.begin = lane ? up : start;
    if (b < B) {
      s.n = static_cast<int>((static_cast<int64_t>(s.end - s.begin) * a.G + rows - 1) / rows);
      s.len = kv_len(a.c, b);
      const int tokens = s.end - s.begin < rows ? s.end - s.begin : rows, least = s.len - (tokens - 1);
      const View<true> view(a, least < 0 ? 0 : least, s.len);
      s.pages = view.pages() + (view.from > 0);  // another group's window may lie across one page more
    }
    start = __builtin_amdgcn_readlane(s.end, 63);
    return s;
  };
  const int start0 = held(uniform_load(a.starts, 0), 0);
  int after0 = start0;
  const Sequence first = sequence(0, after0);
  int chunk = 0;
  const auto shares = [&](const Sequence& s) { return chunk && s.pages > chunk ? s.n * ((s.pages + chunk - 1) / chunk) : s.n; };
  const auto sum = [&](auto of_sequence) {
    int start = after0, all = 0;
    for (int b0 = 0; b0 < B; b0 += 64) all += __builtin_amdgcn_readlane(wave_scan(of_sequence(b0 ? sequence(b0, start) : first)), 63);
    return all;
  };
  if (a.segments) {
    const int room = static_cast<int>(gridDim.x) / a.c.Hk, groups = sum([](const Sequence& s) { return s.n; });
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.count = groups;
    chunk = sum([](const Sequence& s) { return s.n * s.pages; }) / (room - (groups >> 1)) + 1;
    chunk = chunk < a.least ? a.least : chunk;
    while (sum(shares) > room) chunk += (chunk >> 4) + 1;
  }
  Share s;
  s.any = false;
  s.h = static_cast<int>(blockIdx.x) % a.c.Hk;
  s.b = s.qg = s.len = s.p0 = s.p1 = s.first = 0;
  s.splits = 1;
  of->end = of->group = 0;
  int before = 0, groups = 0;
  for (int b0 = 0, start = after0; b0 < B; b0 += 64) {
    const Sequence q = b0 ? sequence(b0, start) : first;
    const int all = shares(q), upto = before + wave_scan(all), group = groups + wave_scan(q.n), last = __builtin_amdgcn_readlane(upto, 63);
    if (at < last) {
      const int l = __popcll(__ballot(upto <= at));  // the lane of the sequence
      const auto its = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
      s.any = true;
      s.b = b0 + l;
      const int in = at - (its(upto) - its(all));  // among the sequence's shares
      s.qg = in;
      int each = 0, share = 0;
      if (chunk) {
        s.splits = its(all) / its(q.n);
        s.qg = in / s.splits;
        share = in - s.qg * s.splits;
        each = (its(q.pages) + s.splits - 1) / s.splits;
      }
      of->group = its(group) - its(q.n) + s.qg;
      s.p0 = share * each;
      of->end = share == s.splits - 1 ? 0x7FFFFFFF : s.p0 + each;  // the last one's: what there is
      s.first = (at - share) * a.c.Hk + s.h;
      of->row0 = its(q.begin);
      of->T = its(q.end) - of->row0;
      s.len = its(q.len);
      break;
    }
    before = last;
    groups = __builtin_amdgcn_readlane(group, 63);
  }
  for (int* f : {&s.b, &s.h, &s.qg, &s.len, &s.p0, &s.splits, &s.first, &of->end, &of->group, &of->row0, &of->T})
    *f = __builtin_amdgcn_readfirstlane(*f);
  return s;
}

// A page that the table does not name is read as page 0 and lies past every
// limit: slots of a table are fewer than kNowhere, and kNowhere + 63 is an int.
constexpr int kNowhere = 0x7FFFFFC0;
struct Page {
  const uint8_t* block;
  int first;
};
template <int D>
__device__ __forceinline__ Page page_of(const kv4_cache& c, int id, int page, int h) {
  const bool named = static_cast<unsigned>(id) < static_cast<unsigned>(c.pages);
  return Page{static_cast<const uint8_t*>(c.data) +
                  (static_cast<size_t>(named ? id : 0) * c.Hk + h) * KvBlock<D>::kBytes,
              named ? page * kPage : kNowhere};
}

// Workgroups per CU that a wavefront's registers allow.  More was slower where
// it could be had: four instead of three with one tile at D = 128, for which
// the keys arrive late, 6% more time (16 sequences of 30000 .. 32768
// tokens, 12 rows a head); two instead of one with two tiles at D = 256, 27 against 26.
constexpr int attend_per_cu(int D, int MT) { return D == 256 && MT == 2 ? 1 : (D / 64 * MT <= 2 ? 3 : 2); }

// What bounds it: with one tile of queries, memory (16 sequences of 30000 ..
// 32768 tokens, four heads of 128: 290 MB in 52 us, 5.5 TB/s, where a large copy
// moves 4.7); with three, memory and the widening and softmax about equally
// (eight sequences of 120000 .. 131072 tokens: 578 MB and 99 GFLOP in 142 us; the
// VALU is busy for 59% of the cycles and the matrix unit for 29%); short
// sequences, latency: of one sequence of 8197 tokens' 16 us a page takes 2.6
// and the joining of four wavefronts' sums 3.
template <int D, int MT, class E, bool WINDOW, bool CHUNK>
__global__ __launch_bounds__(kThreads, attend_per_cu(D, MT)) void attend(const AttendArgs a) {
  constexpr int DB = D / 16;
  constexpr int kRow = D + 8;
  // With the most sums, keys that arrive during the softmax have no registers.
  constexpr bool kLateKeys = D == 128 && MT == 3;
  __shared__ __align__(16) _Float16 qs[MT * 16 * kRow];
  __shared__ float factor[MT * 16];
  __shared__ int limits[MT * 16];  // slots that each row sees
  __shared__ float stat[kWaves][MT * 16][2];
  __shared__ __align__(16) float sums[kWaves][D * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
  ChunkRows of{a.T, 0, 0, 0};
  Share sh = CHUNK ? chunk_share(a, MT * 16, lane, &of) : plan_share<WINDOW>(a, lane);
  if (!sh.any) return;
  const int b = sh.b, h = sh.h, qg = sh.qg, len = sh.len;
  const int T = CHUNK ? of.T : a.T, R = T * a.G;
  // The slots that row r sees without a window, and the least and the most of the workgroup's.
  const auto limit_of = [&](int r) {
    const int n = len - (T - 1 - r / a.G);
    return CHUNK && n < 0 ? 0 : n;
  };
  int least = len - (T - 1), most = len;
  kv4_rows rows = a.q;
  if constexpr (CHUNK) {
    const int r0 = qg * MT * 16, r1 = r0 + MT * 16 < R ? r0 + MT * 16 : R;
    least = limit_of(r0);
    most = limit_of(r1 - 1);
    rows.data = static_cast<const uint16_t*>(rows.data) + of.row0 * rows.row;
    rows.sequence = 0;
  }
  if (CHUNK && a.segments && sh.first == static_cast<int>(blockIdx.x) && threadIdx.x == 0)
    a.segments[of.group * a.c.Hk + h] = ChunkSegment{sh.first, sh.splits, of.row0, qg * MT * 16, R, {}};
  if (!CHUNK && a.split && sh.first == static_cast<int>(blockIdx.x) && threadIdx.x == 0)
    a.split[(b * a.c.Hk + h) * a.QG + qg] = int2{sh.first, sh.splits};
  const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.width;
  const View<WINDOW> view(a, least, most);
  if constexpr (CHUNK) sh.p1 = of.end < view.pages() ? of.end : view.pages();
  int page = sh.p0 + wave;  // of those that the sequence's rows see
  Queries<D, MT> q;
  q.load(rows, b, h, qg, a.G, R);
  KRegs<D> k;
  VRegs<D> v;
  Page now{nullptr, 0}, next{nullptr, 0};
  int next_id = 0;
  if (page < sh.p1) {
    now = page_of<D>(a.c, uniform_load(table, view.page(page)), view.page(page), h);
    next_id = uniform_load(table, view.page(page + kWaves < sh.p1 ? page + kWaves : page));
    k.load(now.block, lane);
    v.load(now.block, lane);
  }
  q.template put<E>(qs, factor);
  if (threadIdx.x < MT * 16) {
    const int r = qg * MT * 16 + threadIdx.x;
    limits[threadIdx.x] = r < R ? limit_of(r) : 0;
  }
  __syncthreads();

  float cm[MT], m[MT], l[MT], l_new[MT];  // l_new: what is not in l yet, of the last pages and of what rounding took
  f32x4 o[MT][DB];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    cm[mt] = fmaxf(a.scale * a.c.gk * kLog2e * factor[mt * 16 + c], kMinNormal);
    m[mt] = -INFINITY;
    l[mt] = 0.0f;
    l_new[mt] = 0.0f;
#pragma unroll
    for (int s = 0; s < DB; ++s) o[mt][s] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // The next page's keys are loaded once this page's have been used, and its
  // values once this page's have: each load has the other product to arrive in,
  // and no registers hold two pages.
  for (; page < sh.p1; page += kWaves) {
    const int first = now.first;
    // Past the last page the prefetch reads this one again.
    next = page + kWaves < sh.p1 ? page_of<D>(a.c, next_id, view.page(page + kWaves), h) : now;
    next_id = uniform_load(table, view.page(page + 2 * kWaves < sh.p1 ? page + 2 * kWaves : page));
    f32x4 s[4][MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[j][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int step = 0; step < D / 32; ++step) {
      f16x8 qf[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        qf[mt] = *reinterpret_cast<const f16x8*>(qs + (mt * 16 + c) * kRow + g * (D / 4) + step * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f16x8 kf = k.frag(j, step);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[j][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[mt], s[j][mt], 0, 0, 0);
      }
      // Without these fences the scheduler widens many steps' codes at once,
      // and their registers cost the second wavefront of a SIMD.
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!kLateKeys) k.load(next.block, lane);
    // Some row does not see the whole page.
    if (first > least - kPage || (WINDOW && first < most - a.window && first + kPage > a.sinks)) {
      int limit[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) limit[mt] = limits[mt * 16 + c];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (hidden<WINDOW>(a, first + 16 * j + 4 * g + e, limit[mt])) s[j][mt][e] = -INFINITY;
      clean_values<WINDOW, D, MT>(a, v, first, len, lane, limit, o);
    }
    bool grow = false;
    float top[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float t = s[0][mt][0];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t = fmaxf(t, s[j][mt][e]);
      top[mt] = max_over_rows(t) * cm[mt];
      grow |= top[mt] > m[mt] + kSlack;
    }
    if (__any(grow)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const bool up = top[mt] > m[mt] + kSlack;
        const float to = up ? top[mt] : m[mt];
        const float alpha = up ? __builtin_amdgcn_exp2f(m[mt] - to) : 1.0f;
        m[mt] = to;
        l[mt] *= alpha;
        l_new[mt] *= alpha;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[mt][d] *= alpha;
      }
    }
    f16x8 p[2][MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const float lifted = m[mt] == -INFINITY ? 0.0f : m[mt] - kLift;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][mt][e], cm[mt], -lifted));
          l_new[mt] += w;
          p[j / 2][mt][(j % 2) * 4 + e] = static_cast<_Float16>(w);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    // A long share's slots may each be too small for the sum of the pages before (512 sequences of 4000 pages, most weight in
    // the first slot: the log-sum was off by 1.6e-4 with one sum).  So l grows by a page at a time, and what its rounding takes
    // goes into the next; with three tiles of rows, which the VALU bounds, by four pages (120000 slots of four rows of 12
    // heads: 153 us, page by page 156; with two tiles at D = 256, eight rows of six, 2000 slots, 39.5 and 39.1 with the weights).
    if (WINDOW || MT < 3 || (page / kWaves) % 4 == 3) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float more = l[mt] + l_new[mt];
        l_new[mt] -= more - l[mt];
        l[mt] = more;
      }
    }
    if constexpr (kLateKeys) k.load(next.block, lane);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f16x2 vs[4];  // scales of the token pairs: tile 2u tokens (0, 1), (2, 3), tile 2u + 1 the same
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        vs[2 * t] = e4m3x2<false>(v.scales[2 * u + t]);
        vs[2 * t + 1] = e4m3x2<true>(v.scales[2 * u + t]);
      }
#pragma unroll
      for (int half = 0; half < (D == 256 ? 2 : 1); ++half) {
        u32x2 pr[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) pr[t] = v.pair(2 * u + t / 2, t % 2, half);
#pragma unroll
        for (int d = 0; d < (D == 64 ? 4 : 8); ++d) {
          f16x8 vf;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const f16x2 x = e2m1_pos(pr[t], d) * vs[t];
            vf[2 * t] = x.x;
            vf[2 * t + 1] = x.y;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            o[mt][half * 8 + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p[u][mt], o[mt][half * 8 + d], 0, 0, 0);
          if (d % 2) __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    v.load(next.block, lane);
    now = next;
  }

  // The wavefronts' sums meet in LDS, one group of 16 queries at a time.
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float total = sum_over_rows(l[mt] + l_new[mt]);
    if (g == 0) {
      stat[wave][mt * 16 + c][0] = m[mt];
      stat[wave][mt * 16 + c][1] = total;
    }
  }
  for (int mt = 0; mt < MT; ++mt) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MT; ++k)
      if (k == mt) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
          *reinterpret_cast<f32x4*>(&sums[wave][(d * 16 + c) * 16 + 4 * g]) = o[k][d];
      }
    __syncthreads();
    const int row = threadIdx.x / 16, at = threadIdx.x % 16;  // query, and the positions at * DB ..
    const int local = mt * 16 + row, r = qg * MT * 16 + local;
    if (r < R) {
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, stat[w][local][0]);
      float f[kWaves], total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = mm == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(stat[w][local][0] - mm);
        total += f[w] * stat[w][local][1];
      }
      const int t = r / a.G;
      const size_t at_row = ((CHUNK ? static_cast<size_t>(of.row0) : static_cast<size_t>(b) * a.T) + t) * a.Hq + h * a.G + r % a.G;
      const size_t at_part = (static_cast<size_t>(blockIdx.x) * MT * 16 + local);
      const float inv = sh.splits > 1 ? 1.0f : (mm == -INFINITY ? 0.0f : a.c.gv / total);
      float x[DB];
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += f[w] * sums[w][(d * 16 + row) * 16 + at];
        x[d] = v * inv;
      }
      if (sh.splits > 1) {
#pragma unroll
        for (int d = 0; d < DB; ++d) a.part[at_part * D + at * DB + d] = x[d];
        if (at == 0) {
          a.stat[at_part * 2] = mm;
          a.stat[at_part * 2 + 1] = total;
        }
      } else {
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at_row * D + at * DB);
#pragma unroll
        for (int d = 0; d < DB; d += 2) dst[d / 2] = elem_pack<E>(x[d], x[d + 1]);
        if (at == 0 && a.lse) a.lse[at_row] = log_sum(mm, total);
      }
    }
  }
}

// Adds the shares of split segments.  A workgroup has one query row: D / 4
// threads with four positions each take every kSets-th share, eight shares'
// loads at a time, and the sets meet in LDS.  33 shares of 384 rows (one
// sequence of 8197 tokens, eight rows of 48 heads): 9.7 us with one set, 5.2
// with eight.
template <int D, int MT, class E, bool CHUNK>
__global__ __launch_bounds__(kThreads) void attend_join(const AttendArgs a) {
  constexpr int kPer = D / 4, kSets = kThreads / kPer, kBatch = 8;
  __shared__ f32x4 sums[kSets][kPer];
  __shared__ float2 stats[kSets];
  const int segment = blockIdx.x, local = blockIdx.y;
  int h, r, stride;
  size_t token0;  // the first of the segment's sequence, among all rows
  int2 split;
  if constexpr (CHUNK) {
    if (segment / a.c.Hk >= *a.count) return;
    const ChunkSegment s = a.segments[segment];
    h = segment % a.c.Hk;
    r = s.r0 + local;
    stride = a.c.Hk;
    token0 = s.row0;
    split = int2{s.first, s.splits};
    if (r >= s.R) return;
  } else {
    const int qg = segment % a.QG, b = segment / a.QG / a.c.Hk;
    h = segment / a.QG % a.c.Hk;
    r = qg * MT * 16 + local;
    stride = a.c.Hk * a.QG;
    token0 = static_cast<size_t>(b) * a.T;
    if (r >= a.T * a.G) return;
    split = a.split[segment];
  }
  if (split.y <= 1) return;
  const int set = threadIdx.x / kPer, at = threadIdx.x % kPer;
  const auto row = [&](int s) { return (static_cast<size_t>(split.x) + static_cast<size_t>(s) * stride) * (MT * 16) + local; };
  float mm = -INFINITY, total = 0.0f;
  f32x4 x{0.0f, 0.0f, 0.0f, 0.0f};
  // A part's reference maximum, sum and values.  One without weight has zeros, and
  // one with nothing but NaN scores the same maximum, -inf, but a NaN sum and values:
  // both are added, times 0.
  const auto add = [&](float m, float l, f32x4 v) {
    const float to = fmaxf(mm, m), about = to == -INFINITY ? 0.0f : to;
    const float f0 = __builtin_amdgcn_exp2f(mm - about), f = __builtin_amdgcn_exp2f(m - about);
    mm = to;
    total = total * f0 + f * l;
    x = x * f0 + f * v;
  };
  for (int s0 = set; s0 < split.y; s0 += kBatch * kSets) {
    float2 st[kBatch];
    f32x4 v[kBatch];
#pragma unroll
    for (int s = 0; s < kBatch; ++s) {
      const size_t p = row(s0 + s * kSets < split.y ? s0 + s * kSets : s0);
      st[s] = *reinterpret_cast<const float2*>(a.stat + p * 2);
      v[s] = *reinterpret_cast<const f32x4*>(a.part + p * D + at * 4);
    }
#pragma unroll
    for (int s = 0; s < kBatch; ++s)
      if (s0 + s * kSets < split.y) add(st[s].x, st[s].y, v[s]);
  }
  sums[set][at] = x;
  if (at == 0) stats[set] = float2{mm, total};
  __syncthreads();
  if (set != 0) return;
#pragma unroll
  for (int s = 1; s < kSets; ++s) add(stats[s].x, stats[s].y, sums[s][at]);
  const size_t at_row = (token0 + r / a.G) * a.Hq + h * a.G + r % a.G;
  x *= mm == -INFINITY ? 0.0f : a.c.gv / total;
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at_row * D + at * 4) =
      u32x2{elem_pack<E>(x[0], x[1]), elem_pack<E>(x[2], x[3])};
  if (at == 0 && a.lse) a.lse[at_row] = log_sum(mm, total);
}

// ---- weights ----------------------------------------------------------------
// The scores again, from the keys alone, in the other orientation (queries as
// rows of the result): a lane's column is its token, and the sum over a head's
// rows is a sum of its own values and of four lanes.
// The log-sum is known only when a row's last share is done, so the keys are
// read twice; keeping the scores instead would move 48 bytes a token and head
// each way for 12 rows, the keys are 72.  With few rows a head (up to 0.07 D) the
// scores would be the smaller; that form is not built.  Bound by memory: 16
// sequences of 30000 .. 32768 tokens, four heads of 128, 161 MB in 32 us (5 TB/s).
struct WeightArgs {
  kv4_cache c;
  kv4_rows q;
  const float* lse;
  const float* acc;
  float* out;
  int T, Hq, G, per;  // per: pages per workgroup
  float scale;
};

template <int D, int MT, class E>
__global__ __launch_bounds__(kThreads) void add_weights(const WeightArgs a) {
  constexpr int kRow = D + 8;
  __shared__ __align__(16) _Float16 qs[MT * 16 * kRow];
  __shared__ float factor[MT * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, c = lane & 15;
  const int groups = (a.c.width + a.per - 1) / a.per;
  int i = blockIdx.x;
  const int chunk = i % groups;
  i /= groups;
  const int h = i % a.c.Hk, b = i / a.c.Hk;
  const int len = kv_len_uniform(a.c, b), R = a.T * a.G;
  const int p0 = chunk * a.per, p1 = p0 + a.per < a.c.width ? p0 + a.per : a.c.width;
  const int used = (len + kPage - 1) / kPage, end = used < p1 ? used : p1;  // pages from `end` on only get zeros
  const float* acc = a.acc + (static_cast<size_t>(b) * a.c.Hk + h) * a.c.width * kPage;
  float* out = a.out + (static_cast<size_t>(b) * a.c.Hk + h) * a.c.width * kPage;
  const int32_t* table = a.c.table + static_cast<size_t>(b) * a.c.width;
  for (int page = (end > p0 ? end : p0) + wave; page < p1; page += kWaves) out[page * kPage + lane] = 0.0f;
  if (p0 >= end) return;
  // Rows in groups of MT * 16; the first group also brings acc along.
  for (int qg = 0; qg * MT * 16 < R; ++qg) {
    Queries<D, MT> q;
    q.load(a.q, b, h, qg, a.G, R);
    KRegs<D> k;
    Page now{nullptr, 0};
    if (p0 + wave < end) {
      now = page_of<D>(a.c, uniform_load(table, p0 + wave), p0 + wave, h);
      k.load(now.block, lane);
    }
    __syncthreads();
    q.template put<E>(qs, factor);
    float sub[MT][4];
    int limit[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = qg * MT * 16 + mt * 16 + 4 * g + e;
        limit[mt][e] = r < R ? len - (a.T - 1 - r / a.G) : 0;
        const float lse = r < R ? a.lse[(static_cast<size_t>(b) * a.T + r / a.G) * a.Hq + h * a.G + r % a.G] : 0.0f;
        // A row of -inf scores only has no weight, and -inf minus itself is NaN.
        sub[mt][e] = lse == -INFINITY ? INFINITY : lse * kLog2e;
      }
    __syncthreads();
    float cm[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) cm[mt][e] = fmaxf(a.scale * a.c.gk * kLog2e * factor[mt * 16 + 4 * g + e], kMinNormal);
    for (int page = p0 + wave; page < end; page += kWaves) {
      const int first = now.first, slot = page * kPage + lane;
      const float before = slot < len ? (qg == 0 ? acc[slot] : out[slot]) : 0.0f;
      const bool more = page + kWaves < end;
      if (more) now = page_of<D>(a.c, uniform_load(table, page + kWaves), page + kWaves, h);
      f32x4 s[4][MT];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) s[j][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int step = 0; step < D / 32; ++step) {
        f16x8 qf[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          qf[mt] = *reinterpret_cast<const f16x8*>(qs + (mt * 16 + c) * kRow + g * (D / 4) + step * 8);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f16x8 kf = k.frag(j, step);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            s[j][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qf[mt], kf, s[j][mt], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // as in attend
      }
      if (more) k.load(now.block, lane);
      float mine = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float w = 0.0f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][mt][e], cm[mt][e], -sub[mt][e]));
            w += first + 16 * j + c < limit[mt][e] ? p : 0.0f;
          }
        w = sum_over_rows(w);
        mine = j == g ? w : mine;  // lane 16 g + c keeps token 16 g + c
      }
      out[slot] = slot < len ? before + mine : 0.0f;
    }
  }
}

// Most tiles of 16 query rows that a wavefront's registers hold: a tile takes
// D / 4 of them for its sums and 16 for a page's scores.
constexpr int max_tiles(int D) { return D == 256 ? 2 : 3; }

// The weights have no sums of values to hold.
constexpr int kWeightTiles = 3;

template <int MOST, class F>
void by_tiles(int tiles, F f) {
  if (tiles == 1) f(std::integral_constant<int, 1>());
  else if (tiles == 2) f(std::integral_constant<int, 2>());
  else if constexpr (MOST > 2) f(std::integral_constant<int, 3>());
}

// f(head size, tiles, type); `most` gives the most tiles of a head size.
template <class M, class F>
hipError_t by_shape(int D, int type, int tiles, M most, F f) {
  const auto run = [&](auto d) {
    by_tiles<most(d())>(tiles, [&](auto mt) {
      if (type == SKINNY_F16) f(d, mt, F16());
      else f(d, mt, BF16());
    });
  };
  if (D == 64) run(std::integral_constant<int, 64>());
  else if (D == 128) run(std::integral_constant<int, 128>());
  else run(std::integral_constant<int, 256>());
  return hipGetLastError();
}

}  // namespace

// Query rows of a head go in the fewest groups of at most max_tiles(D) tiles,
// of equal size.  The grid is what the CUs hold at once, so that no workgroup
// starts when the others are done, or two shares per segment where that is more.
// Four times what the CUs hold in place of the latter: 128 sequences of 1 ..
// 8000 tokens, four heads of 128, one row, 89 us against 71, of 8000 each 135
// against 108, with four rows 134 against 117; seven batches of a few long and
// many short sequences took from 2% less to 52% more.
//
// A share has a page per wavefront at least, and with one tile of queries two, so
// that up to 512 tokens need no join (301 tokens: 6.7 us in one launch; 600, which
// do: 10 to 11).  Longer sequences lose and gain about as much.  Two pages against
// one, one tile, four heads of 128: one sequence of 8197 tokens 12.1 us against
// 11.1, four of 8000 .. 9000 14.3 against 14.9, 32 of up to 20000 44.1 against 44.3;
// three tiles: 8197 tokens 18.8 against 19.2, 2000 tokens 17.0 against 16.1.
//
// With a window a sequence's rows see at most the pages of window + T - 1 slots in
// a row and those of the sinks, and the plan goes by these instead of the width.
// A call that is split has a page per wavefront then: one sequence, a window of
// 1024, 10.4 us with five shares a head, 11.6 with two, 12.9 in one launch; 48
// sequences within 4096, 29.6 either way.
AttendPlan kv4_attend_plan(int B, int T, int Hq, int Hk, int D, int width, int window, int sinks) {
  AttendPlan p;
  if (window) {
    const int64_t pages = (static_cast<int64_t>(window) + T + 61) / kPage + 1 + (static_cast<int64_t>(sinks) + kPage - 1) / kPage;
    width = pages < width ? static_cast<int>(pages) : width;
  }
  constexpr int kCUs = 256;
  const int tiles = (T * (Hq / Hk) + 15) / 16;
  p.QG = (tiles + max_tiles(D) - 1) / max_tiles(D);
  p.MT = (tiles + p.QG - 1) / p.QG;
  p.least = p.MT == 1 ? 2 * kWaves : kWaves;
  const int64_t segments = static_cast<int64_t>(B) * Hk * p.QG;
  p.split = width > p.least;
  if (window) p.least = kWaves;
  int64_t grid = segments;
  if (p.split) {
    grid = kCUs * attend_per_cu(D, p.MT);
    grid = grid < 2 * segments ? 2 * segments : grid;
    const int64_t per_segment = static_cast<int64_t>(B) * ((width + p.least - 1) / p.least) * Hk * p.QG;
    grid = grid < per_segment ? grid : per_segment;
  }
  p.grid = grid;
  const size_t rows = static_cast<size_t>(grid) * p.MT * 16;
  p.split_off = kSyncBytes;
  p.stat_off = p.split_off + static_cast<size_t>((segments * sizeof(int2) + 255) / 256 * 256);
  p.part_off = p.stat_off + rows * 8;
  p.total = p.split ? p.part_off + rows * D * 4 : 0;
  return p;
}

hipError_t launch_kv4_attention(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale, int window,
                                int sinks, void* out, float* lse, void* workspace, hipStream_t stream) {
  const AttendPlan p = kv4_attend_plan(c.B, T, Hq, c.Hk, c.D, c.width, window, sinks);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttendArgs a{c, q, out, lse, nullptr, nullptr, nullptr, T, Hq, Hq / c.Hk, p.QG, p.least, scale, window, sinks, nullptr, 0, nullptr, nullptr};
  if (p.split) {
    a.part = reinterpret_cast<float*>(ws + p.part_off);
    a.stat = reinterpret_cast<float*>(ws + p.stat_off);
    a.split = reinterpret_cast<int2*>(ws + p.split_off);
  }
  const unsigned segments = static_cast<unsigned>(c.B * c.Hk * p.QG);
  return by_shape(c.D, type, p.MT, [](int D) constexpr { return max_tiles(D); }, [&](auto d, auto mt, auto e) {
    const dim3 grid(static_cast<unsigned>(p.grid));
    if (window) attend<d(), mt(), decltype(e), true, false><<<grid, kThreads, 0, stream>>>(a);
    else attend<d(), mt(), decltype(e), false, false><<<grid, kThreads, 0, stream>>>(a);
    if (p.split)
      attend_join<d(), mt(), decltype(e), false><<<dim3(segments, mt() * 16), kThreads, 0, stream>>>(a);
  });
}

// Chunks of few rows: as kv4_attention.  Over few pages every workgroup has all the
// pages of its rows, so that one launch does: the fewest tiles of rows per
// workgroup that leave no more workgroups than the CUs hold at once, as a page takes
// a wavefront the less.  Against the tiles of 256 rows of kv4_chunk.hip with their
// plan and join (D = 128, 8 heads of 4 query heads, 9 rows; us):
//   pages        4    16    32    64   128   256
//   this       7.0  11.1  16.7  27.0  47.3  87.3
//   the other 17.0  32.8  55.5  36.5  37.2  39.6
// and 16.1, 24.5, 40.3, 72.5 against 40.7, 64.7, 65.0, 74.9 with 256 rows and 16
// to 128 pages.  The two meet near 96 pages there and for D = 64 (29 us), and
// between 96 and 128 for D = 256.
//
// Over more pages, or with more groups, these are split into shares.  Of many pages a group of 48 rows
// (32 at D = 256) takes kGroup[D] ns a page and head of the whole card's time, a tile
// of 256 rows with few of them in use kTileOf[D], which has a plan and other
// beginnings to make up for, kFixed ns; shares are coarse where there are many groups.
// Split against tiles of 256 rows, four heads of 12 (128) or 6 (256), us:
//   sequences x rows, pages   D = 128: 128          512          2048    D = 256: 512
//   1 x 48                    17.9  39.0   24.5  46.7   38.5  82.0    33.4  78.0
//   1 x 252                   26.8  44.3   46.6  55.6    119  99.1    72.7  97.1
//   1 x 960                   42.9  49.4    104  85.7    332   252     226   167
//   16 x 48                   39.3  68.0   87.6   194    296   691     246   402
//   16 x 120 or 126           89.0  74.4    260   209    919   718     461   438
//   16 x 252                   126  91.4    391   254   1486   964     886   545
// Every workgroup looks through the lengths of all sequences, which costs more than
// it brings when these are many (8 heads of 4, rows of 8 tokens, up to 97 pages: 512
// sequences 1150 us against 1435 in tiles, 1024 3208 against 2746; up to 32 pages:
// 128 sequences 150 against 166, 256 367 against 302).
//
// A call goes one way, by its mean: 63 single tokens over 4096 slots beside a prompt
// of 2048 (32/8 heads of 128) have a tile each, 317 us, where the prompt alone takes
// 130 and the tokens 49.
SmallChunk kv4_small_chunk(int N, int B, int G, int Hk, int D, int64_t pages) {
  constexpr int kCUs = 256, kMostPages = 96, kFewSequences = 128, kMostSequences = 512;
  SmallChunk s{};
  if (B > kMostSequences) return s;
  const int64_t busy = N < B ? N : B, rows = static_cast<int64_t>(N) * G;  // sequences with rows
  const auto groups = [&](int height) { return (rows + busy * (height - 1)) / height; };
  if (pages <= kMostPages)
    for (int mt = 1; mt <= max_tiles(D); ++mt)
      if (groups(mt * 16) * Hk <= kCUs * attend_per_cu(D, mt)) {
        s.tiles = mt;
        s.groups = s.shares = groups(mt * 16);
        return s;
      }
  const int64_t mean = (rows + busy - 1) / busy;  // rows of a sequence
  const int mt = mean < max_tiles(D) * 16 ? static_cast<int>((mean + 15) / 16) : max_tiles(D);
  const int64_t tall = groups(mt * 16);
  if ((pages <= kMostPages && B > kFewSequences) || tall * (pages + 4) > INT32_MAX) return s;
  constexpr double kGroup[] = {1.6, 2.25, 3.2}, kTileOf[] = {3.9, 5.5, 11.3}, kFixed[] = {16000.0, 16000.0, 35000.0};
  const int size = D / 128;  // 0, 1, 2
  const int64_t whole = busy * ((mean + mt * 16 - 1) / (mt * 16));
  const double split = kGroup[size] * whole, tiled = kTileOf[size] * (busy * ((mean + 255) / 256));
  if (split * 1.15 > tiled && (whole * Hk > 128 || (split - tiled) * Hk * pages > kFixed[size])) return s;
  s.tiles = mt;
  s.groups = tall;
  const int64_t room = kCUs * attend_per_cu(D, mt) / Hk, most = tall * ((pages + kWaves - 1) / kWaves);
  s.shares = room < 2 * tall ? 2 * tall : room;
  s.shares = s.shares < most ? s.shares : most;
  const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  s.count_off = kSyncBytes;
  s.segment_off = s.count_off + 256;
  s.stat_off = s.segment_off + up(static_cast<size_t>(tall) * Hk * sizeof(ChunkSegment));
  s.part_off = s.stat_off + static_cast<size_t>(s.shares) * Hk * mt * 16 * 8;
  s.total = s.part_off + static_cast<size_t>(s.shares) * Hk * mt * 16 * D * 4;
  return s;
}

hipError_t launch_kv4_small_chunk(const kv4_cache& c, const void* q, int64_t row, int64_t head, const int32_t* starts, int N,
                                  int type, int Hq, float scale, int window, int sinks, void* out, float* lse, void* workspace,
                                  const SmallChunk& s, hipStream_t stream) {
  const int wide = window ? window : c.width * kPage;  // a window that leaves nothing out
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttendArgs a{c, {q, 0, row, head}, out, lse, nullptr, nullptr, nullptr, 0, Hq, Hq / c.Hk, 1, kWaves, scale, wide, sinks, starts, N, nullptr, nullptr};
  if (s.total) {
    a.part = reinterpret_cast<float*>(ws + s.part_off);
    a.stat = reinterpret_cast<float*>(ws + s.stat_off);
    a.segments = reinterpret_cast<ChunkSegment*>(ws + s.segment_off);
    a.count = reinterpret_cast<int*>(ws + s.count_off);
  }
  return by_shape(c.D, type, s.tiles, [](int D) constexpr { return max_tiles(D); }, [&](auto d, auto mt, auto e) {
    attend<d(), mt(), decltype(e), true, true><<<dim3(static_cast<unsigned>(s.shares * c.Hk)), kThreads, 0, stream>>>(a);
    if (s.total)
      attend_join<d(), mt(), decltype(e), true><<<dim3(static_cast<unsigned>(s.groups * c.Hk), mt() * 16), kThreads, 0, stream>>>(a);
  });
}

hipError_t launch_kv4_weights(const kv4_cache& c, const kv4_rows& q, int type, int T, int Hq, float scale,
                              const float* lse, const float* acc, float* acc_out, hipStream_t stream) {
  const int G = Hq / c.Hk, all = (T * G + 15) / 16, tiles = all < kWeightTiles ? all : kWeightTiles;
  const int64_t pages = static_cast<int64_t>(c.B) * c.Hk * c.width;
  // Pages of a workgroup: one per wavefront, and up to four where there are
  // enough for 1024 workgroups, which pays for the queries once.  One: 42.6 us,
  // two: 36.0, four: 33.2, eight: 32.2 (16 sequences of 30000 .. 32768 tokens, four
  // heads of 128, one row); 9.8, 12.7, 18.5 and 29.8 (one of 8197, eight rows).
  int64_t per = pages / 1024;
  per = per < kWaves ? kWaves : (per > 16 ? 16 : per);
  WeightArgs a{c, q, lse, acc, acc_out, T, Hq, G, static_cast<int>(per), scale};
  const int64_t groups = (c.width + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(c.B) * c.Hk * groups));
  return by_shape(c.D, type, tiles, [](int) constexpr { return kWeightTiles; }, [&](auto d, auto mt, auto e) {
    add_weights<d(), mt(), decltype(e)><<<grid, kThreads, 0, stream>>>(a);
  });
}

}  // namespace skinny
