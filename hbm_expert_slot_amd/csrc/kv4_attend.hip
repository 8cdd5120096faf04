// Attention of a few new tokens over the 4-bit key/value cache.
//
// For each row q of a sequence and query head, over the places j that the row sees:
//   s_j = scale q . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
// One pass over the pages keeps the running maximum m, the sum and o (fp32).
//
// A head's rows, all query heads that share it times all new tokens, are the
// columns of the 16x16x32 matrix products:  S^T = K Q^T,  O^T = V^T P^T.  The cache
// is read and widened once for up to 32 of them (16 with heads of 256); more columns
// are chunks of their own, which read the head's pages again.  The tokens of S^T that a lane
// gets are those whose P it has to supply to the second product, and the columns
// stay in their lanes, so neither P, the maxima nor the sums ever change lanes
// but for the four lanes of a column.
//
// NVFP4: a code times its E4M3 scale has 6 significant bits and is exact in
// fp16; queries are brought to [2^13, 2^14) by a power of two per row, which
// keeps bf16's 8 bits exact down to 2^-28 of the row's largest.  P is fp16 with
// 1 at 2^14, so that what is rounded below the format's range is below 2^-38 of
// the largest; its 11 bits are as many as the widest output has.
// MXFP4: the scales need bf16's exponent.  fp16 queries and P are split into two
// bf16 parts (16 bits), both multiplied.
//
// The pages of all sequences and heads form one list that is cut into equal
// parts, one per block, whatever the sequences' lengths are.  A part that has only
// some of a head's pages leaves its sums to a second kernel.
//
// What bounds it: HBM.  64 sequences of 717063 tokens in all, 8 key heads and 48 query
// heads of 128, NVFP4: 145 us, 5.7 TB/s (a copy of 1 GiB moves 5.14 TB/s), and 10 us to
// join.  One sequence of 131069 tokens, 64 query heads: 31 us, 4.9 TB/s, and 6 to join.
// MXFP4, the 64 sequences again: 137 us, with fp16 queries in two parts 156.
// With few pages per wavefront starting, the queries' widening and the join count:
// 97680 tokens of 16 sequences, 4 rows each, 8 query heads on each of 4, MXFP4: 32 us and
// 9 where HBM needs 10.  Sixteen rows each, 8 query heads on each of 8, NVFP4 (128
// columns, four chunks): 117 us and 36 to join, where the products need 42.
#include "kv4_device.h"

namespace sc {
namespace kv4 {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
// Parts of the list: as many blocks as run at a time, three per compute unit or two.
// (64 sequences of 717063 tokens: 512 parts 184 us, 768 parts 178, before pieces overlapped.)
constexpr int kMaxParts = 768;
// Pages up to which a head's are one block's, without a second kernel: four steps of a
// wavefront (one sequence of 100 tokens, the one that was measured: 10.7 us a call, with a list 13.4).
constexpr int kDirectPages = 8;
constexpr float kLog2e = 1.44269504088896340736f;

struct AttendArgs {
  Pool pool;
  Seqs seqs;
  const float* ks;
  const float* vs;
  const uint16_t* q;
  uint16_t* out;
  int64_t qs[3], os[3];     // strides: sequence, row, head
  int32_t rows, group;      // new tokens; query heads per key head
  int32_t cols, chunks;     // rows * group; column chunks of a head
  float scale;
  float* part;              // [2 * blocks][16 * NQ][D]: sums of pieces
  float* part_ml;           // [2 * blocks][16 * NQ][2]
  float* lse;               // [sequence][head][cols], base 2; null unless weights are kept
  int32_t nblocks, weight_blocks;
  bool direct;              // a block has all of one head, with no list
};

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

// The operands live until the result is there, so that it takes no register of theirs.
template <bool F16>
__device__ __forceinline__ f32x4 product(u32x4 a, u32x4 b, f32x4 c) {
  f32x4 d;
  if constexpr (F16)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  asm("" : "+v"(d) : "v"(a), "v"(b));
  return d;
}

template <int B>
__device__ __forceinline__ uint32_t widen_f16(uint32_t d) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, B));
}
template <int B>
__device__ __forceinline__ uint32_t widen_bf16(uint32_t d, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, B));
}
__device__ __forceinline__ uint32_t times(uint32_t a, f16x2 s) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) * s);
}
// The conversions take their scale's exponent field as E8M0: 0 is 2^-127, 255 NaN.
__device__ __forceinline__ float e8m0_field(uint32_t d, int byte) { return __uint_as_float((d >> (8 * byte) & 0xFF) << 23); }
// Two E4M3 scales (half W of d) as fp16, exactly.
template <int W>
__device__ __forceinline__ f16x2 scales2(uint32_t d) {
  return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)d, 1.0f, W));
}

// What a lane holds of a step, half a page of 32 tokens: see Layout.
constexpr int kStep = 32;
template <int D, int FMT>
struct Keys {
  typedef Layout<D, FMT> L;
  static constexpr int W = L::C * L::LaneDims / 8;     // words per tile of 16 tokens
  uint32_t q[2][W];
  uint32_t s[(L::SP + 1) / 2];                         // scales of both tiles
};
template <int D, int FMT>
struct Values {
  typedef Layout<D, FMT> L;
  static constexpr int W = L::C * L::VDims / 2;        // words per 16 tokens
  uint32_t q[2][W];
  u32x2 s[L::C];
};

// Pages are read once a call (twice with weights): past the caches.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* d, const uint8_t* p) {
  typedef __attribute__((ext_vector_type(N))) uint32_t V;
  const V v = __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = v[i];
}
template <>
__device__ __forceinline__ void load_words<1>(uint32_t* d, const uint8_t* p) {
  d[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
}

template <int D, int FMT>
__device__ __forceinline__ void load_keys(Keys<D, FMT>& p, const uint8_t* side, int half, int lane) {
  typedef Layout<D, FMT> L;
  const int r = lane & 15, g = lane >> 4;
  constexpr int B = L::LaneDims / 2;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < L::C; ++c)
      load_words<B / 4>(&p.q[t][c * (B / 4)], side + half * (16 * D) + (t * 16 + r) * (D / 2) + c * 64 + g * B);
  const uint8_t* s = side + L::kCodes + half * 2 * L::SP + (r * L::SL + (L::SL == 4 ? g : g >> 1)) * 4 * L::SP;
  if constexpr (L::SP == 1) p.s[0] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(s));
  else load_words<L::SP / 2>(p.s, s);
}
template <int D, int FMT>
__device__ __forceinline__ void load_values(Values<D, FMT>& p, const uint8_t* side, int half, int lane) {
  typedef Layout<D, FMT> L;
  const int n = lane & 15, g = lane >> 4;
  constexpr int B = L::VDims / 2;        // bytes of a token
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int c = 0; c < L::C; ++c)
      load_words<B>(&p.q[t][c * B], side + half * (16 * D) + (((t * 4 + g) * L::C + c) * 16 + n) * 4 * B);
#pragma unroll
  for (int c = 0; c < L::C; ++c) {
    const int s = c * (128 / L::G) + n * L::VDims / L::G;
    p.s[c] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(side + L::kCodes + (g * L::NS + s) * 16 + half * 8));
  }
}

// Operand words of tile T of the keys: words of chunk c, eight dimensions each.
template <int D, int FMT>
__device__ __forceinline__ void widen_keys(const Keys<D, FMT>& p, int t, u32x4 (&out)[Keys<D, FMT>::W]) {
  typedef Layout<D, FMT> L;
  constexpr int WC = L::LaneDims / 8, E = L::SP / L::C;     // words, scales of a chunk
#pragma unroll
  for (int w = 0; w < Keys<D, FMT>::W; ++w) {
    const int c = w / WC, e = c * E + (w % WC) * E / WC;    // the word's scale
    const int at = t * L::SP + e;                           // its byte
    const uint32_t q = p.q[t][w];
    if constexpr (FMT == kNv) {
      const f16x2 pair = at % 4 < 2 ? scales2<0>(p.s[at / 4]) : scales2<1>(p.s[at / 4]);
      const _Float16 h = at % 2 ? pair.y : pair.x;
      const f16x2 s = {h, h};
      out[w] = u32x4{times(widen_f16<0>(q), s), times(widen_f16<1>(q), s), times(widen_f16<2>(q), s),
                     times(widen_f16<3>(q), s)};
    } else {
      const float s = e8m0_field(p.s[at / 4], at % 4);
      out[w] = u32x4{widen_bf16<0>(q, s), widen_bf16<1>(q, s), widen_bf16<2>(q, s), widen_bf16<3>(q, s)};
    }
  }
}

// Two words of two tokens side by side: a and b hold eight (D = 64: four)
// dimensions of a token each; word i of the result pairs dimension i of both.
template <int FMT, int N>
__device__ __forceinline__ void pair_tokens(uint32_t a, uint32_t b, uint32_t sab, int half, uint32_t (&out)[N]) {
  if constexpr (FMT == kNv) {
    const uint32_t even = (a & 0x0F0F0F0Fu) | (b << 4 & 0xF0F0F0F0u);
    const uint32_t odd = (a >> 4 & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
    const f16x2 s = half ? scales2<1>(sab) : scales2<0>(sab);
    out[0] = times(widen_f16<0>(even), s);
    out[1] = times(widen_f16<0>(odd), s);
    out[2] = times(widen_f16<1>(even), s);
    out[3] = times(widen_f16<1>(odd), s);
    if constexpr (N == 8) {
      out[4] = times(widen_f16<2>(even), s);
      out[5] = times(widen_f16<2>(odd), s);
      out[6] = times(widen_f16<3>(even), s);
      out[7] = times(widen_f16<3>(odd), s);
    }
  } else {
    const float sa = e8m0_field(sab, 2 * half), sb = e8m0_field(sab, 2 * half + 1);
    const auto two = [&](uint32_t x, uint32_t y, int i) {
      out[i] = __builtin_amdgcn_perm(y, x, 0x05040100u);
      out[i + 1] = __builtin_amdgcn_perm(y, x, 0x07060302u);
    };
    two(widen_bf16<0>(a, sa), widen_bf16<0>(b, sb), 0);
    two(widen_bf16<1>(a, sa), widen_bf16<1>(b, sb), 2);
    if constexpr (N == 8) {
      two(widen_bf16<2>(a, sa), widen_bf16<2>(b, sb), 4);
      two(widen_bf16<3>(a, sa), widen_bf16<3>(b, sb), 6);
    }
  }
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) {
  if (f16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
// What bf16 leaves of two numbers (NaN of one that is not finite).
__device__ __forceinline__ uint32_t rest16(float a, float b, uint32_t hi) {
  const float x = a - __uint_as_float(hi << 16), y = b - __uint_as_float(hi & 0xFFFF0000u);
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
}

// Over the four lanes of a column.
__device__ __forceinline__ float max_over_g(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_g(float v) {
  v = swap_sum<32>(v, v);
  return swap_sum<16>(v, v);
}

// The columns of one tile: column l % 16 of lane l, and its share of the dimensions.
template <int D, int FMT, bool HALF>
struct Queries {
  typedef Layout<D, FMT> L;
  static constexpr int W = Keys<D, FMT>::W, P = FMT == kMx && HALF ? 2 : 1;
  u32x4 x[W][P];
  float factor;     // of the products, to get scores in base 2
  int row;          // of the column; beyond the last: it sees what the last does
};
// As they are in memory, and then as operands.
template <int D, int FMT, bool HALF>
__device__ __forceinline__ void fetch_queries(Queries<D, FMT, HALF>& q, const AttendArgs& a, int b, int head, int first,
                                              int lane) {
  typedef Layout<D, FMT> L;
  constexpr int WC = L::LaneDims / 8;
  const int col = min(first + (lane & 15), a.cols - 1), g = lane >> 4;
  q.row = col / a.group;
  const uint16_t* p = a.q + b * a.qs[0] + q.row * a.qs[1] + ((int64_t)head * a.group + col % a.group) * a.qs[2];
#pragma unroll
  for (int w = 0; w < Queries<D, FMT, HALF>::W; ++w)
    __builtin_memcpy(&q.x[w][0], p + w / WC * 128 + g * L::LaneDims + w % WC * 8, 16);
}
template <int D, int FMT, bool HALF>
__device__ __forceinline__ void widen_queries(Queries<D, FMT, HALF>& q, const AttendArgs& a, int first, int lane) {
  typedef Queries<D, FMT, HALF> Q;
  const bool in = first + (lane & 15) < a.cols;
  float v[Q::W][8];
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < Q::W; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t raw = q.x[w][0][e / 2] >> (e % 2 * 16) & 0xFFFF;
      v[w][e] = HALF ? (float)__builtin_bit_cast(_Float16, (uint16_t)raw) : __uint_as_float(raw << 16);
      if (!in) v[w][e] = 0.0f;
      top = fmaxf(top, fabsf(v[w][e]));
    }
  float up = 1.0f;
  q.factor = a.scale * kLog2e;
  if constexpr (FMT == kNv) {
    const float ks = a.ks ? *a.ks : 1.0f;
    const bool sane = ks >= 0.0f && ks < INFINITY;
    q.factor *= sane ? ks : 1.0f;
    top = max_over_g(top);
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = top > 0.0f && e < 128 ? max(e, -100) : 13;
    up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
    q.factor *= __uint_as_float((uint32_t)(127 + e - 13) << 23);
    if (!sane) up = NAN;        // a scale that cannot be: NaN scores, but where the mask replaces them
  }
  q.factor = fmaxf(q.factor, 1e-37f);       // masked scores are -inf times this
#pragma unroll
  for (int w = 0; w < Q::W; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[w][2 * e] * up, y = v[w][2 * e + 1] * up;
      q.x[w][0][e] = pack16(x, y, FMT == kNv);
      if constexpr (Q::P == 2) q.x[w][1][e] = rest16(x, y, q.x[w][0][e]);      // NaN: its scores are NaN or infinite anyway
    }
}

template <int FMT>
__device__ __forceinline__ bool nan_scale(uint32_t byte) {
  return FMT == kNv ? (byte & 0x7F) == 0x7F : byte == 0xFF;
}
template <int FMT>
__device__ __forceinline__ uint32_t without_nan(uint32_t four) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    if (nan_scale<FMT>(four >> i & 0xFF)) four &= ~(0xFFu << i);
  return four;
}

// The list of pages.  Its order: sequence, head and chunk, page.
__device__ __forceinline__ int pages_of(const Seqs& s, int b) {
  const int n = b < s.n ? length_of(s, b) : 0;
  return n > 0 ? (n + kPage - 1) / kPage : 0;
}
__device__ __forceinline__ int64_t of_lane(int64_t v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
struct List {
  const Seqs& s;
  int lane, own, upto;             // of the first 64 sequences: pages, and pages up to each
  int64_t total;
  __device__ __forceinline__ List(const Seqs& seqs, int l) : s(seqs), lane(l) {
    own = pages_of(s, lane);
    upto = wave_scan(own);
    total = __builtin_amdgcn_readlane(upto, 63);
    for (int i = 64; i < s.n; i += 64) total += __builtin_amdgcn_readlane(wave_scan(pages_of(s, i + lane)), 63);
  }
  // Pages of the sequences before b.
  __device__ __forceinline__ int64_t before(int b) const {
    int64_t sum = 0;
    for (int i = 0; i <= b; i += 64) {
      const int x = i ? wave_scan(pages_of(s, i + lane)) : upto;
      if (b >= i + 64) sum += __builtin_amdgcn_readlane(x, 63);
      else if (b > i) sum += __builtin_amdgcn_readlane(x, b - i - 1);
    }
    return sum;
  }
  // The sequence that unit u lies in, its pages, and the units before it; `per` units per page of a sequence.
  __device__ __forceinline__ int at(int64_t u, int per, int& pages, int64_t& units_before) const {
    int64_t sum = 0;
    for (int i = 0; i < s.n; i += 64) {
      const int n = i ? pages_of(s, i + lane) : own;
      const int64_t x = sum + (i ? wave_scan(n) : upto);
      const uint64_t beyond = __ballot(x * per > u);
      if (beyond) {
        const int l = __builtin_ctzll(beyond);
        pages = __builtin_amdgcn_readlane(n, l);
        units_before = (of_lane(x, l) - pages) * per;
        return i + l;
      }
      sum = of_lane(x, 63);
    }
    pages = 0;
    units_before = sum * per;
    return s.n;
  }
};
// A sequence's pages, the entries of 64 at a time in a wavefront's lanes.
struct Table {
  const Pool& pool;
  const Seqs& s;
  int b, lane, first, entry;
  __device__ __forceinline__ Table(const Pool& p, const Seqs& seqs, int l) : pool(p), s(seqs), lane(l) {}
  __device__ __forceinline__ void open(int seq, int at) {
    b = seq;
    first = at;
    entry = page_at(pool, s, b, at + lane);
  }
  __device__ __forceinline__ int page(int index) {
    if (index < first || index >= first + 64) {
      first = index;
      entry = page_at(pool, s, b, index + lane);
    }
    return __builtin_amdgcn_readlane(entry, index - first);
  }
};
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {      // of numbers >= 0; most fit 32 bits
  return (a | b) >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : (int64_t)((uint64_t)a / (uint64_t)b);
}
// The list in equal parts.  The longer ones are spread evenly, so heads of one
// length whose number divides that of the parts begin with one.
struct Cuts {
  int64_t units, each;
  uint32_t rest;
  int parts;
  __device__ __forceinline__ Cuts(int64_t n, int p) : units(n), each(quotient(n, p)), rest((uint32_t)(n - each * p)), parts(p) {}
  __device__ __forceinline__ int64_t start(int part) const { return each * part + rest * (uint32_t)part / (uint32_t)parts; }
  // the part that holds unit u
  __device__ __forceinline__ int holds(int64_t u) const { return (int)quotient((u + 1) * parts - 1, units); }
};

template <bool HALF>
__device__ __forceinline__ uint16_t narrow(float v) {
  if constexpr (HALF) return __builtin_bit_cast(uint16_t, (_Float16)v);
  else return __builtin_bit_cast(uint16_t, (__bf16)v);
}
// Base-2 logarithm of the sum of exponentials; P counts from 2^14 with NVFP4.
template <int FMT>
__device__ __forceinline__ float lse2_of(float m, float l) {
  return l == 0.0f ? -INFINITY : m + __builtin_amdgcn_logf(l) - (FMT == kNv ? 14.0f : 0.0f);
}

// The wavefronts of a block take its steps in turn.  A step's keys are fetched while
// the step before is in its softmax and second product, its values during its own
// first product: into the registers that the step before has just left.
template <int D, int FMT, bool HALF, int NQ>
__global__ __launch_bounds__(kThreads, NQ == 1 && D <= 128 ? 3 : 2) void k_kv4_attend(AttendArgs a) {
  typedef Layout<D, FMT> L;
  constexpr bool F16 = FMT == kNv;
  constexpr int W = Keys<D, FMT>::W, VD = L::VDims, NO = L::C * VD;     // output tiles
  constexpr int QP = Queries<D, FMT, HALF>::P, PP = FMT == kMx ? 2 : 1;
  // m is the maximum that P counts from; it follows the scores once they exceed it by kSlack
  constexpr float kShift = F16 ? 14.0f : 0.0f, kSlack = F16 ? 1.875f : 8.0f;
  constexpr int kRow = D + 4;
  __shared__ __align__(16) float red[NQ][kWaves][16][kRow];
  __shared__ f32x2 red_ml[NQ][kWaves][16];
  const int lane = threadIdx.x & 63, wave = wave_index(), g = lane >> 4;
  const int per = a.pool.heads * a.chunks;
  const List list(a.seqs, lane);
  const int64_t units = list.total * per;
  const Cuts cuts(units, a.nblocks);
  const int64_t u0 = a.direct ? blockIdx.x : cuts.start(blockIdx.x);
  const int64_t u1 = a.direct ? u0 + 1 : cuts.start(blockIdx.x + 1);
  if (u0 >= u1) return;
  Queries<D, FMT, HALF> q[NQ];
  Keys<D, FMT> keys;
  Values<D, FMT> vals;
  int b, n, head, chunk, p0, p1, len;      // the piece: pages p0 .. p1 of the n of a head and chunk
  int t0, t1, page;                        // the wavefront's steps, the page of the next
  Table table(a.pool, a.seqs, lane);
  const auto head_at = [&](int pg) { return a.pool.pages + ((int64_t)max(pg, 0) * a.pool.heads + head) * L::kHead; };
  // finds the piece at unit u and sends for what it begins with
  const auto begin = [&](int64_t u) {
    int hc;
    if (a.direct) {
      b = blockIdx.x / per;
      hc = blockIdx.x % per;
      n = p1 = pages_of(a.seqs, b);
      p0 = 0;
    } else {
      int64_t before;
      b = list.at(u, per, n, before);
      hc = (int)quotient(u - before, n);
      p0 = (int)(u - before - (int64_t)hc * n);
      p1 = (int)(u1 - u < n - p0 ? p0 + (u1 - u) : n);
    }
    head = hc / a.chunks;
    chunk = hc % a.chunks;
    len = length_of(a.seqs, b);
    t0 = 2 * p0 + wave;
    t1 = min(2 * p1, (len + kStep - 1) / kStep);
    page = -1;
    if (t0 < t1) {
      table.open(b, t0 >> 1);
      page = table.page(t0 >> 1);
      load_keys(keys, head_at(page), t0 & 1, lane);
      load_values(vals, head_at(page) + L::kSide, t0 & 1, lane);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) fetch_queries(q[i], a, b, head, (chunk * NQ + i) * 16, lane);
  };
  begin(u0);
  if (n == 0) {      // only without a list: no tokens, or a length that cannot be
    const int cols = min(a.cols - chunk * NQ * 16, NQ * 16);
    for (int i = threadIdx.x; i < cols * D; i += kThreads) {
      const int at = chunk * NQ * 16 + i / D;
      a.out[b * a.os[0] + at / a.group * a.os[1] + (head * a.group + at % a.group) * a.os[2] + i % D] =
          narrow<HALF>(len < 0 ? NAN : 0.0f);
      if (a.lse && i % D == 0) a.lse[((int64_t)b * a.pool.heads + head) * a.cols + at] = len < 0 ? NAN : -INFINITY;
    }
    return;
  }
  for (int64_t u = u0; u < u1;) {
    const int seen_by_all = len - a.rows + 1;      // places that every row sees
    float m[NQ], l[NQ];
    f32x4 o[NQ][NO];
#pragma unroll
    for (int i = 0; i < NQ; ++i) widen_queries(q[i], a, (chunk * NQ + i) * 16, lane);
    bool careful = false;      // values that only some rows see are not finite: in a second pass
  again:
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < NO; ++j) o[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int t = t0; t < t1; t += kWaves) {
      f32x4 s[NQ][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        u32x4 kw[W];
        widen_keys(keys, x, kw);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          s[i][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int y = 0; y < QP; ++y)
              s[i][x] = product<F16>(kw[w], q[i].x[w][y], s[i][x]);
        }
      }
      const int tn = t + kWaves < t1 ? t + kWaves : t;
      const int next = table.page(tn >> 1);
      load_keys(keys, head_at(next), tn & 1, lane);
      if (page < 0) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) s[i][0] = s[i][1] = f32x4{NAN, NAN, NAN, NAN};
      }
      if ((t + 1) * kStep > seen_by_all) {
        const int base = t * kStep + 4 * g;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (base + x * 16 + e >= seen_by_all + q[i].row) s[i][x][e] = -INFINITY;
        // scales behind the last token may be anything: zeros
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int left = min(max(len - (base + x * 16), 0), 4);
          const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1;
#pragma unroll
          for (int c = 0; c < L::C; ++c) {
            vals.s[c][x] &= keep;
            if (careful) vals.s[c][x] = without_nan<FMT>(vals.s[c][x]);
          }
        }
      }
      u32x4 pw[NQ][PP];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        float top = s[i][0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[i][e / 4][e % 4]);
        top = max_over_g(top) * q[i].factor;
        if (__any(top > m[i] + kSlack)) {
          const float mn = top > m[i] + kSlack ? top : m[i];       // of this column, whatever the others do
          const float f = __builtin_amdgcn_exp2f(m[i] - (mn == -INFINITY ? 0.0f : mn));
          l[i] *= f;
#pragma unroll
          for (int j = 0; j < NO; ++j) o[i][j] *= f;
          m[i] = mn;
        }
        const float mu = (m[i] == -INFINITY ? 0.0f : m[i]) - kShift;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i][x][e] = __builtin_amdgcn_exp2f(fmaf(s[i][x][e], q[i].factor, -mu));
            l[i] += s[i][x][e];
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f32x4& x = s[i][e / 2];
          pw[i][0][e] = pack16(x[e % 2 * 2], x[e % 2 * 2 + 1], F16);
          if constexpr (PP == 2) pw[i][1][e] = rest16(x[e % 2 * 2], x[e % 2 * 2 + 1], pw[i][0][e]);
        }
      }
#pragma unroll
      for (int c = 0; c < L::C; ++c) {
        uint32_t vw[4][VD];        // pairs of tokens
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t* qd = vals.q[k / 2] + c * (VD / 2);
          const uint32_t sd = vals.s[c][k / 2];
          if constexpr (VD == 8) pair_tokens<FMT, VD>(qd[k % 2 * 2], qd[k % 2 * 2 + 1], sd, k % 2, vw[k]);
          else pair_tokens<FMT, VD>(qd[k % 2] & 0xFFFF, qd[k % 2] >> 16, sd, k % 2, vw[k]);
        }
#pragma unroll
        for (int j = 0; j < VD; ++j) {
          const u32x4 x = {vw[0][j], vw[1][j], vw[2][j], vw[3][j]};
#pragma unroll
          for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int y = 0; y < PP; ++y) o[i][c * VD + j] = product<F16>(x, pw[i][y], o[i][c * VD + j]);
        }
      }
      if (careful && (t + 1) * kStep > seen_by_all) {
        const uint8_t* at = head_at(page) + L::kSide;
        for (int j = t * kStep; j < min((t + 1) * kStep, len); ++j)
#pragma unroll
          for (int k = 0; k < 4 * L::C; ++k) {
            const int c = k / 4, e = k % 4, sg = c * (128 / L::G) + (4 * g + e) * VD / L::G;
            if (!nan_scale<FMT>(at[L::value_scale(j % kPage, sg)])) continue;
#pragma unroll
            for (int i = 0; i < NQ; ++i)
              if (j < seen_by_all + q[i].row) {
#pragma unroll
                for (int x = 0; x < VD; ++x) o[i][c * VD + x][e] = NAN;
              }
          }
      }
      page = next;
      load_values(vals, head_at(next) + L::kSide, tn & 1, lane);
    }
    // 0 times a value that a row does not see is NaN where that is not finite
    if (!careful && a.rows > 1 && t0 < t1 && t1 * kStep > seen_by_all) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) z = fmaf(0.0f, o[i][j][e], z);
      if (__any(z != z)) {
        careful = true;
        page = table.page(t0 >> 1);
        load_keys(keys, head_at(page), t0 & 1, lane);
        load_values(vals, head_at(page) + L::kSide, t0 & 1, lane);
        goto again;
      }
    }
    // what the next piece begins with is on its way while this one's sums are joined
    const bool whole = p1 - p0 == n;
    const int slot = 2 * blockIdx.x + (u != u0), b1 = b, head1 = head, chunk1 = chunk;
    u += a.direct ? 1 : p1 - p0;
    if (u < u1) begin(u);
    const float vscale = a.vs ? *a.vs : 1.0f;
    __syncthreads();           // the sums of the piece before have been read
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      l[i] = sum_over_g(l[i]);
      if (g == 0) red_ml[i][wave][lane] = f32x2{m[i], l[i]};
#pragma unroll
      for (int c = 0; c < L::C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < VD; j += 4)
            // row 4 g + e of the tiles (c, ..): the dimensions of lane 4 g + e
            *reinterpret_cast<f32x4*>(&red[i][wave][lane & 15][c * 128 + (4 * g + e) * VD + j]) =
                f32x4{o[i][c * VD + j][e], o[i][c * VD + j + 1][e], o[i][c * VD + j + 2][e], o[i][c * VD + j + 3][e]};
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      constexpr int N = D / 16;          // dimensions of a thread
      const int col = threadIdx.x >> 4, d = (threadIdx.x & 15) * N, at = (chunk1 * NQ + i) * 16 + col;
      if (at >= a.cols) continue;
      f32x2 ml[kWaves];
      float mt = -INFINITY, lt = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        ml[w] = red_ml[i][w][col];
        mt = fmaxf(mt, ml[w].x);
      }
      f32x4 v[N / 4] = {};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (ml[w].y == 0.0f) continue;
        const float f = __builtin_amdgcn_exp2f(ml[w].x - (mt == -INFINITY ? 0.0f : mt));
        lt += ml[w].y * f;
#pragma unroll
        for (int x = 0; x < N / 4; ++x) v[x] += *reinterpret_cast<const f32x4*>(&red[i][w][col][d + 4 * x]) * f;
      }
      if (whole) {
        const int row = at / a.group, hq = head1 * a.group + at % a.group;
        const float inv = lt == 0.0f ? 0.0f : vscale / lt;
        uint32_t y[N / 2];
#pragma unroll
        for (int x = 0; x < N / 2; ++x) y[x] = pack16(v[x / 2][x % 2 * 2] * inv, v[x / 2][x % 2 * 2 + 1] * inv, HALF);
        __builtin_memcpy(a.out + b1 * a.os[0] + row * a.os[1] + hq * a.os[2] + d, y, sizeof y);
        if (a.lse && d == 0) a.lse[((int64_t)b1 * a.pool.heads + head1) * a.cols + at] = lse2_of<FMT>(mt, lt);
      } else {
        const int64_t p = (int64_t)slot * (16 * NQ) + i * 16 + col;
#pragma unroll
        for (int x = 0; x < N / 4; ++x) *reinterpret_cast<f32x4*>(a.part + p * D + d + 4 * x) = v[x];
        if (d == 0) *reinterpret_cast<f32x2*>(a.part_ml + p * 2) = f32x2{mt, lt};
      }
    }
  }
}

// Joins the pieces of a head that several blocks worked on: one block per
// sequence, head and column; groups of D / 4 threads take pieces in turn.  Also the
// sequences without tokens (zeros), and those whose length cannot be (NaN).
template <int D, int FMT, bool HALF, int NQ>
__global__ __launch_bounds__(kThreads) void k_kv4_join(AttendArgs a) {
  constexpr int T = D / 4, N = kThreads / T;       // threads of a group, groups
  __shared__ float f_of[kMaxParts];
  __shared__ __align__(16) float red[N][D];
  __shared__ float red_m[kWaves], red_l[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int col = blockIdx.x % a.cols, head = blockIdx.x / a.cols % a.pool.heads, b = blockIdx.x / a.cols / a.pool.heads;
  const int n = pages_of(a.seqs, b);
  float lse = -INFINITY, inv = 0.0f;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n == 0) {
    if (length_of(a.seqs, b) < 0) v.x = lse = inv = NAN;
    if (tid < D) red[0][tid] = v.x;
  } else {
    const int per = a.pool.heads * a.chunks, chunk = col / (16 * NQ);
    const List list(a.seqs, lane);
    const int64_t units = list.total * per, start = list.before(b) * per + (int64_t)(head * a.chunks + chunk) * n;
    const Cuts cuts(units, a.nblocks);
    const int w0 = cuts.holds(start), w1 = cuts.holds(start + n - 1);
    if (w0 == w1) return;
    // the first part holds the piece that it ends with, the others those that they begin with
    const auto place = [&](int w) -> int64_t {
      return (int64_t)(2 * w + (w == w0 && cuts.start(w) < start)) * (16 * NQ) + col % (16 * NQ);
    };
    float m = -INFINITY, l = 0.0f;
    for (int w = w0 + tid; w <= w1; w += kThreads) {
      const bool any = cuts.start(w) < cuts.start(w + 1);     // parts may be empty
      const f32x2 ml = any ? *reinterpret_cast<const f32x2*>(a.part_ml + 2 * place(w)) : f32x2{-INFINITY, 0.0f};
      m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (lane == 0) red_m[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, red_m[w]);
    const float mu = m == -INFINITY ? 0.0f : m;
    for (int w = w0 + tid; w <= w1; w += kThreads) {
      const bool any = cuts.start(w) < cuts.start(w + 1);
      const f32x2 ml = any ? *reinterpret_cast<const f32x2*>(a.part_ml + 2 * place(w)) : f32x2{-INFINITY, 0.0f};
      const float f = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - mu);
      f_of[w - w0] = f;
      if (ml.y != 0.0f) l += ml.y * f;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o);
    if (lane == 0) red_l[wave] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) l += red_l[w];
    constexpr int kAhead = 4;            // pieces of a group whose loads are under way together
    const int first = w0 + tid / T;
    for (int w = first; w <= w1; w += kAhead * N) {
      f32x4 x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        x[i] = *reinterpret_cast<const f32x4*>(a.part + place(min(w + i * N, w1)) * D + tid % T * 4);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float f = w + i * N <= w1 ? f_of[w + i * N - w0] : 0.0f;
        if (f != 0.0f) v += x[i] * f;        // what an empty part has is not looked at
      }
    }
    *reinterpret_cast<f32x4*>(&red[tid / T][tid % T * 4]) = v;
    lse = lse2_of<FMT>(m, l);
    inv = l == 0.0f ? 0.0f : (a.vs ? *a.vs : 1.0f) / l;
    __syncthreads();
    if (tid < D) {
      float sum = 0.0f;
#pragma unroll
      for (int g = 0; g < N; ++g) sum += red[g][tid];
      red[0][tid] = l == 0.0f ? 0.0f : sum * inv;
    }
  }
  if (tid < D)
    a.out[b * a.os[0] + col / a.group * a.os[1] + (head * a.group + col % a.group) * a.os[2] + tid] = narrow<HALF>(red[0][tid]);
  if (a.lse && tid == 0) a.lse[((int64_t)b * a.pool.heads + head) * a.cols + col] = lse;
}

// Adds the attention weights of all rows and query heads to the tokens' sums, from
// the keys again and the sums of exponentials that are known now: reading 4-bit
// keys twice costs less than writing and reading the scores.  A step belongs to one
// wavefront, so the order of every sum is fixed.  97680 tokens, 4 key heads, 32 columns
// each, MXFP4: 17 us (2 TB/s; six steps per wavefront, whose start they do not hide).
// With more columns the queries of a chunk are widened again at every step: 8 key heads,
// 128 columns, NVFP4, 146 us.
template <int D, int FMT, bool HALF, int NQ>
__global__ __launch_bounds__(kThreads, 2) void k_kv4_weights(AttendArgs a) {
  typedef Layout<D, FMT> L;
  constexpr bool F16 = FMT == kNv;
  constexpr int W = Keys<D, FMT>::W, QP = Queries<D, FMT, HALF>::P;
  const int lane = threadIdx.x & 63, g = lane >> 4, part = blockIdx.x * kWaves + wave_index();
  const List list(a.seqs, lane);
  const int64_t units = list.total * a.pool.heads * 2;          // steps
  const Cuts cuts(units, gridDim.x * kWaves);
  const int64_t u0 = cuts.start(part), u1 = cuts.start(part + 1);
  for (int64_t u = u0; u < u1;) {
    int64_t before;
    int pages;
    const int b = list.at(u, a.pool.heads * 2, pages, before), n = 2 * pages, len = length_of(a.seqs, b);
    const int head = (int)quotient(u - before, n);
    const int t0 = (int)(u - before - (int64_t)head * n), t1 = (int)(u1 - u < n - t0 ? t0 + (u1 - u) : n);
    Table table(a.pool, a.seqs, lane);
    table.open(b, t0 >> 1);
    const float* lse = a.lse + ((int64_t)b * a.pool.heads + head) * a.cols;
    const int seen_by_all = len - a.rows + 1;
    Queries<D, FMT, HALF> q[NQ];
    float from[NQ];
    const auto columns = [&](int chunk) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int first = (chunk * NQ + i) * 16, col = first + (lane & 15);
        fetch_queries(q[i], a, b, head, first, lane);
        widen_queries(q[i], a, first, lane);
        const float ls = col < a.cols ? lse[col] : -INFINITY;
        if (ls == -INFINITY) q[i].row = -(1 << 30);       // no such column, or one that sees nothing
        from[i] = ls == -INFINITY ? 0.0f : ls;
      }
    };
    if (a.chunks == 1) columns(0);
    // the lane's place of a step
    const int at = (lane >> 2 & 1) * 16 + 4 * g + (lane & 3);
    const auto unit_of = [&](int t) { return (int64_t)max(table.page(t >> 1), 0) * a.pool.heads + head; };
    const int te = min(t1, (len + kStep - 1) / kStep);
    Keys<D, FMT> keys, ahead;
    float old = 0.0f, old_ahead;
    int64_t unit = 0;
    if (t0 < te) {
      unit = unit_of(t0);
      load_keys(keys, a.pool.pages + unit * L::kHead, t0 & 1, lane);
      old = a.pool.weights[unit * kPage + (t0 & 1) * kStep + at];
    }
    for (int t = t0; t < te; ++t) {
      const bool is = table.page(t >> 1) >= 0;
      float* w = a.pool.weights + unit * kPage + (t & 1) * kStep + at;
      // the next step's on their way
      const int tn = min(t + 1, te - 1);
      unit = unit_of(tn);
      load_keys(ahead, a.pool.pages + unit * L::kHead, tn & 1, lane);
      old_ahead = a.pool.weights[unit * kPage + (tn & 1) * kStep + at];
      float sum[2][4] = {};
      for (int chunk = 0; chunk < a.chunks; ++chunk) {
        if (a.chunks > 1) columns(chunk);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          u32x4 kw[W];
          widen_keys(keys, x, kw);
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < W; ++k)
#pragma unroll
              for (int y = 0; y < QP; ++y) s = product<F16>(kw[k], q[i].x[k][y], s);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = __builtin_amdgcn_exp2f(fmaf(s[e], q[i].factor, -from[i]));
              sum[x][e] += t * kStep + x * 16 + 4 * g + e < seen_by_all + q[i].row ? p : 0.0f;
            }
          }
        }
      }
      // over the sixteen columns, halving the eight values while there are pairs: lane n ends with value n % 8
      // (with lane n ^ 7, then n ^ 2, n ^ 1 and n ^ 8)
      const int n3 = lane & 7;
      float h4[4], h2[2], h1;
#pragma unroll
      for (int e = 0; e < 4; ++e) h4[e] = (n3 & 4 ? sum[1][e] : sum[0][e]) + dpp<0x141>(n3 & 4 ? sum[0][e] : sum[1][e]);
#pragma unroll
      for (int e = 0; e < 2; ++e) h2[e] = (n3 & 2 ? h4[2 + e] : h4[e]) + dpp<0x4E>(n3 & 2 ? h4[e] : h4[2 + e]);
      h1 = (n3 & 1 ? h2[1] : h2[0]) + dpp<0xB1>(n3 & 1 ? h2[0] : h2[1]);
      h1 += dpp<0x128>(h1);
      if (is && (lane & 8) == 0 && t * kStep + at < len) *w = old + h1;
      keys = ahead;
      old = old_ahead;
    }
    u += t1 - t0;
  }
}

// Tiles of 16 columns that a block works on at a time.
int tiles_of(int cols, int dim) {
  return cols <= 16 || dim == 256 ? 1 : 2;
}

template <int D, int FMT, bool HALF, int NQ>
hipError_t launch(AttendArgs a, hipStream_t st) {
  hipLaunchKernelGGL((k_kv4_attend<D, FMT, HALF, NQ>), dim3(a.nblocks), dim3(kThreads), 0, st, a);
  if (!a.direct) {
    const unsigned joins = (unsigned)a.seqs.n * a.pool.heads * a.cols;
    hipLaunchKernelGGL((k_kv4_join<D, FMT, HALF, NQ>), dim3(joins), dim3(kThreads), 0, st, a);
  }
  if (a.lse) hipLaunchKernelGGL((k_kv4_weights<D, FMT, HALF, NQ>), dim3(a.weight_blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

sc_status check_attention(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t rows, int32_t q_heads) {
  sc_status s = check_cache(cache);
  if (s == SC_OK) s = check_seqs(seqs);
  if (s != SC_OK) return s;
  if (rows < 1 || rows > SC_KV4_MAX_ROWS) return fail(SC_E_ARG, "rows must be in [1, %d]", SC_KV4_MAX_ROWS);
  if (q_heads < 1 || q_heads % cache->kv_heads || q_heads / cache->kv_heads > SC_KV4_MAX_GROUP)
    return fail(SC_E_ARG, "q_heads must be a multiple of kv_heads, up to %d times", SC_KV4_MAX_GROUP);
  if ((int64_t)seqs->n_seqs * rows * q_heads > (1 << 23)) return fail(SC_E_ARG, "too many query rows for one call");
  return SC_OK;
}

struct Work {
  int nq, chunks, blocks, weight_blocks;
  bool direct;
  size_t part, ml, lse, total;
};
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
Work work_of(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t rows, int32_t q_heads, bool weights) {
  Work w;
  const int cols = rows * (q_heads / cache->kv_heads);
  w.nq = tiles_of(cols, cache->head_dim);
  w.chunks = (cols + 16 * w.nq - 1) / (16 * w.nq);
  const int64_t heads = (int64_t)seqs->n_seqs * cache->kv_heads * w.chunks, pages = heads * seqs->width;
  const int most = w.nq == 1 && cache->head_dim <= 128 ? 768 : 512;        // blocks that run at a time
  w.direct = seqs->width <= kDirectPages;
  w.blocks = (int)(w.direct ? heads : pages < most ? pages : most);
  w.weight_blocks = (int)(pages < 512 ? pages : 512);
  const int slots = w.direct ? 0 : 2 * w.blocks;
  w.part = 0;
  w.ml = round256((size_t)slots * 16 * w.nq * cache->head_dim * 4);
  w.lse = w.ml + round256((size_t)slots * 16 * w.nq * 8);
  w.total = 256 + w.lse + (weights ? round256((size_t)seqs->n_seqs * cache->kv_heads * cols * 4) : 0);
  return w;
}

}  // namespace
}  // namespace kv4
}  // namespace sc

using namespace sc;
using namespace sc::kv4;

extern "C" {

sc_status kv4_attention_workspace_bytes(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t rows,
                                        int32_t q_heads, int32_t accumulate, size_t* bytes) {
  if (!bytes) return fail(SC_E_ARG, "bytes is NULL");
  const sc_status s = check_attention(cache, seqs, rows, q_heads);
  if (s != SC_OK) return s;
  *bytes = work_of(cache, seqs, rows, q_heads, accumulate != 0).total;
  return SC_OK;
}

sc_status kv4_attention(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_query* x, int32_t accumulate,
                        void* d_workspace, void* stream) {
  if (!x) return fail(SC_E_ARG, "query is NULL");
  const sc_status s = check_attention(cache, seqs, x->rows, x->q_heads);
  if (s != SC_OK) return s;
  if (x->type != SC_DTYPE_BF16 && x->type != SC_DTYPE_F16) return fail(SC_E_ARG, "type must be bf16 or fp16");
  if (!(x->scale > 0.0f) || x->scale > SC_ATTENTION_MAX_SCALE) return fail(SC_E_ARG, "scale must be positive and at most 2.3e38");
  if (accumulate && !cache->d_weights) return fail(SC_E_ARG, "the cache keeps no weights");
  if (seqs->n_seqs == 0) return SC_OK;
  if (!x->d_q || !x->d_out || (uintptr_t)x->d_q % 2 || (uintptr_t)x->d_out % 2)
    return fail(SC_E_ARG, "q or out is NULL or not aligned to its elements");
  for (int i = 0; i < 3; ++i)
    if (x->q_stride[i] < 0 || x->out_stride[i] < 0) return fail(SC_E_ARG, "strides must be >= 0");
  if (!d_workspace || (uintptr_t)d_workspace % 256) return fail(SC_E_ARG, "workspace is NULL or not 256-byte aligned");
  const Work w = work_of(cache, seqs, x->rows, x->q_heads, accumulate != 0);
  AttendArgs a{};
  a.pool = pool_of(cache);
  a.seqs = seqs_of(seqs);
  a.ks = cache->d_k_scale;
  a.vs = cache->d_v_scale;
  a.q = static_cast<const uint16_t*>(x->d_q);
  a.out = static_cast<uint16_t*>(x->d_out);
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = x->q_stride[i];
    a.os[i] = x->out_stride[i];
  }
  a.rows = x->rows;
  a.group = x->q_heads / cache->kv_heads;
  a.cols = a.rows * a.group;
  a.chunks = w.chunks;
  a.scale = x->scale;
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.part_ml = reinterpret_cast<float*>(ws + w.ml);
  a.lse = accumulate ? reinterpret_cast<float*>(ws + w.lse) : nullptr;
  a.nblocks = w.blocks;
  a.weight_blocks = w.weight_blocks;
  a.direct = w.direct;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool half = x->type == SC_DTYPE_F16;
  const hipError_t e = by_layout(cache->head_dim, cache->format, [&](auto d, auto f) {
    const auto tiles = [&](auto nq) {
      return half ? launch<d(), f(), true, nq()>(a, st) : launch<d(), f(), false, nq()>(a, st);
    };
    if constexpr (d() < 256) {
      if (w.nq == 2) return tiles(std::integral_constant<int, 2>{});
    }
    return tiles(std::integral_constant<int, 1>{});
  });
  if (e != hipSuccess) return hip_fail(e, "kv4_attention launch");
  return SC_OK;
}

}  // extern "C"
