// Attention of a few new tokens over the 4-bit key/value cache.
//
// For each row q of a sequence and query head, over the places j that the row sees:
//   s_j = scale q . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
// One pass over the pages keeps the running maximum m, the sum and o (fp32).
//
// A head's rows, all query heads that share it times all new tokens, are the
// columns of the 16x16x32 matrix products, so the cache is read and widened once
// for all of them:  S^T = K Q^T,  O^T = V^T P^T.  The tokens of S^T that a lane
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
#include "kv4_device.h"

namespace sc {
namespace kv4 {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kBlocks = 512;             // parts of the list: two per compute unit
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
  int32_t nblocks;
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
      const float s = e8m0((p.s[at / 4] >> (at % 4 * 8)) & 0xFF);
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
    const float sa = e8m0(sab >> (16 * half) & 0xFF), sb = e8m0(sab >> (16 * half + 8) & 0xFF);
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
// What bf16 leaves of two numbers; nothing of one that is not finite.
__device__ __forceinline__ uint32_t rest16(float a, float b, uint32_t hi) {
  const bf16x2 h = __builtin_bit_cast(bf16x2, hi);
  const float x = a - (float)h.x, y = b - (float)h.y;
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(x == x ? x : 0.0f), (__bf16)(y == y ? y : 0.0f)});
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
template <int D, int FMT, bool HALF>
__device__ __forceinline__ void load_queries(Queries<D, FMT, HALF>& q, const AttendArgs& a, int b, int head, int first,
                                             int lane) {
  typedef Layout<D, FMT> L;
  typedef Queries<D, FMT, HALF> Q;
  const int col = first + (lane & 15), g = lane >> 4;
  const bool in = col < a.cols;
  const int c1 = in ? col : a.cols - 1;
  q.row = c1 / a.group;
  const uint16_t* p = a.q + b * a.qs[0] + q.row * a.qs[1] + ((int64_t)head * a.group + c1 % a.group) * a.qs[2];
  constexpr int WC = L::LaneDims / 8;
  float v[Q::W][8];
  float top = 0.0f;
#pragma unroll
  for (int w = 0; w < Q::W; ++w) {
    uint16_t raw[8];
    __builtin_memcpy(raw, p + w / WC * 128 + g * L::LaneDims + w % WC * 8, 16);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[w][e] = HALF ? (float)__builtin_bit_cast(_Float16, raw[e]) : __uint_as_float((uint32_t)raw[e] << 16);
      if (!in) v[w][e] = 0.0f;
      top = fmaxf(top, fabsf(v[w][e]));
    }
  }
  float up = 1.0f;
  q.factor = a.scale * kLog2e * (a.ks ? *a.ks : 1.0f);
  if constexpr (FMT == kNv) {
    top = max_over_g(top);
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = top > 0.0f && e < 128 ? max(e, -100) : 13;
    up = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
    q.factor *= __uint_as_float((uint32_t)(127 + e - 13) << 23);
  }
  q.factor = fmaxf(q.factor, 1e-37f);       // masked scores are -inf times this
#pragma unroll
  for (int w = 0; w < Q::W; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[w][2 * e] * up, y = v[w][2 * e + 1] * up;
      q.x[w][0][e] = pack16(x, y, FMT == kNv);
      if constexpr (Q::P == 2) q.x[w][1][e] = rest16(x, y, q.x[w][0][e]);
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
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ __forceinline__ int64_t of_lane(int64_t v, int l) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
// Pages of the sequences before b, and of all.
__device__ __forceinline__ int64_t pages_before(const Seqs& s, int b, int64_t& total, int lane) {
  int64_t before = 0, sum = 0;
  for (int i = 0; i < s.n; i += 64) {
    const int64_t upto = wave_scan(pages_of(s, i + lane), lane);
    if (b >= i && b < i + 64) before = sum + (b > i ? of_lane(upto, b - i - 1) : 0);
    sum += of_lane(upto, 63);
  }
  total = sum;
  return before;
}
// The sequence that unit u of the list lies in, and the units before it; `per`
// units of the list per page of a sequence.
__device__ __forceinline__ int sequence_at(const Seqs& s, int64_t u, int per, int64_t& before, int lane) {
  int64_t sum = 0;
  for (int i = 0; i < s.n; i += 64) {
    const int64_t n = (int64_t)pages_of(s, i + lane) * per;
    const int64_t upto = sum + wave_scan(n, lane);
    const uint64_t beyond = __ballot(upto > u);
    if (beyond) {
      const int l = __builtin_ctzll(beyond);
      before = of_lane(upto - n, l);
      return i + l;
    }
    sum = of_lane(upto, 63);
  }
  before = sum;
  return s.n;
}
__device__ __forceinline__ int64_t cut(int64_t units, int part, int parts) { return units * part / parts; }
// The part that holds unit u.
__device__ __forceinline__ int part_of(int64_t units, int64_t u, int parts) { return (int)(((u + 1) * parts - 1) / units); }

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
__global__ __launch_bounds__(kThreads, 2) void k_kv4_attend(AttendArgs a) {
  typedef Layout<D, FMT> L;
  constexpr bool F16 = FMT == kNv;
  constexpr int W = Keys<D, FMT>::W, VD = L::VDims, NO = L::C * VD;     // output tiles
  constexpr int QP = Queries<D, FMT, HALF>::P, PP = FMT == kMx ? 2 : 1;
  // m is the maximum that P counts from; it follows the scores once they exceed it by kSlack
  constexpr float kShift = F16 ? 14.0f : 0.0f, kSlack = F16 ? 1.875f : 8.0f;
  constexpr int kRow = D + 4;
  __shared__ __align__(16) float red[kWaves][16][kRow];
  __shared__ float red_m[kWaves][16], red_l[kWaves][16];
  const int lane = threadIdx.x & 63, wave = wave_index(), g = lane >> 4;
  const int per = a.pool.heads * a.chunks;
  int64_t pages;
  pages_before(a.seqs, 0, pages, lane);
  const int64_t units = pages * per;
  const int64_t u0 = cut(units, blockIdx.x, a.nblocks), u1 = cut(units, blockIdx.x + 1, a.nblocks);
  for (int64_t u = u0; u < u1;) {
    int64_t before;
    const int b = sequence_at(a.seqs, u, per, before, lane);
    const int n = pages_of(a.seqs, b), len = length_of(a.seqs, b);
    const int hc = (int)((u - before) / n), head = hc / a.chunks, chunk = hc % a.chunks;
    const int p0 = (int)((u - before) % n), p1 = (int)(u1 - u < n - p0 ? p0 + (u1 - u) : n);
    const int t0 = 2 * p0 + wave, t1 = min(2 * p1, (len + kStep - 1) / kStep);        // steps
    Queries<D, FMT, HALF> q[NQ];
    float m[NQ], l[NQ];
    f32x4 o[NQ][NO];
    Keys<D, FMT> keys;
    Values<D, FMT> vals;
    const int seen_by_all = len - a.rows + 1;      // places that every row sees
    const auto head_at = [&](int page) { return a.pool.pages + ((int64_t)max(page, 0) * a.pool.heads + head) * L::kHead; };
    int page = t0 < t1 ? page_at(a.pool, a.seqs, b, t0 >> 1) : 0;
    if (t0 < t1) {
      load_keys(keys, head_at(page), t0 & 1, lane);
      load_values(vals, head_at(page) + L::kSide, t0 & 1, lane);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) load_queries(q[i], a, b, head, (chunk * NQ + i) * 16, lane);
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
      const int next = page_at(a.pool, a.seqs, b, tn >> 1);
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
        page = page_at(a.pool, a.seqs, b, t0 >> 1);
        load_keys(keys, head_at(page), t0 & 1, lane);
        load_values(vals, head_at(page) + L::kSide, t0 & 1, lane);
        goto again;
      }
    }
    // the wavefronts' sums, tile by tile
    const bool whole = p1 - p0 == n;
    const int slot = 2 * blockIdx.x + (u != u0);
    const float vscale = a.vs ? *a.vs : 1.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      l[i] = sum_over_g(l[i]);
      __syncthreads();
      if (g == 0) {
        red_m[wave][lane] = m[i];
        red_l[wave][lane] = l[i];
      }
      __syncthreads();
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, red_m[w][lane & 15]);
      const float f = m[i] == -INFINITY && l[i] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[i] - (mx == -INFINITY ? 0.0f : mx));
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          // row 4 g + e of output tile (c, j): dimension VD of that lane
          red[wave][lane & 15][j / VD * 128 + (4 * g + e) * VD + j % VD] = o[i][j][e] * f;
      __syncthreads();
      const int col = threadIdx.x >> 4, k = threadIdx.x & 15;
      float mt = -INFINITY, lt = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, red_m[w][col]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        if (red_l[w][col] != 0.0f)
          lt += red_l[w][col] * __builtin_amdgcn_exp2f(red_m[w][col] - (mt == -INFINITY ? 0.0f : mt));
      const int at = (chunk * NQ + i) * 16 + col;
      if (at < a.cols) {
        const int row = at / a.group, hq = head * a.group + at % a.group;
        const float inv = lt == 0.0f ? 0.0f : vscale / lt;
#pragma unroll
        for (int d = k; d < D; d += 16) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) v += red[w][col][d];
          if (whole)
            a.out[b * a.os[0] + row * a.os[1] + hq * a.os[2] + d] = narrow<HALF>(lt == 0.0f ? 0.0f : v * inv);
          else
            a.part[((int64_t)slot * (16 * NQ) + i * 16 + col) * D + d] = v;
        }
        if (k == 0) {
          if (!whole) {
            a.part_ml[((int64_t)slot * (16 * NQ) + i * 16 + col) * 2] = mt;
            a.part_ml[((int64_t)slot * (16 * NQ) + i * 16 + col) * 2 + 1] = lt;
          } else if (a.lse) {
            a.lse[((int64_t)b * a.pool.heads + head) * a.cols + at] = lse2_of<FMT>(mt, lt);
          }
        }
      }
    }
    u += p1 - p0;
  }
}

// Joins the pieces of a head that several blocks worked on: one block per
// sequence, head and column; groups of D / 4 threads take pieces in turn.  Also the
// sequences without tokens (zeros), and those whose length cannot be (NaN).
template <int D, int FMT, bool HALF, int NQ>
__global__ __launch_bounds__(kThreads) void k_kv4_join(AttendArgs a) {
  constexpr int T = D / 4, N = kThreads / T;       // threads of a group, groups
  __shared__ float f_of[kBlocks];
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
    int64_t pages;
    const int64_t before = pages_before(a.seqs, b, pages, lane) * per, units = pages * per;
    const int64_t start = before + (int64_t)(head * a.chunks + chunk) * n;
    const int w0 = part_of(units, start, a.nblocks), w1 = part_of(units, start + n - 1, a.nblocks);
    if (w0 == w1) return;
    // the first part holds the piece that it ends with, the others those that they begin with
    const auto place = [&](int w) -> int64_t {
      return (int64_t)(2 * w + (w == w0 && cut(units, w, a.nblocks) < start)) * (16 * NQ) + col % (16 * NQ);
    };
    float m = -INFINITY, l = 0.0f;
    for (int w = w0 + tid; w <= w1; w += kThreads) {
      const bool any = cut(units, w, a.nblocks) < cut(units, w + 1, a.nblocks);     // parts may be empty
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
      const bool any = cut(units, w, a.nblocks) < cut(units, w + 1, a.nblocks);
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
// wavefront, so the order of every sum is fixed.
template <int D, int FMT, bool HALF, int NQ>
__global__ __launch_bounds__(kThreads, 2) void k_kv4_weights(AttendArgs a) {
  typedef Layout<D, FMT> L;
  constexpr bool F16 = FMT == kNv;
  constexpr int W = Keys<D, FMT>::W, QP = Queries<D, FMT, HALF>::P;
  const int lane = threadIdx.x & 63, g = lane >> 4, part = blockIdx.x * kWaves + wave_index();
  int64_t pages;
  pages_before(a.seqs, 0, pages, lane);
  const int64_t units = pages * a.pool.heads * 2;          // steps
  const int64_t u0 = cut(units, part, a.nblocks * kWaves), u1 = cut(units, part + 1, a.nblocks * kWaves);
  for (int64_t u = u0; u < u1;) {
    int64_t before;
    const int b = sequence_at(a.seqs, u, a.pool.heads * 2, before, lane);
    const int n = 2 * pages_of(a.seqs, b), len = length_of(a.seqs, b), head = (int)((u - before) / n);
    const int t0 = (int)((u - before) % n), t1 = (int)(u1 - u < n - t0 ? t0 + (u1 - u) : n);
    const float* lse = a.lse + ((int64_t)b * a.pool.heads + head) * a.cols;
    const int seen_by_all = len - a.rows + 1;
    Queries<D, FMT, HALF> q[NQ];
    float from[NQ];
    const auto columns = [&](int chunk) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int first = (chunk * NQ + i) * 16, col = first + (lane & 15);
        load_queries(q[i], a, b, head, first, lane);
        const float ls = col < a.cols ? lse[col] : -INFINITY;
        if (ls == -INFINITY) q[i].row = -(1 << 30);       // no such column, or one that sees nothing
        from[i] = ls == -INFINITY ? 0.0f : ls;
      }
    };
    if (a.chunks == 1) columns(0);
    for (int t = t0; t < t1; ++t) {
      const int page = page_at(a.pool, a.seqs, b, t >> 1);
      if (page < 0 || t * kStep >= len) continue;
      const int64_t unit = (int64_t)page * a.pool.heads + head;
      Keys<D, FMT> keys;
      load_keys(keys, a.pool.pages + unit * L::kHead, t & 1, lane);
      // the lane's place of the step, and what it has so far
      const int at = (lane >> 2 & 1) * 16 + 4 * g + (lane & 3);
      float* w = a.pool.weights + unit * kPage + (t & 1) * kStep + at;
      const float old = *w;
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
      const int n3 = lane & 7;
      float h4[4], h2[2], h1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float keep = n3 & 4 ? sum[1][e] : sum[0][e], give = n3 & 4 ? sum[0][e] : sum[1][e];
        h4[e] = keep + __shfl_xor(give, 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float keep = n3 & 2 ? h4[2 + e] : h4[e], give = n3 & 2 ? h4[e] : h4[2 + e];
        h2[e] = keep + __shfl_xor(give, 2);
      }
      h1 = (n3 & 1 ? h2[1] : h2[0]) + __shfl_xor(n3 & 1 ? h2[0] : h2[1], 1);
      h1 += __shfl_xor(h1, 8);
      if ((lane & 8) == 0 && t * kStep + at < len) *w = old + h1;
    }
    u += t1 - t0;
  }
}

// Tiles of 16 columns that a block works on at a time.
int tiles_of(int cols, int dim) {
  return cols <= 16 || dim == 256 ? 1 : 2;
}

int blocks_for(int64_t most_units) { return (int)(most_units < kBlocks ? most_units : kBlocks); }

template <int D, int FMT, bool HALF, int NQ>
hipError_t launch(AttendArgs a, hipStream_t st) {
  hipLaunchKernelGGL((k_kv4_attend<D, FMT, HALF, NQ>), dim3(a.nblocks), dim3(kThreads), 0, st, a);
  const unsigned joins = (unsigned)a.seqs.n * a.pool.heads * a.cols;
  hipLaunchKernelGGL((k_kv4_join<D, FMT, HALF, NQ>), dim3(joins), dim3(kThreads), 0, st, a);
  if (a.lse) hipLaunchKernelGGL((k_kv4_weights<D, FMT, HALF, NQ>), dim3(a.nblocks), dim3(kThreads), 0, st, a);
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
  int nq, chunks, blocks;
  size_t part, ml, lse, total;
};
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
Work work_of(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t rows, int32_t q_heads, bool weights) {
  Work w;
  const int cols = rows * (q_heads / cache->kv_heads);
  w.nq = tiles_of(cols, cache->head_dim);
  w.chunks = (cols + 16 * w.nq - 1) / (16 * w.nq);
  w.blocks = blocks_for((int64_t)seqs->n_seqs * cache->kv_heads * w.chunks * seqs->width);
  w.part = 0;
  w.ml = round256((size_t)2 * w.blocks * 16 * w.nq * cache->head_dim * 4);
  w.lse = w.ml + round256((size_t)2 * w.blocks * 16 * w.nq * 8);
  w.total = w.lse + (weights ? round256((size_t)seqs->n_seqs * cache->kv_heads * cols * 4) : 0);
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
  if (!(x->scale > 0.0f) || x->scale > 3e38f) return fail(SC_E_ARG, "scale must be positive and finite");
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
