// Attention over whole prompts: packed sequences of different lengths, causal,
// query heads in groups that share a key head.
//
//   s_j = scale q . k_j,   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
// over the keys j that a row sees: all up to its own, with rows at the end of
// the keys when there are fewer rows than keys.  One pass over the keys keeps
// the running maximum, the sum and o in fp32.
//
// Scores are formed transposed (keys times queries, 32x32x16 products): a lane
// has one query's scores of the keys that it has to supply to the second product,
// V^T times P^T, so P goes from the first product to the second in its registers.
// V^T comes from the rows of V by LDS loads that transpose.  P is rounded to the
// type of v for that product, as its other operand is.
//
// A block has 128 rows, 32 per wavefront, and two blocks share a compute unit, so
// that one wavefront of a SIMD can be in its softmax while the other multiplies.
// What bounds it: not settled.  16384 rows of 32 heads of 128, fp16: 2.13 to 2.23
// ms, 0.99 to 1.03 PFLOP/s (an 8192^3 bf16 library product on the same card reaches
// 1.22); matrix units busy in 52% of the cycles, no LDS conflicts, at a mean clock of
// 1.85 GHz, which speaks for power but does not prove it.  9708 packed rows of 8 sequences, 48 heads:
// 263 to 276 us, 0.79 to 0.83 PFLOP/s; the rest is starting 3840 blocks and tiles on the diagonal.
// The first kernel here (one buffer through registers, no late maxima, masks
// everywhere) took 7.03 ms and 783 us.
#include "fp4_device.h"
#include "internal.h"

#include <atomic>
#include <type_traits>

namespace sc {
namespace prompt {
namespace {

using namespace fp4;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;       // query rows of a block
// Keys of a tile.  With heads of 256 the sums alone take 128 registers.
template <int D>
constexpr int kKeysOf = D == 256 ? 32 : 64;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  float* lse;               // [rows][heads] or null
  const int32_t* starts;    // [n + 1] rows
  const int32_t* key_starts;
  int64_t qs[2], ks[2], vs[2], os[2];     // strides: row, head
  int32_t n, rows, keys, heads, group;
  float scale;
  int32_t parts;            // that the keys of a block's rows are cut into
  float* part;              // [blocks][parts][wavefronts][32 D] sums of the parts, with parts > 1
  float* part_ml;           // [blocks][parts][wavefronts][32][2]
};

// The operands live until the result is there, so that it takes no register of theirs.
template <bool HALF>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
  f32x16 d;
  if constexpr (HALF)
    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  asm("" : "+v"(d) : "v"(a), "v"(b));
  return d;
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (HALF) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
__device__ __forceinline__ u32x4 load_row(const uint16_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
template <bool HALF>
__device__ __forceinline__ float widen(uint32_t v) {
  if constexpr (HALF) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
  else return __uint_as_float(v << 16);
}
// Eight elements, zeros for those that are not finite.
template <bool HALF>
__device__ __forceinline__ u32x4 finite8(u32x4 v) {
  constexpr uint32_t kInf = HALF ? 0x7C00u : 0x7F80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & kInf) == kInf) v[i] &= 0xFFFF0000u;
    if ((v[i] >> 16 & kInf) == kInf) v[i] &= 0xFFFFu;
  }
  return v;
}
// LDS by its offsets: the products' operands are at a few lane offsets plus constants.
template <typename T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *(const __attribute__((address_space(3))) T*)at;
}
// Four rows of 16 columns, 8 bytes of a row per lane: a lane gets its column.
__device__ __forceinline__ u32x2 load_transposed(uint32_t at) {
  typedef __attribute__((address_space(3))) s16x4 Lds;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)at));
}

// A wavefront's 32 rows of sums, times the lane's inv, to rows of out: lanes exchange
// pieces in LDS so that a store covers whole rows (9708 packed rows of 48 heads of 128,
// 3840 blocks: 263 us; with 8 bytes per lane straight from the registers 281).
template <int NI, bool HALF>
__device__ __forceinline__ void write_rows(uint32_t lds, const f32x16 (&o)[NI], float inv, int lane, int rows, uint16_t* out,
                                           int64_t stride) {
  constexpr int CH = NI * 4, RI = 64 / CH;          // 16-byte pieces of a row, rows of a store
  const int hi = lane >> 5, qc = lane & 31;
  const auto piece = [](int row, int c) { return c ^ (CH >= 16 ? row & 15 : row >> 1 & 7); };
  typedef __attribute__((address_space(3))) u32x2 Lds;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      // dimensions 32 i + 8 e + 4 hi ..
      *(Lds*)(lds + qc * (CH * 16) + piece(qc, i * 4 + e) * 16 + hi * 8) =
          u32x2{pack<HALF>(o[i][e * 4] * inv, o[i][e * 4 + 1] * inv), pack<HALF>(o[i][e * 4 + 2] * inv, o[i][e * 4 + 3] * inv)};
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int it = 0; it < 32 / RI; ++it) {
    const int row = it * RI + lane / CH, c = lane % CH;
    const u32x4 v = lds_at<u32x4>(lds + row * (CH * 16) + piece(row, c) * 16);
    if (row < rows) __builtin_memcpy(out + row * stride + c * 8, &v, 16);
  }
}

// A sequence's rows and keys; none where the starts make no sense.
struct Sequence {
  int row0, rows, key0, keys;
};
__device__ __forceinline__ Sequence sequence(const PromptArgs& a, int b) {
  Sequence s = {0, 0, 0, 0};
  if (b < a.n) {
    s.row0 = a.starts[b];
    s.rows = a.starts[b + 1];
    s.key0 = a.key_starts[b];
    s.keys = a.key_starts[b + 1];
    s.rows = s.row0 >= 0 && s.rows >= s.row0 && s.rows <= a.rows ? s.rows - s.row0 : 0;
    s.keys = s.key0 >= 0 && s.keys >= s.key0 && s.keys <= a.keys ? s.keys - s.key0 : 0;
  }
  return s;
}
// The sequence of tile t of all, and t within it; false behind the last.  The lanes
// hold 64 sequences at a time, so the one that is found needs no further load.
__device__ __forceinline__ bool sequence_at(const PromptArgs& a, int& t, int lane, Sequence& s) {
  int sum = 0;
  for (int i = 0; i < a.n; i += 64) {
    const Sequence x = sequence(a, i + lane);
    const int n = (x.rows + kRows - 1) / kRows, upto = sum + wave_scan(n);
    const uint64_t beyond = __ballot(upto > t);
    if (beyond) {
      const int l = __builtin_ctzll(beyond);
      t -= __builtin_amdgcn_readlane(upto - n, l);
      s = {__builtin_amdgcn_readlane(x.row0, l), __builtin_amdgcn_readlane(x.rows, l),
           __builtin_amdgcn_readlane(x.key0, l), __builtin_amdgcn_readlane(x.keys, l)};
      return true;
    }
    sum = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// The tile and head of a block.  Blocks are dealt out to eight XCDs in turn: heads
// next to each other, which share keys, go to one of them.
__device__ __forceinline__ void block_of(const PromptArgs& a, int& head, int& tile) {
  head = blockIdx.x % a.heads;
  tile = blockIdx.x / a.heads;
  if (a.heads % 8 == 0) {
    const int per = a.heads / 8, xcd = blockIdx.x % 8, slot = blockIdx.x / 8;
    head = xcd * per + slot % per;
    tile = slot / per;
  }
}

// Tiles of keys and values lie in two LDS buffers; the next tile is fetched straight
// into LDS during the products of this one.  Rows follow each other without padding,
// as such loads need it; the 16-byte pieces of a row are exchanged so that lanes that
// are served together meet in no bank.  Loads of 16 bytes are served to sixteen lanes
// at a time (0-3, 12-15, 20-27 of each half, then the rest) from 256 bytes of banks:
// their rows have sixteen places for a piece, two rows' worth with heads of 64.  The
// transposing loads take two pieces of four rows for sixteen lanes, and the two
// pieces after them for the next sixteen.  (With places that repeated after eight and
// four rows a quarter of the kernel's time were conflicts.)
//
// m is the maximum that P counts from; it follows a row's scores only once they
// exceed it by kSlack, so o is seldom multiplied again.
template <int PR>
__device__ __forceinline__ int key_piece(int row, int c) { return c ^ (PR == 8 ? row >> 1 & 7 : row & 15); }
template <int PR>
__device__ __forceinline__ int value_piece(int row, int c) { return c ^ (PR == 8 ? row >> 1 & 1 : row & 3) * 4; }

// 16 bytes per lane from memory to LDS, one after the other from `to` on; waited for
// by vmcnt.  (The builtin makes the compiler wait before every later LDS read.)
__device__ __forceinline__ void load_to_lds(Rsrc from, uint32_t lane, uint32_t at, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to), "v"(lane), "s"(from), "s"(at)
               : "memory", "m0");
}

template <int D, bool HALF, bool DIRECT, bool PARTS>
__global__ __launch_bounds__(kThreads, 2) void k_prompt(PromptArgs a) {
  constexpr int kKeys = kKeysOf<D>, kRow = D * 2, kSide = kKeys * kRow;                // bytes in LDS
  constexpr int NO = D / 32, NK = D / 16, PR = D / 8, NL = kKeys * PR / kThreads;   // pieces of a row, of a thread
  constexpr int RL = kThreads / PR;                                // rows that the block loads at a time
  // fp16 P counts from 2^14, so that what its range cuts off is below 2^-38 of the largest
  constexpr float kShift = HALF ? 14.0f : 0.0f, kSlack = HALF ? 1.875f : 8.0f;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index(), hi = lane >> 5, qc = lane & 31;
  const int part = PARTS ? blockIdx.y : 0;
  int head, tile;
  block_of(a, head, tile);
  Sequence seq;
  if (!sequence_at(a, tile, lane, seq)) return;
  const int row0 = seq.row0, rows = seq.rows, key0 = seq.key0, keys = seq.keys;
  tile = (rows + kRows - 1) / kRows - 1 - tile;      // those with the most keys first
  const int r0 = tile * kRows + wave * 32, row = r0 + qc;
  const int ahead = keys - rows + 1;                 // keys that row 0 sees
  const int mine = min(keys, ahead + min(row, rows - 1));
  int end = min(keys, ahead + min(tile * kRows + kRows, rows) - 1), begin = 0;       // of the block
  if constexpr (PARTS) {
    const int nt = max(0, (end + kKeys - 1) / kKeys);
    begin = (int)((int64_t)nt * part / a.parts) * kKeys;
    end = min(end, (int)((int64_t)nt * (part + 1) / a.parts) * kKeys);
  }
  const int wave_end = r0 < rows ? min(end, ahead + min(r0 + 32, rows) - 1) : 0, wave_all = ahead + r0;
  u32x4 q[NK];
  const uint16_t* qp = a.q + (int64_t)(row0 + min(row, rows - 1)) * a.qs[0] + head * a.qs[1] + hi * 8;
#pragma unroll
  for (int i = 0; i < NK; ++i) q[i] = load_row(qp + 16 * i);
  const uint16_t* kp = a.k + (int64_t)key0 * a.ks[0] + head / a.group * a.ks[1];
  const uint16_t* vp = a.v + (int64_t)key0 * a.vs[0] + head / a.group * a.vs[1];
  const float factor = a.scale * kLog2e;
  const int seen_by_all = ahead + tile * kRows;      // keys that every row of the block sees
  float m, l;
  f32x16 o[NO];
  bool careful = false;      // values that only some rows see are not finite: in a second pass

  const int lr = tid / PR, lc = tid % PR;            // the thread's row and piece
  const uint32_t k_lane = (uint32_t)(lr * a.ks[0] * 2 + key_piece<PR>(lr, lc) * 16);
  const uint32_t k_odd = (uint32_t)(lr * a.ks[0] * 2 + key_piece<PR>(lr + RL, lc) * 16);      // of rows RL later
  const uint32_t v_lane = (uint32_t)(lr * a.vs[0] * 2 + value_piece<PR>(lr, lc) * 16);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  // The lane's key row; its piece of product i differs from that of product 0 in bits 5 to 7 (heads of 64: 5 and 6).
  constexpr int KX = D == 64 ? 4 : 8, VX = D == 64 ? 2 : 4;
  const uint32_t k_at = lds0 + qc * kRow + key_piece<PR>(qc, hi) * 16;
  // Rows 4 hi .. + 3 of the values, 16 dimensions of lane / 16 % 2; output tiles differ in bits 6 and 7 (6).
  const int vr = hi * 4 + (lane & 15) / 4;
  const uint32_t v_at = lds0 + kSide + vr * kRow + value_piece<PR>(vr, (lane >> 4 & 1) * 2 + (lane >> 1 & 1)) * 16 + lane % 2 * 8;
  auto fetch = [&](int j0, int buf) {
    uint8_t* to = lds + buf * 2 * kSide;
    if (DIRECT && j0 + kKeys <= end && !careful) {
      const Rsrc rk = make_rsrc(kp + (int64_t)j0 * a.ks[0], 0x7FFFFFFF), rv = make_rsrc(vp + (int64_t)j0 * a.vs[0], 0x7FFFFFFF);
      const uint32_t at = lds0 + buf * 2 * kSide + wave * 1024;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        load_to_lds(rk, i % 2 ? k_odd : k_lane, (uint32_t)(i * RL * a.ks[0] * 2), at + i * kThreads * 16);
        load_to_lds(rv, v_lane, (uint32_t)(i * RL * a.vs[0] * 2), at + kSide + i * kThreads * 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int r = lr + i * RL, j = j0 + r;
        u32x4 kr = {0, 0, 0, 0}, vr = {0, 0, 0, 0};      // nothing of other sequences
        if (j < end) {
          kr = load_row(kp + (int64_t)j * a.ks[0] + lc * 8);
          vr = load_row(vp + (int64_t)j * a.vs[0] + lc * 8);
        }
        if (careful && j0 + kKeys > seen_by_all) vr = finite8<HALF>(vr);
        *reinterpret_cast<u32x4*>(to + r * kRow + key_piece<PR>(r, lc) * 16) = kr;
        *reinterpret_cast<u32x4*>(to + kSide + r * kRow + value_piece<PR>(r, lc) * 16) = vr;
      }
    }
  };

again:
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < NO; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
  int buf = 0;
  if (begin < end) fetch(begin, 0);
  __builtin_amdgcn_s_waitcnt(0x0F70);        // vmcnt(0): this wavefront's part of the tile is there
  __syncthreads();
  for (int j0 = begin; j0 < end; j0 += kKeys) {
    if (j0 + kKeys < end) fetch(j0 + kKeys, buf ^ 1);
    const uint32_t bk = k_at + buf * 2 * kSide, bv = v_at + buf * 2 * kSide;
    if (j0 < wave_end) {
      f32x16 s[kKeys / 32];
#pragma unroll
      for (int t = 0; t < kKeys / 32; ++t) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
          const u32x4 kw = lds_at<u32x4>((bk ^ i % KX * 32) + i / KX * 256 + t * 32 * kRow);
          s[t] = product<HALF>(kw, q[i], s[t]);
        }
      }
      if (j0 + kKeys > wave_all) {
#pragma unroll
        for (int t = 0; t < kKeys / 32; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (j0 + t * 32 + e / 4 * 8 + hi * 4 + e % 4 >= mine) s[t][e] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int e = 1; e < kKeys / 2; ++e) top = fmaxf(top, s[e / 16][e % 16]);
      top = fmaxf(top, __shfl_xor(top, 32)) * factor;
      if (__any(top > m + kSlack)) {
        const float mn = top > m + kSlack ? top : m;       // of this row, whatever the others do
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        l *= f;
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i] *= f;
        m = mn;
      }
      const float mu = (m == -INFINITY ? 0.0f : m) - kShift;
#pragma unroll
      for (int t = 0; t < kKeys / 32; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          s[t][e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], factor, -mu));
          l += s[t][e];
        }
#pragma unroll
      for (int t = 0; t < kKeys / 16; ++t) {
        const f32x16& x = s[t / 2];
        const int f = t % 2 * 8;
        const u32x4 pw = {pack<HALF>(x[f], x[f + 1]), pack<HALF>(x[f + 2], x[f + 3]), pack<HALF>(x[f + 4], x[f + 5]),
                          pack<HALF>(x[f + 6], x[f + 7])};
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          // of rows 16 t + 4 hi .. + 3, and of those eight later
          const uint32_t p = (bv ^ i % VX * 64) + i / VX * 256 + t * 16 * kRow;
          const u32x2 lo = load_transposed(p), hw = load_transposed(p + 8 * kRow);
          o[i] = product<HALF>(u32x4{lo.x, lo.y, hw.x, hw.y}, pw, o[i]);
        }
      }
      if (careful && j0 + kKeys > seen_by_all) {
        for (int j = j0; j < min(j0 + kKeys, mine); ++j)
#pragma unroll
          for (int i = 0; i < NO; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float x = widen<HALF>(vp[(int64_t)j * a.vs[0] + i * 32 + e / 4 * 8 + hi * 4 + e % 4]);
              if (!(fabsf(x) < INFINITY)) o[i][e] += x;
            }
      }
    }
    buf ^= 1;
    __builtin_amdgcn_s_waitcnt(0x0F70);      // vmcnt(0): this wavefront's part of the next tile is there
    __syncthreads();
  }
  // 0 times a value that a row does not see is NaN where that is not finite
  if (!careful) {
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) z = fmaf(0.0f, o[i][e], z);
    // one of the wavefronts', over LDS that the tiles have left (nothing else is in LDS, so that loads to it
    // stay below 64 KB)
    typedef __attribute__((address_space(3))) uint32_t Lds;
    const bool bad = __any(z != z);
    if (lane == 0) *(Lds*)(lds0 + wave * 4) = bad;
    __syncthreads();
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) any |= lds_at<uint32_t>(lds0 + w * 4);
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(any)) {
      careful = true;
      goto again;
    }
  }
  l += __shfl_xor(l, 32);
  if (r0 >= rows) return;
  if constexpr (PARTS) {
    // as the lanes hold them: whole kilobytes a store, and the join's lanes read the same
    const int64_t at = ((int64_t)blockIdx.x * a.parts + part) * kWaves + wave;
    float* to = a.part + at * (32 * D) + lane * 4;
#pragma unroll
    for (int i = 0; i < NO; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4*>(to + (i * 4 + e) * 256) = f32x4{o[i][e * 4], o[i][e * 4 + 1], o[i][e * 4 + 2], o[i][e * 4 + 3]};
    if (hi == 0) *reinterpret_cast<f32x2*>(a.part_ml + (at * 32 + qc) * 2) = f32x2{m - kShift, l};
    return;
  }
  write_rows<NO, HALF>(lds0 + wave * (32 * kRow), o, l == 0.0f ? 0.0f : 1.0f / l, lane, rows - r0,
                       a.out + (int64_t)(row0 + r0) * a.os[0] + head * a.os[1], a.os[0]);
  if (a.lse && hi == 0 && row < rows)
    a.lse[(int64_t)(row0 + row) * a.heads + head] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l) - kShift) * kLn2;
}

// Joins the parts of a wavefront's 32 rows, two tiles of 32 dimensions at a time.
template <int D, bool HALF>
__global__ __launch_bounds__(kThreads) void k_prompt_join(PromptArgs a) {
  __shared__ __align__(1024) uint8_t lds[kWaves * 32 * 128];
  const int lane = threadIdx.x & 63, wave = wave_index(), qc = lane & 31;
  int head, tile;
  block_of(a, head, tile);
  Sequence seq;
  if (!sequence_at(a, tile, lane, seq)) return;
  tile = (seq.rows + kRows - 1) / kRows - 1 - tile;      // as the blocks have them
  const int r0 = tile * kRows + wave * 32;
  if (r0 >= seq.rows) return;
  float m = -INFINITY, l = 0.0f;
  f32x16 o[2] = {};
  for (int p = 0; p < a.parts; ++p) {
    const int64_t at = ((int64_t)blockIdx.x * a.parts + p) * kWaves + wave;
    const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + (at * 32 + qc) * 2);
    const float* from = a.part + at * (32 * D) + blockIdx.y * (8 * 256) + lane * 4;
    f32x4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const f32x4*>(from + i * 256);
    // a part that the row sees nothing of has sums of 0
    const float mn = ml.y == 0.0f ? m : fmaxf(m, ml.x), mu = mn == -INFINITY ? 0.0f : mn;
    const float f = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - mu), fp = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - mu);
    l = l * f + ml.y * fp;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i / 16][i % 16] = o[i / 16][i % 16] * f + x[i / 4][i % 4] * fp;
    m = mn;
  }
  const int dim = blockIdx.y * 64;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  write_rows<2, HALF>(lds0 + wave * (32 * 128), o, l == 0.0f ? 0.0f : 1.0f / l, lane, seq.rows - r0,
                      a.out + (int64_t)(seq.row0 + r0) * a.os[0] + head * a.os[1] + dim, a.os[0]);
  if (a.lse && dim == 0 && lane < 32 && r0 + qc < seq.rows)
    a.lse[(int64_t)(seq.row0 + r0 + qc) * a.heads + head] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <int D, bool HALF, bool DIRECT, bool PARTS>
hipError_t launch(const PromptArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)((a.rows / kRows + a.n) * a.heads);
  constexpr int kLds = 4 * kKeysOf<D> * D * 2;
  // once per device: more LDS than a block has by default
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_prompt<D, HALF, DIRECT, PARTS>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    if (dev < 64) allowed.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  hipLaunchKernelGGL((k_prompt<D, HALF, DIRECT, PARTS>), dim3(grid, a.parts), dim3(kThreads), kLds, st, a);
  e = hipGetLastError();
  if (!PARTS || e != hipSuccess) return e;
  hipLaunchKernelGGL((k_prompt_join<D, HALF>), dim3(grid, D / 64), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}
// Loads to LDS take 16 aligned bytes; other keys and values go through registers.
template <int D, bool HALF>
hipError_t by_alignment(const PromptArgs& a, hipStream_t st) {
  const bool direct = ((uintptr_t)a.k | (uintptr_t)a.v) % 16 == 0 && (a.ks[0] | a.ks[1] | a.vs[0] | a.vs[1]) % 8 == 0;
  if (a.parts > 1) return direct ? launch<D, HALF, true, true>(a, st) : launch<D, HALF, false, true>(a, st);
  return direct ? launch<D, HALF, true, false>(a, st) : launch<D, HALF, false, false>(a, st);
}

sc_status check(const sc_prompt* p) {
  if (!p) return fail(SC_E_ARG, "the description is NULL");
  if (p->type != SC_DTYPE_BF16 && p->type != SC_DTYPE_F16) return fail(SC_E_ARG, "type must be bf16 or fp16");
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
    return fail(SC_E_ARG, "head_dim must be 64, 128 or 256");
  if (p->kv_heads < 1 || p->q_heads < 1 || p->q_heads > SC_PROMPT_MAX_HEADS || p->q_heads % p->kv_heads)
    return fail(SC_E_ARG, "q_heads must be a multiple of kv_heads and at most %d", SC_PROMPT_MAX_HEADS);
  if (p->n_seqs < 0 || p->n_seqs > SC_PROMPT_MAX_SEQS || p->rows < 0 || p->rows > SC_PROMPT_MAX_ROWS || p->keys < 0)
    return fail(SC_E_ARG, "n_seqs, rows or keys are out of range");
  // a launch of 2^32 threads or more would run only in part
  if (((int64_t)p->rows / kRows + p->n_seqs) * p->q_heads >= (1 << 24)) return fail(SC_E_ARG, "too many rows for one call");
  return SC_OK;
}

// The keys are cut into parts where blocks of whole rows would leave compute units
// idle (two blocks fit on each of 256), at once or because the rows with the most
// keys take longer than an even share, and every part still has two thousand keys:
// the parts' sums are written and read again.  1107 rows of 16 heads of 256 over
// 13527 keys: 144 blocks 339 us, in 3 parts 155.  Longest block of 2.0 even shares: 4
// heads of 128, 16384 rows, 347 us, in 2 parts 311; 8 heads of 256, 8192 rows, 402 and
// 303.  Of 1.6: 16 heads of 128, 5000 rows, 126 us and 157.
//
// Rows that see no key are no work: rows beyond the keys do not count in the shares.
// Shares are of rows, so sequences of a few rows look uneven however many they are: 16
// rows of 64 sequences over 2500 to 30000 keys, 32 heads, 2304 blocks, take 1347 us, in 2
// parts 1221 (all over 6000 keys: 535 and 585); 8056 blocks 6538 and 6596.  kMostBlocks
// ends that, and the sums' memory with it: 2 kMostBlocks blocks have at most 676 MB.
constexpr int64_t kMostBlocks = 5 * 512;
int parts_of(const sc_prompt* p) {
  const int64_t blocks = ((int64_t)p->rows / kRows + p->n_seqs) * p->q_heads, by_keys = p->keys / p->n_seqs / SC_PROMPT_PART_KEYS;
  // a block's keys on average, and of the last rows
  const int seeing = p->rows < p->keys ? p->rows : p->keys;
  const double most = (double)p->keys / p->n_seqs, mean = most - 0.5 * seeing / p->n_seqs;
  const bool uneven = blocks <= kMostBlocks && 512.0 * kRows * most > 1.8 * p->q_heads * seeing * mean;
  const int64_t by_units = 512 / blocks > 1 ? 512 / blocks : uneven ? 2 : 1, n = by_units < by_keys ? by_units : by_keys;
  return n < 2 ? 1 : n < 8 ? (int)n : 8;
}
size_t part_rows(const sc_prompt* p, int parts) {
  return ((size_t)p->rows / kRows + p->n_seqs) * p->q_heads * parts * kRows;
}
size_t part_bytes(const sc_prompt* p, int parts) { return part_rows(p, parts) * p->head_dim * 4; }

}  // namespace
}  // namespace prompt
}  // namespace sc

using namespace sc;

extern "C" {

sc_status prompt_attention_workspace_bytes(const sc_prompt* p, size_t* bytes) {
  if (!bytes) return fail(SC_E_ARG, "bytes is NULL");
  const sc_status s = prompt::check(p);
  if (s != SC_OK) return s;
  *bytes = 0;
  if (p->n_seqs == 0 || p->rows == 0) return SC_OK;
  const int parts = prompt::parts_of(p);
  if (parts > 1) *bytes = prompt::part_bytes(p, parts) + prompt::part_rows(p, parts) * 8;
  return SC_OK;
}

sc_status prompt_attention(const sc_prompt* p, void* d_workspace, void* stream) {
  const sc_status s = prompt::check(p);
  if (s != SC_OK) return s;
  if (!(p->scale > 0.0f) || p->scale > SC_ATTENTION_MAX_SCALE) return fail(SC_E_ARG, "scale must be positive and at most 2.3e38");
  if (p->n_seqs == 0 || p->rows == 0) return SC_OK;
  if (!p->d_q || !p->d_out || (p->keys > 0 && (!p->d_k || !p->d_v))) return fail(SC_E_ARG, "q, k, v or out is NULL");
  if ((uintptr_t)p->d_q % 2 || (uintptr_t)p->d_k % 2 || (uintptr_t)p->d_v % 2 || (uintptr_t)p->d_out % 2 ||
      (uintptr_t)p->d_lse % 4)
    return fail(SC_E_ARG, "q, k, v, out or lse is not aligned to its elements");
  if (!p->d_starts || !p->d_key_starts || (uintptr_t)p->d_starts % 4 || (uintptr_t)p->d_key_starts % 4)
    return fail(SC_E_ARG, "starts are NULL or not 4-byte aligned");
  prompt::PromptArgs a{};
  a.q = static_cast<const uint16_t*>(p->d_q);
  a.k = static_cast<const uint16_t*>(p->d_k);
  a.v = static_cast<const uint16_t*>(p->d_v);
  a.out = static_cast<uint16_t*>(p->d_out);
  a.lse = p->d_lse;
  a.starts = p->d_starts;
  a.key_starts = p->d_key_starts;
  for (int i = 0; i < 2; ++i) {
    if (p->q_stride[i] < 0 || p->k_stride[i] < 0 || p->v_stride[i] < 0 || p->out_stride[i] < 0)
      return fail(SC_E_ARG, "strides must be >= 0");
    if (p->k_stride[0] > SC_PROMPT_MAX_STRIDE || p->v_stride[0] > SC_PROMPT_MAX_STRIDE)
      return fail(SC_E_ARG, "keys and values must be at most %d elements apart", SC_PROMPT_MAX_STRIDE);
    a.qs[i] = p->q_stride[i];
    a.ks[i] = p->k_stride[i];
    a.vs[i] = p->v_stride[i];
    a.os[i] = p->out_stride[i];
  }
  a.n = p->n_seqs;
  a.rows = p->rows;
  a.keys = p->keys;
  a.heads = p->q_heads;
  a.group = p->q_heads / p->kv_heads;
  a.scale = p->scale;
  a.parts = prompt::parts_of(p);
  if (a.parts > 1) {
    if (!d_workspace || (uintptr_t)d_workspace % 16) return fail(SC_E_ARG, "workspace is NULL or not 16-byte aligned");
    a.part = static_cast<float*>(d_workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(d_workspace) + prompt::part_bytes(p, a.parts));
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const auto run = [&](auto half) {
    return p->head_dim == 64    ? prompt::by_alignment<64, half()>(a, st)
           : p->head_dim == 128 ? prompt::by_alignment<128, half()>(a, st)
                                : prompt::by_alignment<256, half()>(a, st);
  };
  const hipError_t e = p->type == SC_DTYPE_F16 ? run(std::true_type{}) : run(std::false_type{});
  if (e != hipSuccess) return hip_fail(e, "prompt_attention launch");
  return SC_OK;
}

}  // extern "C"
