// y = x W^T + bias for weights held in 4 bits.
#include "fp4_device.h"
#include "internal.h"

namespace sc {
namespace {

using namespace fp4;

struct LinearArgs {
  const uint8_t* codes;    // [N][K/2]
  const uint8_t* scales;   // [N][K/G]
  const float* gs;         // scale of the matrix (null: 1)
  const uint16_t* x;       // [M][K], row stride ldx
  void* y;                 // [M][N], row stride ldy
  const float* bias;       // [N] or null
  int64_t ldx, ldy;
  int N, K, M;
  int wk;                  // wavefronts of a block that share its rows along K (1, 2 or 4)
  int kc;                  // K-elements of the operand that LDS holds at a time
  int out;                 // sc_dtype of y
  int mblocks;             // tiles of rows (k_fp4_tiles)
};

template <typename T>
__device__ __forceinline__ uint16_t bits16(float v) {
  return __builtin_bit_cast(uint16_t, (T)v);
}
__device__ __forceinline__ void store_out(void* y, int64_t i, float v, int out) {
  if (out == SC_DTYPE_F32) static_cast<float*>(y)[i] = v;
  else if (out == SC_DTYPE_BF16) static_cast<uint16_t*>(y)[i] = bits16<__bf16>(v);
  else static_cast<uint16_t*>(y)[i] = bits16<_Float16>(v);
}

// Eight elements of an operand row, which need not be aligned to more than themselves.
__device__ __forceinline__ u32x4 load_x16(const uint16_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, sizeof v);
  return v;
}

constexpr int kRowPad = 16;   // bytes between operand rows in LDS: four rows' reads fall into different banks

// ---- up to four rows ---------------------------------------------------------------
//
// Every weight is used once, so this is a stream: a wavefront walks 512-element
// steps of eight weight rows with three steps of loads under way, and the operand
// rows lie in LDS.  Where the rows alone give too few wavefronts, up to four share
// a row's steps and add their sums in LDS, in wavefront order.  Bound by HBM, and
// in small matrices by the start and end of the launch: 1 x 6144 x 6144 8.4 us (2.5
// TB/s), 4 x 32768 x 4096 in MXFP4 17.7 us (4.1 TB/s).
template <int FMT, bool ODD, bool HALF, int ROWS, int Q, int D>
__global__ __launch_bounds__(256) void k_fp4_rows(LinearArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  constexpr int V = Q * ROWS;
  constexpr int G = FMT == kNv ? 16 : 32;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = a.wk, kw = wave & (wk - 1), rw = wave / wk;
  const int block_rows = 4 * Q * (4 / wk);
  const int row_base = blockIdx.x * block_rows;
  const int nrows = min(a.N - row_base, block_rows);
  const int row0 = rw * 4 * Q;                            // of the wavefront, within the block
  const int row_lds = a.kc * 2 + kRowPad;
  const Reader<FMT> rd = reader<FMT>(a.codes + (size_t)row_base * (a.K / 2), a.scales + (size_t)row_base * (a.K / G),
                                     (uint32_t)nrows, a.K);
  bool in[Q];
#pragma unroll
  for (int j = 0; j < Q; ++j) in[j] = row0 + 4 * j + (lane & 3) < nrows;

  float acc[Q][ROWS];
#pragma unroll
  for (int j = 0; j < Q; ++j)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[j][r] = 0.0f;

  const int r0 = lane & 3;
  const uint8_t* xs[(ROWS + 3) / 4];
#pragma unroll
  for (int s = 0; s < (ROWS + 3) / 4; ++s) xs[s] = lds + (4 * s + r0 < ROWS ? 4 * s + r0 : 0) * row_lds + rd.klane * 2;
  for (int kc = 0; kc < a.K; kc += a.kc) {
    const int kend = min(a.K, kc + a.kc);
    const int steps = (kend - kc + kStepK - 1) / kStepK;
    const int n = steps > kw ? (steps - kw + wk - 1) / wk : 0;
    Stage<FMT, ODD, Q> st[D];
    const int k0 = kc + kw * kStepK;
#pragma unroll
    for (int d = 0; d < D; ++d)
      load_stage<FMT, ODD, Q>(st[d], rd, row0, 4, k0 + d * wk * kStepK, kend, in);
    if (kc) __syncthreads();
    // the operand rows of this range, zero behind the last element
    const int per_row = steps * (kStepK / 8);
    for (int i = threadIdx.x; i < a.M * per_row; i += 256) {
      const int r = i / per_row, c = (i - r * per_row) * 8;
      u32x4 v = {0, 0, 0, 0};
      if (kc + c < kend) v = load_x16(a.x + (int64_t)r * a.ldx + kc + c);
      *reinterpret_cast<u32x4*>(lds + r * row_lds + c * 2) = v;
    }
    __syncthreads();
    for (int i = 0; i < n; i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i + d < n) {
          use_stage<FMT, ODD, Q, ROWS, HALF>(st[d], xs, ((i + d) * wk + kw) * kStepK * 2, acc);
          load_stage<FMT, ODD, Q>(st[d], rd, row0, 4, k0 + (i + d + D) * wk * kStepK, kend, in);
        }
      }
    }
  }

  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i / ROWS][i % ROWS];
  tile_sum<V>(v);
  // each wavefront's sums of its K share, then their total in wavefront order
  __syncthreads();
  float* red = reinterpret_cast<float*>(lds);
  if (tile_sum_owner<V>(lane)) {
    const int first = tile_sum_first<V>(lane);
#pragma unroll
    for (int i = 0; i < kTileOut<V>; ++i) red[(wave * V + first + i) * 4 + (lane & 3)] = v[i];
  }
  __syncthreads();
  const float gs = a.gs ? *a.gs : 1.0f;
  for (int i = threadIdx.x; i < block_rows * a.M; i += 256) {
    const int r = i / block_rows, n = i - r * block_rows;
    if (n >= nrows) continue;
    const int w = n / (4 * Q), q = (n / 4) % Q;
    float s = 0.0f;
    for (int k = 0; k < wk; ++k) s += red[((w * wk + k) * V + q * ROWS + r) * 4 + (n & 3)];
    s *= gs;
    if (a.bias) s += a.bias[row_base + n];
    store_out(a.y, (int64_t)r * a.ldy + row_base + n, s, a.out);
  }
}

template <int FMT, bool ODD, bool HALF, int ROWS>
hipError_t launch_rows(LinearArgs a, hipStream_t st) {
  constexpr int Q = 2, D = 3;
  const int steps = (a.K + kStepK - 1) / kStepK;
  const long tiles = ((long)a.N + 4 * Q - 1) / (4 * Q);
  a.wk = 1;
  while (a.wk < 4 && a.wk * 2 <= steps && tiles * a.wk < 4096) a.wk *= 2;
  const int cap = ROWS == 1 ? 16384 : ROWS == 2 ? 8192 : ROWS == 4 ? 6144 : 2048;
  a.kc = steps * kStepK < cap ? steps * kStepK : cap;
  const int block_rows = 4 * Q * (4 / a.wk);
  // rows behind the last are read by the lanes that stand for them, and not used
  size_t lds = (size_t)ROWS * (a.kc * 2 + kRowPad);
  const size_t red = 4 * 4 * sizeof(float) * (Q * ROWS);
  if (lds < red) lds = red;
  hipLaunchKernelGGL((k_fp4_rows<FMT, ODD, HALF, ROWS, Q, D>), dim3((unsigned)(((long)a.N + block_rows - 1) / block_rows)),
                     dim3(256), lds, st, a);
  return hipGetLastError();
}

template <int FMT, bool ODD, bool HALF>
hipError_t rows_by_count(const LinearArgs& a, hipStream_t st) {
  if (a.M == 1) return launch_rows<FMT, ODD, HALF, 1>(a, st);
  if (a.M == 2) return launch_rows<FMT, ODD, HALF, 2>(a, st);
  return launch_rows<FMT, ODD, HALF, 4>(a, st);
}

// ---- many rows -------------------------------------------------------------------
//
// Tiles of BM operand rows and WN NT 16 weight rows on the 16x16x32 matrix
// instruction.  A block has KS groups of WN wavefronts; a group takes every KS-th
// 128-element chunk of K, and the groups' sums are added at the end, in group
// order.  The wavefronts of a group share the operand's chunk through LDS and own
// different weight rows, so a weight is widened once per block.  What bounds it up
// to a few hundred rows is a wavefront's chain of chunks (load, wait, barrier,
// multiply: half a microsecond each), not its arithmetic: the KS groups shorten the
// chain and hide each other's waits (4096 x 12288, 16 rows, us: 47 with one group
// per block, 32 with four, 15.6 with eight on tiles a quarter as wide), while a
// second chunk under way in registers gained nothing.  From there on it is the
// widening, done once per block of rows.  A lane reads 16
// bytes of codes: 32 elements of row l % 16 at 32 (l / 16) of a 128-element chunk;
// the order of K within a chunk is free as long as the operand is read in the
// same order.  Widened weights carry their group scale, exactly: an E2M1 code
// times an E4M3 scale has 6 significant bits, times a power of two 2.
//   NVFP4, bf16: through fp32 products      (2 instructions per weight)
//   NVFP4, fp16: packed fp16 products       (1)
//   MXFP4: the scale goes into the conversion (1/2), always to bf16, whose
//   exponent holds every E8M0 scale; fp16 operands are split into two bf16
//   parts (11 = 8 + 3 significant bits), both multiplied.
constexpr int kChunk = 128;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 x, u32x4 w, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, w), c, 0, 0,
                                                   0);
}

// Two codes (byte B of d), times their scale s.
template <int FMT, bool F16, int B>
__device__ __forceinline__ uint32_t scaled2(uint32_t d, float s) {
  if constexpr (FMT == kMx) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, B));
  } else if constexpr (F16) {
    const _Float16 h = (_Float16)s;
    const f16x2 v = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, B));
    return __builtin_bit_cast(uint32_t, v * f16x2{h, h});
  } else {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, B);
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(v.x * s), (__bf16)(v.y * s)});
  }
}
template <int FMT, bool F16>
__device__ __forceinline__ u32x4 scaled8(uint32_t d, float s) {
  return u32x4{scaled2<FMT, F16, 0>(d, s), scaled2<FMT, F16, 1>(d, s), scaled2<FMT, F16, 2>(d, s),
               scaled2<FMT, F16, 3>(d, s)};
}

template <int FMT, bool ODD, bool HALF, int BM, int NT, int WN, int KS>
__global__ __launch_bounds__(64 * WN * KS) void k_fp4_tiles(LinearArgs a) {
  extern __shared__ __align__(16) uint8_t lds_all[];
  constexpr bool F16 = HALF && FMT == kNv;                 // type of the products
  constexpr int P = HALF && FMT == kMx ? 2 : 1;            // bf16 parts of the operand
  constexpr int MT = BM / 16, BN = WN * NT * 16, T = 64 * WN, G = FMT == kNv ? 16 : 32;
  constexpr int kRow = kChunk * 2 + 16, kPlane = BM * kRow;   // bytes; rows shifted by four banks each
  constexpr int XL = BM * kChunk / 8 / T;                // 16-byte pieces of the operand chunk per thread
  const int lane = threadIdx.x & 63, wave = wave_index() % WN, kg = wave_index() / WN, tid = threadIdx.x % T;
  uint8_t* lds = lds_all + kg * (2 * P * kPlane);
  // blocks that share weight rows follow each other on one XCD (they are dealt out to eight in turn)
  const int nb = gridDim.x / a.mblocks, id = blockIdx.x;
  const int per = (nb + 7) / 8, xcd = id % 8, slot = id / 8;
  int bn = xcd * per + slot / a.mblocks, bm = slot % a.mblocks;
  if (nb % 8) {
    bn = id / a.mblocks;
    bm = id % a.mblocks;
  }
  const int n0 = bn * BN + wave * NT * 16, m0 = bm * BM;
  const int rows = min(a.N - bn * BN, BN);
  const uint32_t cb = (uint32_t)a.K / 2, sb = (uint32_t)a.K / G;
  const Rsrc rc = make_rsrc(a.codes + (size_t)bn * BN * cb, (uint32_t)rows * cb);
  const Rsrc rs = make_rsrc(a.scales + (size_t)bn * BN * sb, (uint32_t)rows * sb);
  const int g = lane >> 4, r = lane & 15;

  u32x4 q[NT];
  uint32_t sc[NT];
  // cached loads: the blocks of other rows read the same weights (256 rows: 50 us, 54 past the cache)
  auto load_w = [&](int kc) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = wave * NT * 16 + t * 16 + r, k = kc + 32 * g;
      const bool in = row < rows && k < a.K;
      const uint32_t oc = (uint32_t)row * cb + k / 2, os = (uint32_t)row * sb + k / G;
      if constexpr (ODD) {
        const bool in2 = in && k + 16 < a.K;
        const u32x2 lo = load8<kReuse>(rc, in ? oc : kBeyond, 0), hi = load8<kReuse>(rc, in2 ? oc + 8 : kBeyond, 0);
        q[t] = u32x4{lo.x, lo.y, hi.x, hi.y};
        sc[t] = load1<kReuse>(rs, in ? os : kBeyond, 0) | load1<kReuse>(rs, in2 ? os + 1 : kBeyond, 0) << 8;
      } else {
        q[t] = load16<kReuse>(rc, in ? oc : kBeyond, 0);
        sc[t] = FMT == kMx ? load1<kReuse>(rs, in ? os : kBeyond, 0) : load2<kReuse>(rs, in ? os : kBeyond, 0);
      }
    }
  };
  u32x4 xr[XL];
  auto load_x = [&](int kc) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int e = tid + i * T, m = min(m0 + e / (kChunk / 8), a.M - 1), k = kc + e % (kChunk / 8) * 8;
      xr[i] = u32x4{0, 0, 0, 0};
      if (k < a.K) xr[i] = load_x16(a.x + (int64_t)m * a.ldx + k);
    }
  };
  auto put_x = [&](uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int e = tid + i * T;
      uint8_t* p = buf + e / (kChunk / 8) * kRow + e % (kChunk / 8) * 16;
      if constexpr (P == 1) {
        *reinterpret_cast<u32x4*>(p) = xr[i];
      } else {
        u32x4 hi, lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f16x2 v = __builtin_bit_cast(f16x2, (uint32_t)xr[i][j]);
          const bf16x2 h = {(__bf16)(float)v.x, (__bf16)(float)v.y};
          // what is not finite stands in the first part alone
          const float d0 = (float)v.x - (float)h.x, d1 = (float)v.y - (float)h.y;
          const bf16x2 l = {(__bf16)(d0 == d0 ? d0 : 0.0f), (__bf16)(d1 == d1 ? d1 : 0.0f)};
          hi[j] = __builtin_bit_cast(uint32_t, h);
          lo[j] = __builtin_bit_cast(uint32_t, l);
        }
        *reinterpret_cast<u32x4*>(p) = hi;
        *reinterpret_cast<u32x4*>(p + kPlane) = lo;
      }
    }
  };

  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // group kg takes every KS-th chunk; behind the last one it multiplies zeros
  load_x(kg * kChunk);
  load_w(kg * kChunk);
  put_x(lds);
  __syncthreads();
  int buf = 0;
  for (int kc = kg * kChunk; kc - kg * kChunk < a.K; kc += KS * kChunk) {
    u32x4 cq[NT];
    f32x2 cs[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      cq[t] = q[t];
      cs[t] = lane_scales<FMT>(sc[t]);
    }
    const bool more = kc - kg * kChunk + KS * kChunk < a.K;
    if (more) {
      load_x(kc + KS * kChunk);
      load_w(kc + KS * kChunk);
    }
    const uint8_t* xb = lds + buf * (P * kPlane) + r * kRow + g * 64;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) w[t] = scaled8<FMT, F16>(cq[t][j], j < 2 ? cs[t].x : cs[t].y);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(xb + p * kPlane + i * 16 * kRow + j * 16);
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[i][t] = mfma16<F16>(x, w[t], acc[i][t]);
        }
    }
    if (more) put_x(lds + (buf ^ 1) * (P * kPlane));
    __syncthreads();
    buf ^= 1;
  }
  if constexpr (KS > 1) {
    // the groups' sums in group order; the loop's last barrier has freed the chunks
    static_assert((KS - 1) * MT * NT * 16 * T <= KS * 2 * P * kPlane, "the sums fit where the chunks were");
    f32x4* part = reinterpret_cast<f32x4*>(lds_all);
    if (kg) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[(((kg - 1) * MT + i) * NT + t) * T + tid] = acc[i][t];
    }
    __syncthreads();
    if (kg) return;
#pragma unroll
    for (int o = 0; o < KS - 1; ++o)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[i][t] += part[((o * MT + i) * NT + t) * T + tid];
  }
  const float gs = a.gs ? *a.gs : 1.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + t * 16 + r;
    if (n >= a.N) continue;
    const float b = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = m0 + i * 16 + g * 4 + e;
        if (m < a.M) store_out(a.y, (int64_t)m * a.ldy + n, acc[i][t][e] * gs + b, a.out);
      }
  }
}

template <int FMT, bool ODD, bool HALF, int BM, int NT, int WN, int KS>
hipError_t launch_tiles(LinearArgs a, hipStream_t st) {
  constexpr int P = HALF && FMT == kMx ? 2 : 1;
  a.mblocks = (int)(((int64_t)a.M + BM - 1) / BM);
  const long blocks = (long)a.mblocks * (((long)a.N + 16 * NT * WN - 1) / (16 * NT * WN));
  hipLaunchKernelGGL((k_fp4_tiles<FMT, ODD, HALF, BM, NT, WN, KS>), dim3((unsigned)blocks), dim3(64 * WN * KS),
                     KS * 2 * P * BM * (kChunk * 2 + 16), st, a);
  return hipGetLastError();
}

// Up to four rows fill the 4x4x4 instruction, more would waste the 16x16 one less:
// 4096 x 4096, 4 rows 7.1 us against 7.3 with 16x16 tiles, 5 rows 8.4 against 7.3.
//
// From there on: the smallest tiles that give each of the 256 compute units at most one block: a
// compute unit's time is that of its blocks' longest chain of chunks, which more
// units and more shares of K shorten, while larger tiles read and widen less.
// Measured, us, bf16 NVFP4 4096 x 4096 (16x16 / 16x32 / 32x32 / 32x64 / 64x64 /
// 64x128): 16 rows 7.5 / 9.2 / 10.5 / 14.5 / - / -, 64 rows 15 / 13.7 / 11.3 /
// 15.0 / 20 / 31, 256 rows - / - / - / 23.8 / 20.8 / 31, 1024 rows - / - / - / 92 /
// 62 / 54.  Two blocks of 64x64 share a unit.  Tiles of 128x192, which widen least,
// pay from two blocks per unit on (6144 x 6144, 1024 rows: 256 blocks, 114 against
// 107 with 64x128; 2048 rows: 163 against 218).  The sweep was made for this format
// and type only; the others take the same sizes.  6144 x 6144 with 16 / 64 / 256 /
// 1024 / 2048 rows, caches cold: NVFP4 bf16 16.4 / 29.3 / 54.8 / 119 / 174, NVFP4
// fp16 16.2 / 29.3 / 55.5 / 118 / 168, MXFP4 bf16 16.0 / 28.5 / 54.8 / 116 / 156, MXFP4
// fp16, with twice the products, 18.0 / 33.3 / 117 / 229 / 398.
template <int FMT, bool ODD, bool HALF>
hipError_t by_count(const LinearArgs& a, hipStream_t st) {
  constexpr bool kTwo = HALF && FMT == kMx;        // operand in two parts: twice the LDS
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (a.M <= 4) return rows_by_count<FMT, ODD, HALF>(a, st);
  if (tiles(16, 16) <= 256) return launch_tiles<FMT, ODD, HALF, 16, 1, 1, 8>(a, st);
  if (a.M <= 16 || tiles(16, 32) <= 256) return launch_tiles<FMT, ODD, HALF, 16, 1, 2, 8>(a, st);
  if (tiles(32, 32) <= 256) return launch_tiles<FMT, ODD, HALF, 32, 1, 2, kTwo ? 4 : 8>(a, st);
  if (a.M <= 32 || tiles(32, 64) <= 256) return launch_tiles<FMT, ODD, HALF, 32, 1, 4, 4>(a, st);
  if (tiles(64, 64) <= 512) return launch_tiles<FMT, ODD, HALF, 64, 1, 4, 2>(a, st);
  if constexpr (!kTwo)
    if (tiles(128, 192) >= 512) return launch_tiles<FMT, ODD, HALF, 128, 3, 4, 1>(a, st);
  return launch_tiles<FMT, ODD, HALF, 64, 2, 4, 1>(a, st);
}

template <bool HALF>
hipError_t by_format(const LinearArgs& a, int fmt, hipStream_t st) {
  if (fmt == SC_FP4_MX) return by_count<kMx, false, HALF>(a, st);
  if (a.K / 16 % 2) return by_count<kNv, true, HALF>(a, st);
  return by_count<kNv, false, HALF>(a, st);
}

// A launch has less than 2^32 threads, and runs only part of a larger grid without an error.  Up to 32
// rows take 32 threads per weight row at most, more of them 256 per 64 x 128 outputs (tiles with more
// threads per output are taken for up to 512 blocks only); indexes of rows stay below 2^31 with a tile to spare.
hipError_t in_pieces(const LinearArgs& all, bool half, int fmt, hipStream_t st) {
  constexpr int kMostN = 1 << 25;
  const int N0 = all.N < kMostN ? all.N : kMostN;
  const int64_t most_m = 64 * ((((int64_t)1 << 24) - 1) / (((int64_t)N0 + 127) / 128));
  const int row_codes = all.K / 2, row_scales = all.K / (fmt == SC_FP4_NV ? 16 : 32), size = all.out == SC_DTYPE_F32 ? 4 : 2;
  for (int64_t n = 0; n < all.N; n += kMostN)
    for (int64_t m = 0; m < all.M; m += most_m) {
      LinearArgs a = all;
      a.N = (int)(all.N - n < kMostN ? all.N - n : kMostN);
      a.M = (int)(all.M - m < most_m ? all.M - m : most_m);
      a.codes += n * row_codes;
      a.scales += n * row_scales;
      if (a.bias) a.bias += n;
      a.x += m * a.ldx;
      a.y = static_cast<uint8_t*>(a.y) + (m * a.ldy + n) * size;
      const hipError_t e = half ? by_format<true>(a, fmt, st) : by_format<false>(a, fmt, st);
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace
}  // namespace sc

using namespace sc;

extern "C" sc_status fp4_linear(const sc_fp4_matrix* w, const void* d_x, int32_t x_type, int64_t ldx, int32_t M,
                                const float* d_bias, void* d_y, int32_t y_type, int64_t ldy, void* stream) {
  sc_status s = check_fp4_matrix(w);
  if (s != SC_OK) return s;
  if (x_type != SC_DTYPE_BF16 && x_type != SC_DTYPE_F16) return fail(SC_E_ARG, "x_type must be bf16 or fp16");
  if (y_type != SC_DTYPE_BF16 && y_type != SC_DTYPE_F16 && y_type != SC_DTYPE_F32)
    return fail(SC_E_ARG, "unknown y_type %d", y_type);
  if (M < 0) return fail(SC_E_ARG, "M must be >= 0");
  if (M == 0 || w->rows == 0) return SC_OK;
  if (!d_x || !d_y) return fail(SC_E_ARG, "x or y is NULL");
  if (ldx < w->cols || ldy < w->rows) return fail(SC_E_ARG, "row strides must cover the rows");
  if ((uintptr_t)d_x % 2 || (uintptr_t)d_y % (y_type == SC_DTYPE_F32 ? 4 : 2) || (uintptr_t)d_bias % 4)
    return fail(SC_E_ARG, "x, y or bias is not aligned to its elements");
  LinearArgs a{};
  a.codes = static_cast<const uint8_t*>(w->d_codes);
  a.scales = static_cast<const uint8_t*>(w->d_scales);
  a.gs = w->d_global_scale;
  a.bias = d_bias;
  a.ldx = ldx;
  a.ldy = ldy;
  a.N = w->rows;
  a.K = w->cols;
  a.out = y_type;
  a.M = M;
  a.x = static_cast<const uint16_t*>(d_x);
  a.y = d_y;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = in_pieces(a, x_type == SC_DTYPE_F16, w->format, st);
  if (e != hipSuccess) return hip_fail(e, "fp4_linear launch");
  return SC_OK;
}
