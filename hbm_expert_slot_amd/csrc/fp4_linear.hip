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
  int vec;                 // x rows can be read 16 bytes at a time
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

constexpr int kRowPad = 16;   // bytes between operand rows in LDS: four rows' reads fall into different banks

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
      if (kc + c < kend) {
        const uint16_t* p = a.x + (int64_t)r * a.ldx + kc + c;
        if (a.vec) {
          v = *reinterpret_cast<const u32x4*>(p);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = p[2 * e] | (uint32_t)p[2 * e + 1] << 16;
        }
      }
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
  hipLaunchKernelGGL((k_fp4_rows<FMT, ODD, HALF, ROWS, Q, D>), dim3((unsigned)((a.N + block_rows - 1) / block_rows)),
                     dim3(256), lds, st, a);
  return hipGetLastError();
}

template <int FMT, bool ODD, bool HALF>
hipError_t rows_by_count(const LinearArgs& a, hipStream_t st) {
  if (a.M == 1) return launch_rows<FMT, ODD, HALF, 1>(a, st);
  if (a.M == 2) return launch_rows<FMT, ODD, HALF, 2>(a, st);
  if (a.M <= 4) return launch_rows<FMT, ODD, HALF, 4>(a, st);
  if (a.M <= 8) return launch_rows<FMT, ODD, HALF, 8>(a, st);
  return launch_rows<FMT, ODD, HALF, 16>(a, st);
}

template <bool HALF>
hipError_t rows_by_format(const LinearArgs& a, int fmt, hipStream_t st) {
  if (fmt == SC_FP4_MX) return rows_by_count<kMx, false, HALF>(a, st);
  if (a.K / 16 % 2) return rows_by_count<kNv, true, HALF>(a, st);
  return rows_by_count<kNv, false, HALF>(a, st);
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
  a.vec = (uintptr_t)d_x % 16 == 0 && ldx % 8 == 0;
  const size_t ysize = y_type == SC_DTYPE_F32 ? 4 : 2;
  for (int64_t m = 0; m < M; m += 16) {
    a.M = (int)(M - m < 16 ? M - m : 16);
    a.x = static_cast<const uint16_t*>(d_x) + m * ldx;
    a.y = static_cast<uint8_t*>(d_y) + (size_t)(m * ldy) * ysize;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const hipError_t e = x_type == SC_DTYPE_F16 ? rows_by_format<true>(a, w->format, st)
                                                : rows_by_format<false>(a, w->format, st);
    if (e != hipSuccess) return hip_fail(e, "fp4_linear launch");
  }
  return SC_OK;
}
