// Quantising a weight matrix to 4 bits, and reading it back.
//
// NVFP4: the matrix scale g = max|w| / 2688 (so that the largest group scale is
// 448 and the largest code 6), a group's scale s = E4M3(max of the group / (6 g)),
// an element's code = E2M1(w / (s g)).  MXFP4: s = 2^(floor(log2 max) - 2).
// Every rounding is to nearest, ties to even, of the exact quotient: codes are
// whole numbers and a neighbour would be off by half of its value, so a
// quotient of rounded numbers next to a border is settled in fp64.
//
// The max and the codes need one pass each; the second finds a matrix of up to
// 256 MB in the memory-side cache.  4096 x 6144 bf16: max 10.6 us (4.7 TB/s; 19 us
// after 1 GiB of stores, which that cache then still has to write back), codes 24
// us (vector instructions: 32 products and 16 conversions per 16 elements; with every
// group scale's quotient in fp64 25 us), reading back to fp32 17.7 us (6.5 TB/s, into that cache).
#include "fp4_device.h"
#include "fp4_round.h"
#include "internal.h"

#include <type_traits>

namespace sc {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr unsigned kGrid = 1280; // blocks of k_fp4_codes at most: what the card holds at a time (one group per thread: 32 us)
constexpr unsigned kMaxBlocks = 512;
static_assert(kMaxBlocks * 4 <= SC_FP4_QUANT_WORKSPACE_BYTES, "one maximum per block");
constexpr int kMaxThreads = 512, kAhead = 4;   // k_fp4_max; pieces of a thread whose loads are under way together

struct QuantArgs {
  const void* w;
  int64_t ldw;
  uint8_t* codes;
  uint8_t* scales;
  float* gs;             // NVFP4: read when given, else written
  uint32_t* partial;     // per-block maxima (bits of |w|), null when the scale is given
  int nparts;
  uint32_t n16;          // groups of 16 elements in the matrix
  uint32_t per_row;      // groups of 16 per row
  int K;
};

// Sixteen elements of one row as they are in memory, which need not be aligned to
// more than themselves, and as fp32.
template <typename T>
struct Raw16 {
  u32x4 q[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load16_of(const QuantArgs& a, uint32_t i) {
  int64_t off = (int64_t)i * 16;
  if (a.ldw != a.K) {
    const uint32_t row = i / a.per_row;
    off = (int64_t)row * a.ldw + (i - row * a.per_row) * 16;
  }
  Raw16<T> r;
  __builtin_memcpy(&r, static_cast<const T*>(a.w) + off, sizeof r);
  return r;
}
template <typename T>
__device__ __forceinline__ void to_f32(const Raw16<T>& r, float (&v)[16]) {
  typedef __attribute__((ext_vector_type(16 / sizeof(T)))) T TV;
  constexpr int W = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = (float)__builtin_bit_cast(TV, r.q[i / W])[i % W];
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
  for (int o = 32; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  return m;
}

// Max of the magnitudes of 16 bytes as they order in memory's type, infinities and NaN too.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(u32x4 q) {
  if constexpr (sizeof(T) == 4) {
    return max(max(q.x & 0x7FFFFFFFu, q.y & 0x7FFFFFFFu), max(q.z & 0x7FFFFFFFu, q.w & 0x7FFFFFFFu));
  } else {
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, q[i] & 0x7FFF7FFFu));
    return max(m.x, m.y);
  }
}

// Every wavefront reads 1 KB pieces, kAhead of them under way at a time.
template <typename T>
__global__ __launch_bounds__(kMaxThreads) void k_fp4_max(QuantArgs a) {
  constexpr uint32_t kInf = sizeof(T) == 4 ? 0x7F800000u : std::is_same_v<T, __bf16> ? 0x7F80u : 0x7C00u;
  constexpr int W = 16 / sizeof(T);          // elements of a piece
  const uint64_t n = (uint64_t)a.n16 * sizeof(T), stride = (uint64_t)gridDim.x * kMaxThreads;
  uint32_t m = 0;
  for (uint64_t i = (uint64_t)blockIdx.x * kMaxThreads + threadIdx.x; i < n; i += kAhead * stride) {
    u32x4 q[kAhead];          // behind the last piece: that one again
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint64_t j = min(i + u * stride, n - 1);
      int64_t off = (int64_t)j * W;
      if (a.ldw != a.K) off += (int64_t)((uint32_t)(j / sizeof(T)) / a.per_row) * (a.ldw - a.K);
      __builtin_memcpy(&q[u], static_cast<const T*>(a.w) + off, 16);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      uint32_t t = top_bits<T>(q[u]);
      if (t < kInf) {
        m = max(m, t);
      } else {
        const uint32_t mask = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFFu;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          t = q[u][e * sizeof(T) / 4] >> (e * sizeof(T) % 4 * 8) & mask;
          m = max(m, t < kInf ? t : 0u);
        }
      }
    }
  }
  __shared__ uint32_t part[kMaxThreads / 64];
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kMaxThreads / 64; ++i) m = max(m, part[i]);
    typedef std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t> Bits;
    a.partial[blockIdx.x] = __float_as_uint((float)__builtin_bit_cast(T, (Bits)m));
  }
}

// One thread takes 16 elements: an NVFP4 group, or half of an MXFP4 group (the
// halves trade their maxima with the neighbouring lane).
template <typename T, int FMT>
__device__ __forceinline__ void codes_of(const QuantArgs& a, uint64_t i, const Raw16<T>& raw, float gs) {
  float v[16];
  to_f32(raw, v);
  uint32_t sbyte;
  u32x2 codes;
  round16<FMT, sizeof(T) == 2>(v, gs, sbyte, codes);
  *reinterpret_cast<u32x2*>(a.codes + i * 8) = codes;
  if constexpr (FMT == kNv) a.scales[i] = (uint8_t)sbyte;
  else if ((i & 1) == 0) a.scales[i >> 1] = (uint8_t)sbyte;
}

// A thread goes on to the next group of its grid, whose load is under way while it
// works on this one; a wavefront joins the per-block maxima once, not per group.
template <typename T, int FMT>
__global__ __launch_bounds__(kThreads) void k_fp4_codes(QuantArgs a) {
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  Raw16<T> raw = load16_of<T>(a, (uint32_t)min(i, (uint64_t)a.n16 - 1));
  float gs = 1.0f;
  if constexpr (FMT == kNv) {
    if (a.partial) {
      uint32_t m = 0;
      for (int p = threadIdx.x & 63; p < a.nparts; p += 64) m = max(m, a.partial[p]);
      gs = __uint_as_float(wave_max(m)) / 2688.0f;
      if (!(gs > 0.0f)) gs = 1.0f;   // a matrix of zeros
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.gs = gs;
    } else {
      gs = *a.gs;
    }
  }
  for (; i < a.n16; i += stride) {
    const Raw16<T> next = load16_of<T>(a, (uint32_t)min(i + stride, (uint64_t)a.n16 - 1));
    codes_of<T, FMT>(a, i, raw, gs);
    raw = next;
  }
}

// ---- reading back ------------------------------------------------------------
// A thread writes 16 bytes at a time, so that a wavefront's stores are one piece.
template <int FMT, typename T>
__global__ __launch_bounds__(kThreads) void k_fp4_values(const uint8_t* codes, const uint8_t* scales, const float* gsp,
                                                         T* out, int64_t ld, uint64_t n, uint32_t K) {
  constexpr int W = 16 / sizeof(T), G = FMT == kNv ? 16 : 32;
  typedef __attribute__((ext_vector_type(W))) T TW;
  const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const float gs = gsp ? *gsp : 1.0f;
  uint32_t d;
  if constexpr (W == 8) d = reinterpret_cast<const uint32_t*>(codes)[i];
  else d = reinterpret_cast<const uint16_t*>(codes)[i];
  const uint32_t sb = scales[i * W / G];
  const float s = FMT == kNv ? __builtin_amdgcn_cvt_pk_f32_fp8((int)sb, false)[0] : e8m0(sb);
  float v[W];
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    const f32x2 t = e == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0)
                    : e == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1)
                    : e == 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2)
                             : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
    // code times group scale is exact; one rounding by the matrix scale
    v[e] = t.x * s * gs;
    v[e + 1] = t.y * s * gs;
  }
  int64_t off = (int64_t)i * W;
  if (ld != K) {
    const uint32_t g16 = (uint32_t)(i * W / 16), row = g16 / (K / 16);     // fits: check_fp4_matrix
    off += (int64_t)row * (ld - K);
  }
  TW o;
#pragma unroll
  for (int e = 0; e < W; ++e) o[e] = (T)v[e];
  __builtin_memcpy(out + off, &o, sizeof o);
}

unsigned blocks_of(uint64_t n) { return (unsigned)((n + kThreads - 1) / kThreads); }
int type_size(int t) { return t == SC_DTYPE_F32 ? 4 : 2; }

template <typename T>
hipError_t run_quantize(const QuantArgs& a, int fmt, hipStream_t st) {
  if (a.partial) hipLaunchKernelGGL((k_fp4_max<T>), dim3(a.nparts), dim3(kMaxThreads), 0, st, a);
  const unsigned blocks = blocks_of(a.n16), grid = blocks < kGrid ? blocks : kGrid;
  if (fmt == SC_FP4_NV) hipLaunchKernelGGL((k_fp4_codes<T, kNv>), dim3(grid), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((k_fp4_codes<T, kMx>), dim3(grid), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

// Rows at a time: a launch has less than 2^32 threads, and runs only part of a larger grid without an error.
template <typename T>
hipError_t run_values(const sc_fp4_matrix* m, void* out, int64_t ld, hipStream_t st) {
  constexpr int W = 16 / sizeof(T);
  const int64_t cols = m->cols, most = ((int64_t)1 << 31) * W / cols;
  for (int64_t r = 0; r < m->rows; r += most) {
    const uint64_t n = (uint64_t)(m->rows - r < most ? m->rows - r : most) * cols / W;
    const unsigned grid = blocks_of(n);
    const uint8_t* c = static_cast<const uint8_t*>(m->d_codes) + r * (cols / 2);
    const uint8_t* s = static_cast<const uint8_t*>(m->d_scales) + r * (cols / (m->format == SC_FP4_NV ? 16 : 32));
    T* o = static_cast<T*>(out) + r * ld;
    if (m->format == SC_FP4_NV)
      hipLaunchKernelGGL((k_fp4_values<kNv, T>), dim3(grid), dim3(kThreads), 0, st, c, s, m->d_global_scale, o, ld, n,
                         (uint32_t)cols);
    else
      hipLaunchKernelGGL((k_fp4_values<kMx, T>), dim3(grid), dim3(kThreads), 0, st, c, s, m->d_global_scale, o, ld, n,
                         (uint32_t)cols);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

sc_status check_fp4_matrix(const sc_fp4_matrix* w) {
  if (!w) return fail(SC_E_ARG, "matrix is NULL");
  if (w->format != SC_FP4_NV && w->format != SC_FP4_MX) return fail(SC_E_ARG, "unknown format %d", w->format);
  const int g = w->format == SC_FP4_NV ? 16 : 32;
  if (w->rows < 0) return fail(SC_E_ARG, "rows must be >= 0");
  if (w->cols < g || w->cols % g || w->cols > kMaxFp4Cols)
    return fail(SC_E_ARG, "cols must be a positive multiple of %d and at most %d", g, kMaxFp4Cols);
  if ((uint64_t)w->rows * w->cols / 16 > 0xFFFFFFFFull) return fail(SC_E_ARG, "matrix has too many elements");
  if (w->rows == 0) return SC_OK;
  if (!w->d_codes || !w->d_scales) return fail(SC_E_ARG, "codes or scales are NULL");
  if ((uintptr_t)w->d_codes % 16 || (uintptr_t)w->d_scales % 2 || (uintptr_t)w->d_global_scale % 4)
    return fail(SC_E_ARG, "codes must be 16-byte aligned, scales 2-byte, the global scale 4-byte");
  return SC_OK;
}

}  // namespace sc

using namespace sc;

extern "C" {

sc_status fp4_quantize(const void* d_w, int32_t w_type, int64_t ldw, const sc_fp4_matrix* out, int32_t scale_given,
                       void* d_workspace, void* stream) {
  sc_status s = check_fp4_matrix(out);
  if (s != SC_OK) return s;
  if (w_type != SC_DTYPE_BF16 && w_type != SC_DTYPE_F16 && w_type != SC_DTYPE_F32)
    return fail(SC_E_ARG, "unknown w_type %d", w_type);
  if (ldw < out->cols) return fail(SC_E_ARG, "the row stride must cover the row");
  const bool nv = out->format == SC_FP4_NV;
  if (nv && !out->d_global_scale) return fail(SC_E_ARG, "NVFP4 needs a global scale");
  if (nv && !scale_given && (!d_workspace || (uintptr_t)d_workspace % 4))
    return fail(SC_E_ARG, "the max over the matrix needs a 4-byte aligned workspace");
  if (out->rows == 0) return SC_OK;
  const int size = type_size(w_type);
  if (!d_w || (uintptr_t)d_w % size) return fail(SC_E_ARG, "w is NULL or not aligned to its elements");
  QuantArgs a{};
  a.w = d_w;
  a.ldw = ldw;
  a.codes = static_cast<uint8_t*>(out->d_codes);
  a.scales = static_cast<uint8_t*>(out->d_scales);
  a.gs = out->d_global_scale;
  a.K = out->cols;
  a.per_row = (uint32_t)out->cols / 16;
  a.n16 = (uint32_t)out->rows * a.per_row;
  if (nv && !scale_given) {
    a.partial = static_cast<uint32_t*>(d_workspace);
    // one block per 16 KB until the card is full
    const uint64_t blocks = ((uint64_t)a.n16 * 16 * size + 16383) / 16384;
    a.nparts = (int)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = w_type == SC_DTYPE_F32   ? run_quantize<float>(a, out->format, st)
                       : w_type == SC_DTYPE_F16 ? run_quantize<_Float16>(a, out->format, st)
                                                : run_quantize<__bf16>(a, out->format, st);
  if (e != hipSuccess) return hip_fail(e, "fp4_quantize launch");
  return SC_OK;
}

sc_status fp4_dequantize(const sc_fp4_matrix* w, void* d_w, int32_t w_type, int64_t ldw, void* stream) {
  sc_status s = check_fp4_matrix(w);
  if (s != SC_OK) return s;
  if (w_type != SC_DTYPE_BF16 && w_type != SC_DTYPE_F16 && w_type != SC_DTYPE_F32)
    return fail(SC_E_ARG, "unknown w_type %d", w_type);
  if (ldw < w->cols) return fail(SC_E_ARG, "the row stride must cover the row");
  if (w->rows == 0) return SC_OK;
  if (!d_w || (uintptr_t)d_w % type_size(w_type)) return fail(SC_E_ARG, "w is NULL or not aligned to its elements");
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = w_type == SC_DTYPE_F32   ? run_values<float>(w, d_w, ldw, st)
                       : w_type == SC_DTYPE_F16 ? run_values<_Float16>(w, d_w, ldw, st)
                                                : run_values<__bf16>(w, d_w, ldw, st);
  if (e != hipSuccess) return hip_fail(e, "fp4_dequantize launch");
  return SC_OK;
}

}  // extern "C"
