// Device helpers of the 4-bit weight operators: guarded loads through buffer
// descriptors, FP4 widening, and products of a few operand rows with 4-bit
// weights on the 4x4x4 matrix instruction.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace sc {
namespace fp4 {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// 4-bit formats: E2M1 codes with one E4M3 scale per 16 elements (and an fp32
// scale of the matrix), or with one E8M0 scale per 32.
enum Format { kNv = 0, kMx = 1 };

// The lane, hidden from the optimiser: what depends on it is computed where it
// is used.  In a kernel of many phases it would else be moved out of the task
// loops and spilled, and each reload waits for every load in flight.
__device__ __forceinline__ int fresh_lane() {
  int lane;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(lane));
  return lane;
}
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
__device__ __forceinline__ int fresh_thread() { return wave_index() * 64 + fresh_lane(); }

// A buffer descriptor over [p, p + bytes).  A load whose lane offset is kBeyond
// returns zeros and touches no memory, so tails need no branches; every other
// lane offset plus the uniform one stays within the bytes.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t kBeyond = 0x80000000u;   // lies beyond every descriptor
constexpr int kStream = 2;                  // nontemporal: weights are read once per call
constexpr int kReuse = 0;                   // cached: several blocks read them

// lane: offset of the lane; at: uniform offset
template <int AUX = kStream>
__device__ __forceinline__ u32x4 load16(Rsrc r, uint32_t lane, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)lane, (int)at, AUX);
}
template <int AUX = kStream>
__device__ __forceinline__ u32x2 load8(Rsrc r, uint32_t lane, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, (int)lane, (int)at, AUX);
}
template <int AUX = kStream>
__device__ __forceinline__ uint32_t load2(Rsrc r, uint32_t lane, uint32_t at) {
  return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)lane, (int)at, AUX);
}
template <int AUX = kStream>
__device__ __forceinline__ uint32_t load1(Rsrc r, uint32_t lane, uint32_t at) {
  return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)lane, (int)at, AUX);
}

// Four codes (bytes B and B+1 of d) as bf16 or fp16.  The conversions are
// exact; the byte selector has to be an immediate.
template <bool HALF, int B>
__device__ __forceinline__ u32x2 widen4(uint32_t d) {
  u32x2 w;
  if constexpr (HALF) {
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, B));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, B + 1));
  } else {
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, B));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, B + 1));
  }
  return w;
}

// Sixteen independent 4x4 tiles, four products deep.  Lane l works on tile
// l / 4: it holds row l % 4 of the operand and column l % 4 of the weights
// (four consecutive K-elements each) and gets column l % 4 of the result, its
// four rows in the four registers.  Products are exact, sums are fp32.
//
// KEEP: the operands live until the result is there, so that no result is written
// over them; and the instructions stay in the order written, which needs fewer
// registers (16 rows of the MoE layer: 168 to 158, and 442 to 422 us; without
// "volatile" the compiler stretches their lives and spills).  A kernel whose sums
// the compiler places in the accumulation registers has the first by itself.
#ifdef FP4_SUMS_IN_VGPRS
constexpr bool kKeepOperands = true;
#else
constexpr bool kKeepOperands = false;
#endif
template <bool HALF, bool KEEP>
__device__ __forceinline__ f32x4 mfma4(u32x2 x, u32x2 w, f32x4 c) {
  f32x4 d;
  if constexpr (HALF)
    d = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, x), __builtin_bit_cast(f16x4, w), c, 0, 0, 0);
  else
    d = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, x), __builtin_bit_cast(s16x4, w), c, 0, 0, 0);
  if constexpr (KEEP) asm volatile("" : "+v"(d) : "v"(x), "v"(w));
  return d;
}

// An E8M0 byte: 2^(b - 127); 255 is NaN.
__device__ __forceinline__ float e8m0(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23;
  return __uint_as_float(bits);
}

// The two scales of a lane's 32 elements of one step.
template <int FMT>
__device__ __forceinline__ f32x2 lane_scales(uint32_t raw) {
  if constexpr (FMT == kNv) {
    return __builtin_amdgcn_cvt_pk_f32_fp8((int)raw, false);
  } else {
    const float s = e8m0(raw);
    return f32x2{s, s};
  }
}

// Sums over lanes that agree in lane % 4 (the sixteen tiles).  V values per
// lane (a power of two) are halved while there are pairs to trade: after the
// two lane-swap steps a lane holds the totals of kTileOut<V> values, from
// tile_sum_first on.  Every total is added in the same tree, whatever V is.
template <int O>
__device__ __forceinline__ float swap_sum(float a, float b) {
  if constexpr (O == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
// Sums over the lanes up to each.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = dpp_add<0x111, 0xF>(v);      // from 1, 2, 4 and 8 lanes before in the row of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);      // a row's last lane to the next row, the second row's to both behind
  return dpp_add<0x143, 0xC>(v);
}
template <int V>
constexpr int kTileOut = V >= 4 ? V / 4 : 1;
template <int V>
__device__ __forceinline__ void tile_sum(float (&v)[V]) {
  static_assert((V & (V - 1)) == 0, "values are traded in pairs");
  constexpr int H1 = V >= 2 ? V / 2 : 1, H2 = kTileOut<V>;
#pragma unroll
  for (int i = 0; i < H1; ++i) v[i] = swap_sum<32>(v[i], v[V >= 2 ? i + H1 : i]);
#pragma unroll
  for (int i = 0; i < H2; ++i) v[i] = swap_sum<16>(v[i], v[V >= 4 ? i + H2 : i]);
#pragma unroll
  for (int i = 0; i < H2; ++i) {
    v[i] += dpp<0x128>(v[i]);   // rotated by 8 in the row of 16
    v[i] += dpp<0x124>(v[i]);   // and by 4
  }
}
// First value that a lane holds, and whether it is the lane that hands it on.
template <int V>
__device__ __forceinline__ int tile_sum_first(int lane) {
  return (V >= 2 ? ((lane >> 5) & 1) * (V / 2) : 0) + (V >= 4 ? ((lane >> 4) & 1) * (V / 4) : 0);
}
template <int V>
__device__ __forceinline__ bool tile_sum_owner(int lane) {
  return (lane & (V >= 4 ? 12 : V >= 2 ? 28 : 60)) == 0;
}

// ---- few rows against 4-bit weights ------------------------------------------
//
// A wavefront owns Q quads of weight rows.  In one step its lanes cover 512
// K-elements of each of a quad's four rows: lane l takes 32 elements (16 bytes
// of codes, 256 contiguous bytes per row across the wavefront) of row l % 4.
// The block's operand rows lie in LDS; each matrix instruction multiplies four
// of them by the lane's four weights.  A scale group never leaves its lane, so
// its sum over exact products is scaled once, in fp32: per weight half a
// conversion and ROWS/16 (NVFP4) multiply-adds, whatever the row count.
constexpr int kStepK = 512;

template <int FMT, bool ODD, int Q>
struct Stage {
  u32x4 q[Q];
  uint32_t s[Q];
};

// What a lane reads of a matrix: its own offsets (row l % 4 of a quad, element
// 32 (l / 4) of a step) and the distances between a wavefront's quads.
template <int FMT>
struct Reader {
  Rsrc rc, rs;
  uint32_t code, scale;              // of the lane
  uint32_t row_code, row_scale;      // bytes per row
  int klane;
};
template <int FMT>
__device__ __forceinline__ Reader<FMT> reader(const uint8_t* codes, const uint8_t* scales, uint32_t rows, int K) {
  constexpr int G = FMT == kNv ? 16 : 32;
  const int lane = fresh_lane();
  Reader<FMT> r;
  r.row_code = (uint32_t)K / 2;
  r.row_scale = (uint32_t)K / G;
  r.rc = make_rsrc(codes, rows * r.row_code);
  r.rs = make_rsrc(scales, rows * r.row_scale);
  r.klane = (lane >> 2) * 32;
  r.code = (lane & 3) * r.row_code + r.klane / 2;
  r.scale = (lane & 3) * r.row_scale + r.klane / G;
  return r;
}

// Step at element k of quads row, row + apart, ...: `in` says that the lane's
// row is there; lanes past kend read nothing (codes and scales are zero there).
template <int FMT, bool ODD, int Q>
__device__ __forceinline__ void load_stage(Stage<FMT, ODD, Q>& st, const Reader<FMT>& r, uint32_t row, uint32_t apart,
                                           int k, int kend, const bool (&in)[Q]) {
  constexpr int G = FMT == kNv ? 16 : 32;
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    const uint32_t ac = (row + j * apart) * r.row_code + k / 2, as = (row + j * apart) * r.row_scale + k / G;
    const bool on = r.klane + k < kend && in[j];
    const uint32_t lc = on ? r.code : kBeyond, ls = on ? r.scale : kBeyond;
    if constexpr (ODD) {
      // an odd number of groups per row: rows are 8-byte aligned, scale pairs
      // may lie at odd addresses, and the row may end between the two groups
      const bool on2 = r.klane + k + 16 < kend && in[j];
      const u32x2 lo = load8(r.rc, lc, ac), hi = load8(r.rc, on2 ? r.code + 8 : kBeyond, ac);
      st.q[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
      st.s[j] = load1(r.rs, ls, as) | load1(r.rs, on2 ? r.scale + 1 : kBeyond, as) << 8;
    } else {
      st.q[j] = load16(r.rc, lc, ac);
      st.s[j] = FMT == kMx ? load1(r.rs, ls, as) : load2(r.rs, ls, as);
    }
  }
}

// acc[j][r] += sum of the stage's products with operand row r.  xs[a] + at: the
// lane's operand row of set a (row 4a + l % 4) in LDS, 32 elements at this step.
// A lane of a row behind the last reads any memory: its results are not used.
//
// W quads are worked on at a time: their widened codes are live together, and
// their chains of matrix instructions run side by side.
//
// SPLIT: the operand is fp32, held as three bf16 parts that add up to it (24
// bits).  With one row the parts stand as three rows of its set and their sums
// are added; otherwise part p lies at + p * part_bytes and the matrix
// instructions add all three into one sum.
template <int FMT, bool ODD, int Q, int ROWS, bool HALF, bool SPLIT = false, int W = Q < 2 ? Q : 2, bool KEEP = kKeepOperands>
__device__ __forceinline__ void use_stage(const Stage<FMT, ODD, Q>& st,
                                          const uint8_t* const (&xs)[(ROWS + 3) / 4], int at, float (&acc)[Q][ROWS],
                                          int part_bytes = 0) {
  constexpr int NA = (ROWS + 3) / 4, NP = SPLIT && ROWS > 1 ? 3 : 1;
  static_assert(Q % W == 0, "");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      u32x4 x[NP][2];
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        const uint8_t* px = xs[a] + at + t * part_bytes + h * 32;
        x[t][0] = *reinterpret_cast<const u32x4*>(px);
        x[t][1] = *reinterpret_cast<const u32x4*>(px + 16);
      }
#pragma unroll
      for (int j0 = 0; j0 < Q; j0 += W) {
        u32x2 w[W][4];
        f32x4 p[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const u32x4& q = st.q[j0 + j];
          const uint32_t d0 = h == 0 ? q.x : q.z, d1 = h == 0 ? q.y : q.w;
          w[j][0] = widen4<HALF, 0>(d0);
          w[j][1] = widen4<HALF, 2>(d0);
          w[j][2] = widen4<HALF, 0>(d1);
          w[j][3] = widen4<HALF, 2>(d1);
          p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int t = 0; t < NP; ++t) {
#pragma unroll
          for (int j = 0; j < W; ++j) p[j] = mfma4<HALF, KEEP>(u32x2{x[t][0].x, x[t][0].y}, w[j][0], p[j]);
#pragma unroll
          for (int j = 0; j < W; ++j) p[j] = mfma4<HALF, KEEP>(u32x2{x[t][0].z, x[t][0].w}, w[j][1], p[j]);
#pragma unroll
          for (int j = 0; j < W; ++j) p[j] = mfma4<HALF, KEEP>(u32x2{x[t][1].x, x[t][1].y}, w[j][2], p[j]);
#pragma unroll
          for (int j = 0; j < W; ++j) p[j] = mfma4<HALF, KEEP>(u32x2{x[t][1].z, x[t][1].w}, w[j][3], p[j]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const f32x2 sc = lane_scales<FMT>(st.s[j0 + j]);
          const float s = h == 0 ? sc.x : sc.y;
          if constexpr (SPLIT && ROWS == 1) {
            acc[j0 + j][0] = fmaf(p[j][0] + (p[j][1] + p[j][2]), s, acc[j0 + j][0]);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (a * 4 + r < ROWS) acc[j0 + j][a * 4 + r] = fmaf(p[j][r], s, acc[j0 + j][a * 4 + r]);
          }
        }
      }
    }
  }
}

}  // namespace fp4
}  // namespace sc
