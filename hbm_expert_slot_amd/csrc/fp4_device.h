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

// A buffer descriptor over [p, p + bytes): a load whose offset lies beyond it
// returns zeros and touches no memory, so tails need no branches.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
constexpr uint32_t kBeyond = 0x80000000u;   // an offset that lies beyond every descriptor
constexpr int kStream = 2;                  // nontemporal: weights are read once per call

__device__ __forceinline__ u32x4 load16(Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kStream);
}
__device__ __forceinline__ u32x2 load8(Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, kStream);
}
__device__ __forceinline__ uint32_t load2(Rsrc r, uint32_t off) {
  return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, kStream);
}
__device__ __forceinline__ uint32_t load1(Rsrc r, uint32_t off) {
  return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, (int)off, 0, kStream);
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
template <bool HALF>
__device__ __forceinline__ f32x4 mfma4(u32x2 x, u32x2 w, f32x4 c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, x), __builtin_bit_cast(f16x4, w), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, x), __builtin_bit_cast(s16x4, w), c, 0, 0,
                                                  0);
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

// Byte offsets of a lane in a quad's rows.  codes: row * K/2, scales: row * K/G.
template <int FMT, bool ODD, int Q>
__device__ __forceinline__ void load_stage(Stage<FMT, ODD, Q>& st, Rsrc rc, Rsrc rs, uint32_t code0, uint32_t scale0,
                                           uint32_t code_quad, uint32_t scale_quad, int k, int K) {
  // lanes past the end of the row read nothing: codes and scales are zero there
  const bool in = k < K;
#pragma unroll
  for (int j = 0; j < Q; ++j) {
    const uint32_t oc = code0 + j * code_quad + (uint32_t)k / 2;
    if constexpr (ODD) {
      // an odd number of groups per row: rows are 8-byte aligned, scale pairs
      // may lie at odd addresses, and the row may end between the two groups
      const bool in2 = k + 16 < K;
      const u32x2 lo = load8(rc, in ? oc : kBeyond), hi = load8(rc, in2 ? oc + 8 : kBeyond);
      st.q[j] = u32x4{lo.x, lo.y, hi.x, hi.y};
      const uint32_t os = scale0 + j * scale_quad + (uint32_t)k / 16;
      st.s[j] = load1(rs, in ? os : kBeyond) | load1(rs, in2 ? os + 1 : kBeyond) << 8;
      continue;
    }
    st.q[j] = load16(rc, in ? oc : kBeyond);
    if constexpr (FMT == kMx) {
      st.s[j] = load1(rs, in ? scale0 + j * scale_quad + (uint32_t)k / 32 : kBeyond);
    } else {
      st.s[j] = load2(rs, in ? scale0 + j * scale_quad + (uint32_t)k / 16 : kBeyond);
    }
  }
}

// acc[j][r] += sum of the stage's products with operand row r.  xs[a] + at: the
// lane's operand row of set a (row 4a + l % 4) in LDS, 32 elements at this step.
// A lane of a row behind the last reads any memory: its results are not used.
//
// SPLIT: the operand is fp32, held as three bf16 parts that add up to it (24
// bits).  With one row the parts stand as three rows of its set and their sums
// are added; otherwise part p lies at + p * part_bytes and the matrix
// instructions add all three into one sum.
template <int FMT, bool ODD, int Q, int ROWS, bool HALF, bool SPLIT = false>
__device__ __forceinline__ void use_stage(const Stage<FMT, ODD, Q>& st,
                                          const uint8_t* const (&xs)[(ROWS + 3) / 4], int at, float (&acc)[Q][ROWS],
                                          int part_bytes = 0) {
  constexpr int NA = (ROWS + 3) / 4, NP = SPLIT && ROWS > 1 ? 3 : 1;
  f32x2 sc[Q];
#pragma unroll
  for (int j = 0; j < Q; ++j) sc[j] = lane_scales<FMT>(st.s[j]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x2 w[Q][4];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const uint32_t d0 = h == 0 ? st.q[j].x : st.q[j].z, d1 = h == 0 ? st.q[j].y : st.q[j].w;
      w[j][0] = widen4<HALF, 0>(d0);
      w[j][1] = widen4<HALF, 2>(d0);
      w[j][2] = widen4<HALF, 0>(d1);
      w[j][3] = widen4<HALF, 2>(d1);
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      f32x4 p[Q];
#pragma unroll
      for (int j = 0; j < Q; ++j) p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        const uint8_t* x = xs[a] + at + t * part_bytes + h * 32;
        const u32x4 x0 = *reinterpret_cast<const u32x4*>(x), x1 = *reinterpret_cast<const u32x4*>(x + 16);
#pragma unroll
        for (int j = 0; j < Q; ++j) p[j] = mfma4<HALF>(u32x2{x0.x, x0.y}, w[j][0], p[j]);
#pragma unroll
        for (int j = 0; j < Q; ++j) p[j] = mfma4<HALF>(u32x2{x0.z, x0.w}, w[j][1], p[j]);
#pragma unroll
        for (int j = 0; j < Q; ++j) p[j] = mfma4<HALF>(u32x2{x1.x, x1.y}, w[j][2], p[j]);
#pragma unroll
        for (int j = 0; j < Q; ++j) p[j] = mfma4<HALF>(u32x2{x1.z, x1.w}, w[j][3], p[j]);
      }
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const float s = h == 0 ? sc[j].x : sc[j].y;
        if constexpr (SPLIT && ROWS == 1) {
          acc[j][0] = fmaf(p[j][0] + (p[j][1] + p[j][2]), s, acc[j][0]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (a * 4 + r < ROWS) acc[j][a * 4 + r] = fmaf(p[j][r], s, acc[j][a * 4 + r]);
        }
      }
    }
  }
}

}  // namespace fp4
}  // namespace sc
