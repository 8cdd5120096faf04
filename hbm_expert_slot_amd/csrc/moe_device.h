// What the kernels of the whole MoE layer share: their arguments, the hand-over
// between blocks, and the routing.
//
// What one block hands to another goes through stores and loads at agent scope
// (each XCD has an L2 of its own): written through, waited for, then counted or
// flagged.  A release fence would write back every dirty line of the L2 instead,
// other kernels' among them (measured: 12 of 21 us of a router product).
// Logits and picks are their own flags: a word that is not there yet holds a
// value that no result has, and whoever needs it polls the word itself.
#pragma once

#define FP4_SUMS_IN_VGPRS    // three blocks of 256 or one of 768 threads per compute unit
#include "fp4_device.h"
#include "internal.h"

#include <limits>
#include <type_traits>

namespace sc {
namespace moe {

using namespace fp4;

constexpr int kMaxTokens = SC_MOE_MAX_ROWS;
constexpr int kPad = 16;           // bytes between operand rows in LDS: four rows' reads fall into different banks
constexpr int kRouterShares = 4;   // shares of H in the router product of five rows and more
constexpr int kShards = 16, kLine = 32;   // parts of a counter, and words per cache line

// Polls of a wait before the call is given up (about a second): only a
// workspace that was not prepared, or that two calls share, gets there.
constexpr int kMaxPolls = 1 << 21;

struct MoeArgs {
  const uint16_t* router;    // [E][H] bf16
  const float* score_bias;   // [E] or null
  const uint8_t* blobs;      // [E][blob]
  const float* gs;           // [E][2]
  const uint8_t* shared;     // blob of the shared expert or null
  const float* sgs;          // [2]
  const uint16_t* x;         // [M][H]
  void* y;                   // [M][H]
  int32_t* ids_out;          // [M][k] or null
  float* w_out;              // [M][k] or null
  int32_t* ctl;              // control words, zero between calls
  uint32_t* logits;          // [KS][M][E] partial sums over shares of H, kNoLogit between calls
  uint64_t* picks;           // [P] expert + 1 and weight, 0 between calls
  float* h;                  // [P][I], then [M][Is] of the shared expert
  float* part;               // [P][H], then [M][H]
  int64_t ldx, ldy, blob;
  int M, H, I, E, k, Is, score, out, vec;
  int lds;                   // bytes of LDS for operand rows
  int dense;                 // x lies in LDS whole, token by token
  int router_tiles, ks;      // ks: shares of H in the router product
  int logit_words;           // of the workspace
  float scale;
};

// Hand-over between blocks.
template <typename T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T* p) {
  return __hip_atomic_load(const_cast<T*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int add(int32_t* p, int v) {
  return __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
constexpr int kAgent = 16;   // buffer load at agent scope (sc1)
// The wavefront's stores have been performed.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// One poll of a wait that has lasted `i` polls: false when the call is given up.
__device__ __forceinline__ bool poll_on(int32_t* error, int i) {
  if (i >= kMaxPolls) put(error, 1);
  if ((i & 63) == 63 && get(error)) return false;
  __builtin_amdgcn_s_sleep(4);
  return true;
}

// ---- routing -------------------------------------------------------------------

constexpr uint32_t kNoLogit = 0xFFFFFFFFu;   // a NaN that no logit is: NaN logits are stored as 0x7FC00000
__device__ __forceinline__ void put_logit(uint32_t* p, float z) {
  put(p, z != z ? 0x7FC00000u : __float_as_uint(z));
}

__device__ __forceinline__ u32x4 load_x8(const MoeArgs& a, const uint16_t* p) {
  if (a.vec) return *reinterpret_cast<const u32x4*>(p);
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
  return v;
}

constexpr int kTileWaves = 4;

// Logits of four experts for up to MR (4) rows: each wavefront sums a quarter of
// H, all its loads in flight together up to H = 6144, and the quarters are added
// in wavefront order.
template <int MR>
__device__ __forceinline__ void router_tile(const MoeArgs& a, int tile, float* red) {
  constexpr int EB = 4, V = EB * MR, N = 3;
  const int lane = fresh_lane(), wave = threadIdx.x >> 6;
  const int e0 = tile * EB;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  for (int c0 = (wave * 64 + lane) * 8; c0 < a.H; c0 += N * (64 * kTileWaves) * 8) {
    u32x4 w[N][EB], x[N][MR];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = min(c0 + n * (64 * kTileWaves) * 8, a.H - 8);
#pragma unroll
      for (int m = 0; m < MR; ++m) x[n][m] = load_x8(a, a.x + min(m, a.M - 1) * a.ldx + c);
#pragma unroll
      for (int e = 0; e < EB; ++e)
        w[n][e] = *reinterpret_cast<const u32x4*>(a.router + (int64_t)min(e0 + e, a.E - 1) * a.H + c);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (c0 + n * (64 * kTileWaves) * 8 >= a.H) break;
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[m * EB + e] =
                __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (uint32_t)w[n][e][i]),
                                                __builtin_bit_cast(bf16x2, (uint32_t)x[n][m][i]), acc[m * EB + e], false);
    }
  }
  tile_sum<V>(acc);
#pragma unroll
  for (int i = 0; i < kTileOut<V>; ++i) {
    acc[i] += dpp<0x4E>(acc[i]);
    acc[i] += dpp<0xB1>(acc[i]);
  }
  if (tile_sum_owner<V>(lane) && (lane & 3) == 0) {
    const int first = tile_sum_first<V>(lane);
#pragma unroll
    for (int i = 0; i < kTileOut<V>; ++i) red[wave * V + first + i] = acc[i];
  }
  __syncthreads();
  const int i = threadIdx.x, m = i / EB, e = e0 + i % EB;
  if (i < V && m < a.M && e < a.E)
    put_logit(&a.logits[m * a.E + e], ((red[i] + red[V + i]) + red[2 * V + i]) + red[3 * V + i]);
}

// From five rows on: 16 experts and one of `ks` shares of H on the 16x16x32
// matrix instruction (rows of x times rows of the router; lane l holds row
// l % 16 of both, elements 8 (l / 16) .. + 7 of 32).  Four shares, so that the
// products of 256 experts are spread over 64 blocks.
__device__ __forceinline__ void router_tile_mfma(const MoeArgs& a, int tile, float* red) {
  typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
  constexpr int N = 12;
  const int lane = fresh_lane(), wave = threadIdx.x >> 6;
  const int share = tile % a.ks, e0 = tile / a.ks * 16, stride = a.ks * kTileWaves * 32;
  const uint16_t* pw = a.router + (int64_t)min(e0 + (lane & 15), a.E - 1) * a.H + (lane >> 4) * 8;
  const uint16_t* px = a.x + min(lane & 15, a.M - 1) * a.ldx + (lane >> 4) * 8;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = (share * kTileWaves + wave) * 32; k0 < a.H; k0 += N * stride) {
    u32x4 w[N], x[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int k = min(k0 + n * stride, a.H - 32);
      w[n] = *reinterpret_cast<const u32x4*>(pw + k);
      x[n] = load_x8(a, px + k);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (k0 + n * stride >= a.H) break;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[n]), __builtin_bit_cast(bf16x8, w[n]),
                                                    acc, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) red[(wave * 4 + i) * 64 + lane] = acc[i];
  __syncthreads();
  const int i = threadIdx.x;
  const float z = ((red[i] + red[256 + i]) + red[512 + i]) + red[768 + i];
  const int m = (i >> 4 & 3) * 4 + (i >> 6), e = e0 + (i & 15);   // lane i % 64 of register i / 64
  if (m < a.M && e < a.E) put_logit(&a.logits[(share * a.M + m) * a.E + e], z);
}

// Keys that order as the scores do: NaN below -inf, -0 equal to +0.
__device__ __forceinline__ int order_key(float z) {
  if (z != z) return INT32_MIN + 1;
  const int b = (int)__float_as_uint(z + 0.0f);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}
__device__ __forceinline__ int64_t order_key(double z) {
  if (z != z) return INT64_MIN + 1;
  const int64_t b = __double_as_longlong(z + 0.0);
  return b >= 0 ? b : b ^ INT64_MAX;
}

// What the picks are ordered by.  Sigmoids without a bias order as their logits do,
// also where they are one fp32 number (from 17.3 on all are 1).  With one the sum is
// formed in fp64 from the sigmoid's distance to 0 or 1, t / (1 + t) with t =
// exp(-|z|), whose relative error of |z| 2^-23 and a few steps is the logit's own.
// In the kernels of up to four rows its fp32 rounding settles nearly every pick, and
// where two of those agree, exact_picks does: one row, 8 of 1000 experts of 1024 x 256,
// 24.3 us, with a bias 25.1 (26.4 and 27.3 with 64-bit keys throughout).  The kernel of
// more rows has 64-bit keys: the call would cost its products registers (16 rows, 4 of
// 16 experts of 6144 x 2048: 135 us, 141 with the call).
__device__ __forceinline__ double exact_score(float z, float bias) {
  const float y = fabsf(z) * -1.4426950408889634f, n = __builtin_rintf(fmaxf(y, -2000.0f));
  const double t = ldexp((double)__builtin_amdgcn_exp2f(y - n), (int)n);
  const double d = t * (double)__builtin_amdgcn_rcpf(1.0f + (float)t);
  return (z > 0.0f ? 1.0 - d : z == z ? d : (double)z) + (double)bias;
}
template <typename Key>
__device__ __forceinline__ Key pick_key(const MoeArgs& a, float z, float bias) {
  if constexpr (sizeof(Key) == 8) return order_key(a.score_bias ? exact_score(z, bias) : (double)z);
  if (!a.score_bias) return order_key(z);
  const float t = __builtin_amdgcn_exp2f(fabsf(z) * -1.4426950408889634f), d = t * __builtin_amdgcn_rcpf(1.0f + t);
  return order_key((float)((double)bias + (z > 0.0f ? 1.0 - (double)d : (double)d)));
}

// Reductions over the wavefront in registers: halves and 16-lane rows trade by
// lane swaps, the rest through DPP.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F f) {
  auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = f(r[0], r[1]);
  r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(r[0], r[1]);
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  return f(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
}
__device__ __forceinline__ int wave_max_i(int v) {
  return (int)wave_reduce((uint32_t)v, [](uint32_t x, uint32_t y) { return (uint32_t)max((int)x, (int)y); });
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
  }));
}

// The lanes that have the largest key: by its upper half, then by the lower.  Every
// lane takes part in both reductions.
__device__ __forceinline__ uint64_t top_lanes(int64_t key) {
  const int hi = (int)(key >> 32), most_hi = wave_max_i(hi);
  const bool in = hi == most_hi;
  const uint64_t top = __ballot(in);
  if (!(top & (top - 1))) return top;
  const int lo = in ? (int)((uint32_t)key ^ 0x80000000u) : INT32_MIN, most_lo = wave_max_i(lo);
  return __ballot(in && lo == most_lo);
}

// The k experts of largest sigmoid and bias in fp64, one per lane; lane l looks
// after experts l * epl .. of the logits in LDS.  Not inlined: it hardly ever runs,
// and costs the kernels no registers.
static __device__ __noinline__ int exact_picks(const float* logits, const float* bias, int E, int k) {
  constexpr int EPL = kMaxExperts / 64;
  const int lane = fresh_lane(), epl = (E + 63) / 64;
  int64_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * epl + i;
    const bool in = i < epl && e < E;
    key[i] = in ? order_key(exact_score(logits[in ? e : 0], bias[in ? e : 0])) : INT64_MIN;
  }
  int my_id = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    int64_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < EPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const int src = __builtin_ctzll(top_lanes(best));
    const int e = src * epl + __builtin_amdgcn_readlane(at, src);
    if (lane == j) my_id = e;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane == src && i == at) key[i] = INT64_MIN;
  }
  return my_id;
}

// One wavefront picks row m's experts, lane j the j-th.  Lane l looks after
// experts l * epl .. and keeps them sorted (up to eight; more are looked through
// each time), so that a pick costs one reduction: the lowest lane with the
// largest key holds the lowest id.  sval: the logits, LDS, [E].  The logits are set back to
// kNoLogit.  After `patience` polls it returns kLate with nothing done.
enum Routed { kDone = 0, kLate, kGivenUp };
template <int EPL, int KS>
__device__ __forceinline__ Routed pick_row(const MoeArgs& a, int32_t* error, int m, float* sval, int patience,
                                           int& my_id, bool& tied) {
  constexpr bool SORT = EPL <= 8;
  typedef std::conditional_t<KS == 1, int, int64_t> Key;
  constexpr Key kNone = std::numeric_limits<Key>::min();
  const int lane = fresh_lane();
  const int epl = (a.E + 63) / 64;
  const Rsrc rl = make_rsrc(a.logits, (uint32_t)(KS * a.M * a.E) * 4);
  const Rsrc rb = make_rsrc(a.score_bias, a.score_bias ? (uint32_t)a.E * 4 : 0);   // none: zeros
  float bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * epl + i;
    bias[i] = __uint_as_float(
        __builtin_amdgcn_raw_buffer_load_b32(rb, i < epl && e < a.E ? e * 4 : (int)kBeyond, 0, 0));
  }
  constexpr int QB = EPL * KS <= 32 ? KS : 32 / EPL;   // shares loaded at a time
  float sum[EPL];
#pragma unroll
  for (int q0 = 0; q0 < KS; q0 += QB) {
    uint32_t part[EPL][QB];
    for (int poll = 0;; ++poll) {
      bool all = true;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * epl + i;
#pragma unroll
        for (int q = 0; q < QB; ++q)
          part[i][q] = __builtin_amdgcn_raw_buffer_load_b32(
              rl, i < epl && e < a.E ? (((q0 + q) * a.M + m) * a.E + e) * 4 : (int)kBeyond, 0, kAgent);
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i)
#pragma unroll
        for (int q = 0; q < QB; ++q) all = all && part[i][q] != kNoLogit;
      if (!__ballot(!all)) break;
      if (poll >= patience) return kLate;
      if (!poll_on(error, poll)) return kGivenUp;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
#pragma unroll
      for (int q = 0; q < QB; ++q)
        sum[i] = q0 + q == 0 ? __uint_as_float(part[i][q]) : sum[i] + __uint_as_float(part[i][q]);
  }
  Key key[EPL];
  int id[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float z = sum[i];
    const Key by = pick_key<Key>(a, z, bias[i]);
    id[i] = lane * epl + i;
    const bool in = i < epl && id[i] < a.E;
    if (in) {
      sval[id[i]] = z;
#pragma unroll
      for (int q = 0; q < KS; ++q) put(&a.logits[(q * a.M + m) * a.E + id[i]], kNoLogit);
    }
    key[i] = in ? by : kNone;
  }
  if constexpr (SORT) {
#pragma unroll
    for (int n = EPL - 1; n > 0; --n)
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const bool up = key[i + 1] > key[i];       // equal keys keep their order
        const Key k0 = key[i];
        const int i0 = id[i];
        key[i] = up ? key[i + 1] : k0;
        id[i] = up ? id[i + 1] : i0;
        key[i + 1] = up ? k0 : key[i + 1];
        id[i + 1] = up ? i0 : id[i + 1];
      }
  }
  Key last = kNone;
  my_id = 0;
  tied = false;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    Key best = key[0];
    int at = id[0];
    if constexpr (!SORT) {
#pragma unroll
      for (int i = 1; i < EPL; ++i)
        if (key[i] > best) {
          best = key[i];
          at = id[i];
        }
    }
    uint64_t top;
    if constexpr (KS == 1) {
      const int most = wave_max_i(best);
      tied = tied || most == last;
      last = most;
      top = __ballot(best == most);
    } else {
      top = top_lanes(best);
    }
    const int src = __builtin_ctzll(top);
    const int e = __builtin_amdgcn_readlane(at, src);
    if (lane == j) my_id = e;
    if constexpr (SORT) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        key[i] = lane == src ? (i + 1 < EPL ? key[i + 1] : kNone) : key[i];
        id[i] = lane == src && i + 1 < EPL ? id[i + 1] : id[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (id[i] == e) key[i] = kNone;
    }
  }
  if constexpr (KS == 1) {
    int rest = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) rest = max(rest, key[i]);
    const int next = wave_max_i(rest);
    tied = tied || next == last;
  }
  return kDone;
}

// One wavefront picks row m's experts and publishes them.
template <int KS>
__device__ __forceinline__ Routed route_row(const MoeArgs& a, int32_t* error, int m, float* sval,
                                            int patience = INT32_MAX) {
  int my_id;
  bool tied;      // two of the 32-bit keys picked, or the last of them and the next
  const Routed r = a.E <= 256   ? pick_row<4, KS>(a, error, m, sval, patience, my_id, tied)
                   : a.E <= 512 ? pick_row<8, KS>(a, error, m, sval, patience, my_id, tied)
                                : pick_row<16, KS>(a, error, m, sval, patience, my_id, tied);
  if (r != kDone) return r;
  // equal logits are a tie, equal fp32 sums need not be
  if (KS == 1 && a.score_bias && __ballot(tied)) my_id = exact_picks(sval, a.score_bias, a.E, a.k);
  const int lane = fresh_lane();
  // weights; NaN counts as the lowest score, picks of +inf share the weight,
  // and picks that all have the lowest score share it too
  const bool on = lane < a.k;
  const float my_val = on ? sval[my_id] : 0.0f;
  const float z = my_val != my_val ? -INFINITY : my_val;
  const float zmax = __uint_as_float(wave_reduce(__float_as_uint(on ? z : -INFINITY), [](uint32_t x, uint32_t y) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  }));
  float w;
  if (a.score == SC_SCORE_SIGMOID) {
    // all times exp(-max) where that is negative: sigmoids below fp32's range keep their proportion
    constexpr float kLog2e = 1.4426950408889634f;
    const float q = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-fabsf(z) * kLog2e));
    w = !on || z == -INFINITY ? 0.0f : z > 0.0f ? q : __builtin_amdgcn_exp2f((z - fminf(zmax, 0.0f)) * kLog2e) * q;
  } else {
    w = !on ? 0.0f : zmax == INFINITY ? (z == INFINITY ? 1.0f : 0.0f) : zmax == -INFINITY ? 1.0f : expf(z - zmax);
  }
  const float total = wave_sum_f(w);
  w = (total > 0.0f ? w / total : 1.0f / (float)a.k) * a.scale;
  if (on) {
    const int p = m * a.k + lane;
    put(&a.picks[p], (uint64_t)(uint32_t)(my_id + 1) << 32 | __float_as_uint(w));
    if (a.ids_out) put(&a.ids_out[p], my_id);
    if (a.w_out) put(&a.w_out[p], w);
  }
  return kDone;
}

// ---- expert products -------------------------------------------------------------

__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// Four fp32 values as three bf16 parts that add up to them.
__device__ __forceinline__ void split3(f32x4 v, uint8_t* dst, int part_bytes) {
  uint16_t p[3][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __bf16 p0 = (__bf16)v[e];
    const float f0 = (float)p0, d1 = v[e] - f0;
    const bool fin = fabsf(f0) < INFINITY;      // what is not finite stands in the first part alone
    const __bf16 p1 = (__bf16)(fin ? d1 : 0.0f);
    const __bf16 p2 = (__bf16)(fin ? d1 - (float)p1 : 0.0f);
    p[0][e] = __builtin_bit_cast(uint16_t, p0);
    p[1][e] = __builtin_bit_cast(uint16_t, p1);
    p[2][e] = __builtin_bit_cast(uint16_t, p2);
  }
#pragma unroll
  for (int t = 0; t < 3; ++t)
    *reinterpret_cast<u32x2*>(dst + t * part_bytes) =
        u32x2{p[t][0] | (uint32_t)p[t][1] << 16, p[t][2] | (uint32_t)p[t][3] << 16};
}

// Written through, like all that these kernels store: a line of y left in one XCD's L2 could reach memory
// after the NaN that the block which leaves last, on another XCD, writes for a call that was given up.
__device__ __forceinline__ void store_y(const MoeArgs& a, int m, int r, float v) {
  const int64_t o = m * a.ldy + r;
  if (a.out == SC_DTYPE_F32) put(static_cast<float*>(a.y) + o, v);
  else put(static_cast<uint16_t*>(a.y) + o, __builtin_bit_cast(uint16_t, (__bf16)v));
}

// A phase's tasks as one block takes them: task t is number t / 16 of part t % 16.
// `ahead` (thread 0) is the next number of the block's own part, asked for while
// the task before runs; when that part is used up, the others are looked through.
struct Taker {
  int32_t* c;
  int n, home, ahead;
  __device__ __forceinline__ int limit(int shard) const { return (n - shard + kShards - 1) / kShards; }
  __device__ __forceinline__ void ask() {
    if (threadIdx.x == 0) ahead = add(c + home * kLine, 1);
  }
  // the next task, or -1 when every task is taken; the block agrees on it through *tick
  __device__ __forceinline__ int next(int32_t* tick) {
    __syncthreads();
    if (threadIdx.x < 64) {
      int t = __builtin_amdgcn_readfirstlane(ahead);
      t = t < limit(home) ? t * kShards + home : -1;
      const int lane = threadIdx.x;
      while (t < 0) {
        const bool left = lane < kShards && get(c + lane * kLine) < limit(lane);
        const uint32_t m = (uint32_t)__ballot(left);
        if (!m) break;
        const uint32_t rot = (m >> home | m << (kShards - home)) & ((1u << kShards) - 1);
        const int s = (home + __builtin_ctz(rot)) % kShards;
        int k = 0;
        if (lane == 0) k = add(c + s * kLine, 1);
        k = __builtin_amdgcn_readfirstlane(k);
        if (k < limit(s)) {
          t = k * kShards + s;
          home = s;
        }
      }
      if (lane == 0) *tick = t;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*tick);
  }
};
// After a call that was given up, by the block that leaves last (the others' stores have been performed): y is
// NaN, and what is handed over is cleared.
__device__ __forceinline__ void abandon(const MoeArgs& a) {
  for (int i = threadIdx.x; i < a.M * a.H; i += blockDim.x) store_y(a, i / a.H, i % a.H, NAN);
  for (int i = threadIdx.x; i < a.logit_words; i += blockDim.x) put(&a.logits[i], kNoLogit);
}

// Control words of the one-row kernel (moe_one.hip).
constexpr int kOneWords = 1024 + (2 * kShards + 3) * kLine;
// *fits: the device can hold the kernel's shares; if not, nothing is launched.
hipError_t launch_moe_one(const MoeArgs& a, hipStream_t st, bool* fits);

}  // namespace moe
}  // namespace sc
