// A whole mixture-of-experts layer for up to 16 tokens in one launch: router
// product, top-k, gate/up, SiLU, down, weighted combine and the shared expert.
//
// Bound: HBM, by the bytes of the experts picked.  Between the products there
// is nothing to compute, only data to hand over, so the layer is one kernel of
// tasks that blocks take in order from a counter:
//   router tiles | shared gate/up tiles | routed gate/up tiles | down tiles
// A task waits only for tasks before it: a router tile for none, a routed
// gate/up tile for the picks (made by the block that ends the last router
// tile), a down tile for all h of its expert.  The first unfinished task is
// always held by a running block and waits for finished ones only, so every
// wait ends, whatever part of the grid is resident.  A down tile starts its
// weight loads before it waits.
//
// What one block hands to another goes through stores and loads at agent scope
// (each XCD has an L2 of its own): written through, waited for, then counted.
// A release fence would write back every dirty line of the L2 instead, other
// kernels' among them (measured: 12 of 21 us of the router product).
#include "fp4_device.h"
#include "internal.h"

namespace sc {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxTokens = SC_MOE_MAX_ROWS;
constexpr int kMaxPk = kMaxTokens * kMaxTopK;
constexpr int kPad = 16;           // bytes between operand rows in LDS: four rows' reads fall into different banks
constexpr int kUpRows = 32;        // rows of h per gate/up task
constexpr int kDownRows = 64;      // output rows per down task

// Control words, zero between calls: the block that leaves last clears them.
// C_ROUTED holds the number of unique experts + 1 once the picks are made; the
// hot ones lie in cache lines of their own.
enum Ctl { C_TICKET = 0, C_ARRIVED = 32, C_ROUTED = 64, C_EXITS = 96, C_ERROR = 97, C_HDONE = 128 };
constexpr int kHdone = kMaxPk + 1;                 // gate/up tiles done, per unique expert, then the shared one
constexpr int kTiles = 32768 / kDownRows;          // down tasks done, per tile
constexpr int kCtlWords = C_HDONE + kHdone + kTiles;
constexpr int C_TILES = C_HDONE + kHdone;

// Polls of a wait before the call is given up (about a second): only a
// workspace that was not prepared, or that two calls share, gets there.
constexpr int kMaxPolls = 1 << 20;

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
  int32_t* ctl;
  float* logits;             // [M][E]
  uint64_t* uniq;            // [U] expert, first pick and pick count
  uint32_t* uniq_picks;      // [P]
  float* pick_w;             // [P]
  float* h;                  // [P][I], then [M][Is] of the shared expert
  float* part;               // [P][H], then [M][H]
  int64_t ldx, ldy, blob;
  int M, H, I, E, k, Is, score, out, vec;
  int lds;                   // bytes of LDS for operand rows
  int dense;                 // x lies in LDS whole, token by token
  int router_tiles;
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
constexpr int kAgent = 16;   // buffer load at agent scope (sc1)
// The wavefront's stores have been performed.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ---- routing -------------------------------------------------------------------

// Logits of EB experts for up to MR rows: each wavefront sums a share of H, the
// shares are added in wavefront order.
template <int EB, int MR>
__device__ __forceinline__ void router_tile(const MoeArgs& a, int tile, float* red) {
  constexpr int V = EB * MR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = tile * EB;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  for (int c = (wave * 64 + lane) * 8; c < a.H; c += kThreads * 8) {
    u32x4 w[EB];
#pragma unroll
    for (int e = 0; e < EB; ++e)
      w[e] = *reinterpret_cast<const u32x4*>(a.router + (int64_t)min(e0 + e, a.E - 1) * a.H + c);
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      if (m >= a.M) break;
      const uint16_t* p = a.x + m * a.ldx + c;
      u32x4 x;
      if (a.vec) {
        x = *reinterpret_cast<const u32x4*>(p);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
      }
#pragma unroll
      for (int e = 0; e < EB; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[m * EB + e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (uint32_t)w[e][i]),
                                                            __builtin_bit_cast(bf16x2, (uint32_t)x[i]), acc[m * EB + e], false);
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
  for (int i = threadIdx.x; i < V; i += kThreads) {
    const int m = i / EB, e = e0 + i % EB;
    if (m < a.M && e < a.E) put(&a.logits[m * a.E + e], ((red[i] + red[V + i]) + red[2 * V + i]) + red[3 * V + i]);
  }
}

// Keys that order as the scores do: NaN below -inf, -0 equal to +0.
__device__ __forceinline__ int order_key(float z) {
  if (z != z) return INT32_MIN + 1;
  const int b = (int)__float_as_uint(z + 0.0f);
  return b >= 0 ? b : b ^ 0x7FFFFFFF;
}

__device__ __forceinline__ int wave_max_i(int v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = max(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

struct RouteLds {
  uint32_t rows[kMaxExperts];     // rows that picked the expert, then its place among the unique experts
  int32_t off[kMaxExperts];       // first pick of the expert
  int16_t id[kMaxPk];
  int32_t nu;
};

// One wavefront picks a row's experts: lane l looks after experts l * epl ..,
// so the lowest lane with the largest key holds the lowest id.
template <int EPL>
__device__ __forceinline__ void route_row(const MoeArgs& a, int m, RouteLds& s) {
  const int lane = threadIdx.x & 63;
  const int epl = (a.E + 63) / 64;
  int key[EPL];
  float val[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * epl + i;
    key[i] = INT32_MIN;
    val[i] = 0.0f;
    if (i < epl && e < a.E) {
      float z = get(&a.logits[m * a.E + e]);
      if (a.score == SC_SCORE_SIGMOID) {
        z = 1.0f / (1.0f + expf(-z));
        val[i] = z;
        if (a.score_bias) z += a.score_bias[e];
      } else {
        val[i] = z;
      }
      key[i] = order_key(z);
    }
  }
  int my_id = 0;
  float my_val = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    int best = key[0], at = 0;
    float bv = val[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) {
      if (key[i] > best) {
        best = key[i];
        at = i;
        bv = val[i];
      }
    }
    const int top = wave_max_i(best);
    const int src = __builtin_ctzll(__ballot(best == top));
    const int id = __builtin_amdgcn_readlane(lane * epl + at, src);
    const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(bv), src));
    if (lane == j) {
      my_id = id;
      my_val = v;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane == src && i == at) key[i] = INT32_MIN;
  }
  // weights; NaN counts as the lowest score, picks of +inf share the weight,
  // and picks that all have the lowest score share it too
  const bool on = lane < a.k;
  float z = my_val != my_val ? -INFINITY : my_val, w;
  if (a.score == SC_SCORE_SIGMOID) {
    w = on && z > 0.0f ? z : 0.0f;
  } else {
    float zmax = on ? z : -INFINITY;
#pragma unroll
    for (int o = 32; o; o >>= 1) zmax = fmaxf(zmax, __shfl_xor(zmax, o));
    w = !on ? 0.0f : zmax == INFINITY ? (z == INFINITY ? 1.0f : 0.0f) : zmax == -INFINITY ? 1.0f : expf(z - zmax);
  }
  const float sum = wave_sum_f(w);
  w = sum > 0.0f ? w / sum : 1.0f / (float)a.k;
  w *= a.scale;
  if (on) {
    const int p = m * a.k + lane;
    s.id[p] = (int16_t)my_id;
    put(&a.pick_w[p], w);
    if (a.ids_out) a.ids_out[p] = my_id;
    if (a.w_out) a.w_out[p] = w;
    atomicOr(&s.rows[my_id], 1u << m);
  }
}

// Picks of all rows, and the picks grouped by expert (experts ascending, an
// expert's rows ascending).
__device__ __forceinline__ void route_all(const MoeArgs& a, RouteLds& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < a.E; e += kThreads) s.rows[e] = 0;
  __syncthreads();
  for (int m = wave; m < a.M; m += kWaves) {
    if (a.E <= 256) route_row<4>(a, m, s);
    else if (a.E <= 512) route_row<8>(a, m, s);
    else route_row<16>(a, m, s);
  }
  __syncthreads();
  if (wave == 0) {
    int nu = 0, np = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < a.E ? __popc(s.rows[e]) : 0;
      const uint64_t mask = __ballot(n > 0);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(incl, o);
        if (lane >= o) incl += t;
      }
      if (n > 0) {
        const int u = nu + __popcll(mask & ((1ull << lane) - 1));
        put(&a.uniq[u], (uint64_t)(uint32_t)e << 32 | (uint32_t)(np + incl - n) << 8 | (uint32_t)n);
        s.off[e] = np + incl - n;
      }
      nu += __popcll(mask);
      np += __shfl(incl, 63);
    }
    if (lane == 0) s.nu = nu;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.M * a.k; p += kThreads) {
    const int e = s.id[p], m = p / a.k;
    put(&a.uniq_picks[s.off[e] + __popc(s.rows[e] & ((1u << m) - 1))], (uint32_t)p);
  }
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0) put(&a.ctl[C_ROUTED], s.nu + 1);
}

// Counts the block in, once all that its threads put has been performed; true
// in the block that completes `total`.
__device__ __forceinline__ bool arrive(int32_t* counter, int total, int32_t* flag) {
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0)
    *flag = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  __syncthreads();
  return *flag != 0;
}
// Same without asking who was last.
__device__ __forceinline__ void post(int32_t* counter) {
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0) __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits until *p >= value (one thread); false when the call was given up.
__device__ __forceinline__ bool wait_for(const MoeArgs& a, const int32_t* p, int value) {
  for (int i = 0; get(p) < value; ++i) {
    if (get(&a.ctl[C_ERROR])) return false;
    if (i >= kMaxPolls) {
      put(&a.ctl[C_ERROR], 1);
      return false;
    }
    __builtin_amdgcn_s_sleep(1);
  }
  return true;
}

// ---- expert products ----------------------------------------------------------

// One expert's rows: routed (its picks) or the shared expert (every row).
struct Work {
  const uint8_t* blob;
  float gs13, gs2;
  int inter, n;            // n rows
  int first;               // offset in the list of picks, or -1 for the shared expert
  int u;                   // unique index; U for the shared expert
};

// The picks as a block keeps them.
struct BlockLds {
  uint64_t uniq[kMaxPk];
  uint16_t pick[kMaxPk];
  int32_t tick, flag, U;
};

__device__ __forceinline__ Work work_of(const MoeArgs& a, const BlockLds& b, int u, bool shared) {
  Work w;
  w.u = u;
  if (!shared) {
    const uint64_t d = b.uniq[u];
    const int e = __builtin_amdgcn_readfirstlane((int)(d >> 32));
    const int lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)d);
    w.first = lo >> 8;
    w.n = lo & 255;
    w.blob = a.blobs + e * a.blob;
    w.gs13 = a.gs[2 * e];
    w.gs2 = a.gs[2 * e + 1];
    w.inter = a.I;
  } else {
    w.first = -1;
    w.n = a.M;
    w.blob = a.shared;
    w.gs13 = a.sgs[0];
    w.gs2 = a.sgs[1];
    w.inter = a.Is;
  }
  return w;
}
// The expert's c-th pick (P + row for the shared expert) and its token.
__device__ __forceinline__ int pick_at(const MoeArgs& a, const BlockLds& b, const Work& w, int c) {
  return w.first < 0 ? a.M * a.k + c : b.pick[w.first + c];
}
__device__ __forceinline__ int token_at(const MoeArgs& a, const BlockLds& b, const Work& w, int c) {
  return w.first < 0 ? c : (int)((uint32_t)b.pick[w.first + c] / (uint32_t)a.k);
}
// First element of a pick's row of h: picks [P][I], then the shared expert's [M][Is]
__device__ __forceinline__ uint32_t h_at(const MoeArgs& a, int p) {
  const uint32_t P = a.M * a.k;
  return (uint32_t)p < P ? (uint32_t)p * a.I : P * a.I + ((uint32_t)p - P) * a.Is;
}

__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// K-elements of ROWS operand rows of `parts` bf16 parts that fit in LDS.
__device__ __forceinline__ int lds_range(int lds, int rows, int parts, int K) {
  const int fit = (lds / (rows * parts) - kPad) / 2 / kStepK * kStepK;
  const int need = (K + kStepK - 1) / kStepK * kStepK;
  return fit < need ? fit : need;
}

// `n` rows of x from column kc to kend (rounded up to whole steps, zeros behind
// the end) into LDS; row c is token tok(c).
template <typename F>
__device__ __forceinline__ void stage_x(const MoeArgs& a, uint8_t* lds, int row_lds, int n, int kc, int kend, F tok) {
  const int per_row = (kend - kc + kStepK - 1) / kStepK * (kStepK / 8);
  for (int i = threadIdx.x; i < n * per_row; i += kThreads) {
    const int c = i / per_row, o = (i - c * per_row) * 8;
    u32x4 v = {0, 0, 0, 0};
    if (kc + o < kend) {
      const uint16_t* p = a.x + tok(c) * a.ldx + kc + o;
      if (a.vec) {
        v = *reinterpret_cast<const u32x4*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p[2 * e] | (uint32_t)p[2 * e + 1] << 16;
      }
    }
    *reinterpret_cast<u32x4*>(lds + c * row_lds + o * 2) = v;
  }
}

// h rows [tile * 32, +32) of an expert: a wavefront takes HQ quads of gate rows
// at a time and the quads of up rows that belong to them.  x_there: all of x
// lies in LDS (dense) and needs no staging.
template <int ROWS>
__device__ __forceinline__ void gateup_task(const MoeArgs& a, const BlockLds& b, const Work& w, int tile, uint8_t* lds,
                                            bool x_there) {
  constexpr int HQ = ROWS <= 4 ? 2 : 1, D = 2, NA = (ROWS + 3) / 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = a.H;
  const uint32_t cb = H / 2, sb = H / 16, up = (uint32_t)w.inter;
  const Rsrc rc = make_rsrc(w.blob, 2u * up * cb), rs = make_rsrc(w.blob + (int64_t)2 * up * cb, 2u * up * sb);
  const int klane = (lane >> 2) * 32, r0 = lane & 3;
  const int KC = a.dense ? (H + kStepK - 1) / kStepK * kStepK : lds_range(a.lds, ROWS, 1, H);
  const int row_lds = KC * 2 + kPad;
  const uint8_t* xs[NA];
#pragma unroll
  for (int s = 0; s < NA; ++s) {
    const int c = 4 * s + r0 < w.n ? 4 * s + r0 : 0;
    xs[s] = lds + (a.dense ? token_at(a, b, w, c) : c) * row_lds + klane * 2;
  }
  for (int part = 0; part < kUpRows / 4 / kWaves; part += HQ) {
    const int row0 = tile * kUpRows + (wave * (kUpRows / 4 / kWaves) + part) * 4;
    const uint32_t r = row0 + r0;
    float acc[2 * HQ][ROWS];
#pragma unroll
    for (int j = 0; j < 2 * HQ; ++j)
#pragma unroll
      for (int c = 0; c < ROWS; ++c) acc[j][c] = 0.0f;
    for (int kc = 0; kc < H; kc += KC) {
      const int kend = min(H, kc + KC), steps = (kend - kc + kStepK - 1) / kStepK;
      Stage<kNv, false, HQ> g[D], u[D];
      auto load = [&](int d, int s) {
        const int k = kc + s * kStepK + klane;
        load_stage<kNv, false, HQ>(g[d], rc, rs, r * cb, r * sb, 4 * cb, 4 * sb, k, kend);
        load_stage<kNv, false, HQ>(u[d], rc, rs, (r + up) * cb, (r + up) * sb, 4 * cb, 4 * sb, k, kend);
      };
#pragma unroll
      for (int d = 0; d < D; ++d) load(d, d);
      if (!x_there) {
        __syncthreads();
        if (a.dense) stage_x(a, lds, row_lds, a.M, 0, H, [&](int c) { return c; });
        else stage_x(a, lds, row_lds, w.n, kc, kend, [&](int c) { return token_at(a, b, w, c); });
        __syncthreads();
      }
      for (int s = 0; s < steps; s += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s + d < steps) {
            Stage<kNv, false, 2 * HQ> st;
#pragma unroll
            for (int j = 0; j < HQ; ++j) {
              st.q[j] = g[d].q[j];
              st.s[j] = g[d].s[j];
              st.q[HQ + j] = u[d].q[j];
              st.s[HQ + j] = u[d].s[j];
            }
            use_stage<kNv, false, 2 * HQ, ROWS, false>(st, xs, (s + d) * kStepK * 2, acc);
            load(d, s + d + D);
          }
        }
      }
    }
    x_there = x_there || a.dense;
    constexpr int V = HQ * ROWS;
    float vg[V], vu[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      vg[i] = acc[i / ROWS][i % ROWS];
      vu[i] = acc[HQ + i / ROWS][i % ROWS];
    }
    tile_sum<V>(vg);
    tile_sum<V>(vu);
    if (tile_sum_owner<V>(lane)) {
      const int first = tile_sum_first<V>(lane);
#pragma unroll
      for (int i = 0; i < kTileOut<V>; ++i) {
        const int q = (first + i) / ROWS, c = (first + i) % ROWS;
        if (c < w.n)
          put(&a.h[h_at(a, pick_at(a, b, w, c)) + row0 + 4 * q + r0], silu(vg[i] * w.gs13) * (vu[i] * w.gs13));
      }
    }
  }
}

// Output rows [tile * 64, +64) of an expert's down product, per pick.  h is
// used to its 24 bits, in three bf16 parts: rounded to one part it would put
// 2^-9 of itself into y, more than all fp32 sums together.  False when the call
// was given up.
template <int ROWS>
__device__ __forceinline__ bool down_task(const MoeArgs& a, BlockLds& b, const Work& w, int tile, uint8_t* lds) {
  constexpr int Q = ROWS <= 4 ? 4 : 2, D = 2, NA = (ROWS + 3) / 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int I = w.inter;
  const uint32_t cb = I / 2, sb = I / 16;
  const int64_t w13 = (int64_t)2 * I * (a.H / 2) + (int64_t)2 * I * (a.H / 16), codes = (int64_t)a.H * cb;
  const Rsrc rc = make_rsrc(w.blob + w13, (uint32_t)codes), rs = make_rsrc(w.blob + w13 + codes, (uint32_t)a.H * sb);
  const Rsrc rh = make_rsrc(a.h, (uint32_t)(a.M * (a.k * a.I + a.Is)) * 4);
  const int klane = (lane >> 2) * 32, r0 = lane & 3;
  const int KC = lds_range(a.lds, ROWS, 3, I);
  const int part_lds = KC * 2 + kPad, row_lds = 3 * part_lds;
  const uint8_t* xs[NA];
#pragma unroll
  for (int s = 0; s < NA; ++s) {
    // one row: its parts are the rows of the set
    const int c = 4 * s + r0 < w.n ? 4 * s + r0 : 0;
    xs[s] = lds + (ROWS == 1 ? (r0 < 3 ? r0 : 0) * part_lds : c * row_lds) + klane * 2;
  }
  bool waited = false;
  for (int part = 0; part < kDownRows / 4 / kWaves; part += Q) {
    const int row0 = tile * kDownRows + (wave * (kDownRows / 4 / kWaves) + part) * 4;
    const uint32_t r = row0 + r0;
    float acc[Q][ROWS];
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int c = 0; c < ROWS; ++c) acc[j][c] = 0.0f;
    for (int kc = 0; kc < I; kc += KC) {
      const int kend = min(I, kc + KC), steps = (kend - kc + kStepK - 1) / kStepK;
      Stage<kNv, false, Q> st[D];
#pragma unroll
      for (int d = 0; d < D; ++d)
        load_stage<kNv, false, Q>(st[d], rc, rs, r * cb, r * sb, 4 * cb, 4 * sb, kc + d * kStepK + klane, kend);
      if (!waited) {
        if (threadIdx.x == 0) b.flag = wait_for(a, &a.ctl[C_HDONE + w.u], I / kUpRows);
        waited = true;
      }
      if (part == 0 || KC < I) {
        __syncthreads();
        if (!b.flag) return false;
        const int per_row = steps * (kStepK / 4);
        for (int i = threadIdx.x; i < w.n * per_row; i += kThreads) {
          const int c = i / per_row, o = (i - c * per_row) * 4;
          const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(
              rh, kc + o < kend ? (int)((h_at(a, pick_at(a, b, w, c)) + kc + o) * 4) : (int)kBeyond, 0, kAgent);
          const f32x4 v = __builtin_bit_cast(f32x4, t);
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
          for (int t3 = 0; t3 < 3; ++t3)
            *reinterpret_cast<u32x2*>(lds + c * row_lds + t3 * part_lds + o * 2) =
                u32x2{p[t3][0] | (uint32_t)p[t3][1] << 16, p[t3][2] | (uint32_t)p[t3][3] << 16};
        }
        __syncthreads();
      }
      for (int s = 0; s < steps; s += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s + d < steps) {
            use_stage<kNv, false, Q, ROWS, false, true>(st[d], xs, (s + d) * kStepK * 2, acc, part_lds);
            load_stage<kNv, false, Q>(st[d], rc, rs, r * cb, r * sb, 4 * cb, 4 * sb, kc + (s + d + D) * kStepK + klane,
                                      kend);
          }
        }
      }
    }
    constexpr int V = Q * ROWS;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = acc[i / ROWS][i % ROWS];
    tile_sum<V>(v);
    if (tile_sum_owner<V>(lane)) {
      const int first = tile_sum_first<V>(lane);
#pragma unroll
      for (int i = 0; i < kTileOut<V>; ++i) {
        const int q = (first + i) / ROWS, c = (first + i) % ROWS;
        if (c < w.n) put(&a.part[(int64_t)pick_at(a, b, w, c) * a.H + row0 + 4 * q + r0], v[i] * w.gs2);
      }
    }
  }
  return true;
}

__device__ __forceinline__ void store_y(const MoeArgs& a, int m, int r, float v) {
  const int64_t o = m * a.ldy + r;
  if (a.out == SC_DTYPE_F32) static_cast<float*>(a.y)[o] = v;
  else static_cast<uint16_t*>(a.y)[o] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// y of 64 rows: the picks in rank order, then the shared expert.
__device__ __forceinline__ void combine_tile(const MoeArgs& a, int tile) {
  const int P = a.M * a.k;
  for (int i = threadIdx.x; i < a.M * kDownRows; i += kThreads) {
    const int m = i / kDownRows, r = tile * kDownRows + i % kDownRows;
    float s = 0.0f;
    for (int j = 0; j < a.k; ++j)
      s = fmaf(get(&a.pick_w[m * a.k + j]), get(&a.part[(int64_t)(m * a.k + j) * a.H + r]), s);
    if (a.shared) s += get(&a.part[(int64_t)(P + m) * a.H + r]);
    store_y(a, m, r, s);
  }
}

template <int MAXR>
__device__ __forceinline__ void run_gateup(const MoeArgs& a, const BlockLds& b, const Work& w, int tile, uint8_t* lds,
                                           bool x_there) {
  if (MAXR == 1 || w.n == 1) return gateup_task<1>(a, b, w, tile, lds, x_there);
  if (w.n == 2) return gateup_task<2>(a, b, w, tile, lds, x_there);
  if (MAXR == 4 || w.n <= 4) return gateup_task<4>(a, b, w, tile, lds, x_there);
  if constexpr (MAXR > 4) return gateup_task<16>(a, b, w, tile, lds, x_there);
}
template <int MAXR>
__device__ __forceinline__ bool run_down(const MoeArgs& a, BlockLds& b, const Work& w, int tile, uint8_t* lds) {
  if (MAXR == 1 || w.n == 1) return down_task<1>(a, b, w, tile, lds);
  if (w.n == 2) return down_task<2>(a, b, w, tile, lds);
  if (MAXR == 4 || w.n <= 4) return down_task<4>(a, b, w, tile, lds);
  if constexpr (MAXR > 4) return down_task<16>(a, b, w, tile, lds);
  return true;
}

template <int MAXR>
__global__ __launch_bounds__(kThreads, MAXR <= 4 ? 3 : 2) void k_moe_layer(MoeArgs a) {
  constexpr int EB = MAXR == 1 ? 1 : MAXR == 4 ? 2 : 4;   // experts per router tile
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ BlockLds b;
  const int R = a.router_tiles, S = a.shared ? a.Is / kUpRows : 0, tu = a.I / kUpRows, td = a.H / kDownRows;
  const int ns = a.shared ? 1 : 0;
  int U = -1, total = INT32_MAX;
  bool x_there = false;
  if (threadIdx.x == 0) b.tick = __hip_atomic_fetch_add(&a.ctl[C_TICKET], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (;;) {
    __syncthreads();
    const int t = __builtin_amdgcn_readfirstlane(b.tick);
    if (t >= total) break;
    // the next ticket is on its way while the task runs
    int next = 0;
    if (threadIdx.x == 0) next = __hip_atomic_fetch_add(&a.ctl[C_TICKET], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (t < R) {
      router_tile<EB, MAXR>(a, t, reinterpret_cast<float*>(lds));
      if (arrive(&a.ctl[C_ARRIVED], R, &b.flag)) route_all(a, *reinterpret_cast<RouteLds*>(lds));
    } else if (t < R + S) {
      run_gateup<MAXR>(a, b, work_of(a, b, kMaxPk, true), t - R, lds, x_there);
      x_there = a.dense;
      post(&a.ctl[C_HDONE + kMaxPk]);
    } else {
      if (U < 0) {
        if (threadIdx.x == 0) b.U = wait_for(a, &a.ctl[C_ROUTED], 1) ? get(&a.ctl[C_ROUTED]) - 1 : -1;
        __syncthreads();
        U = __builtin_amdgcn_readfirstlane(b.U);
        if (U < 0 || U > a.M * a.k) break;
        total = R + S + U * tu + (U + ns) * td;
        for (int i = threadIdx.x; i < U; i += kThreads) b.uniq[i] = get(&a.uniq[i]);
        for (int i = threadIdx.x; i < a.M * a.k; i += kThreads) b.pick[i] = (uint16_t)get(&a.uniq_picks[i]);
        __syncthreads();
        if (t >= total) break;
      }
      const int g = t - R - S;
      if (g < U * tu) {
        const int u = g / tu;
        run_gateup<MAXR>(a, b, work_of(a, b, u, false), g - u * tu, lds, x_there);
        x_there = a.dense;
        post(&a.ctl[C_HDONE + u]);
      } else {
        // the shared expert's h is there first
        const int d = g - U * tu, u = d / td, tile = d - u * td;
        const bool sh = ns && u == 0;
        if (!run_down<MAXR>(a, b, work_of(a, b, sh ? kMaxPk : u - ns, sh), tile, lds)) break;
        if (arrive(&a.ctl[C_TILES + tile], U + ns, &b.flag)) combine_tile(a, tile);
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) b.tick = next;
  }
  // the last block out clears the control words; a call that was given up has no result
  __syncthreads();
  if (threadIdx.x == 0)
    b.flag = __hip_atomic_fetch_add(&a.ctl[C_EXITS], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
             (int)gridDim.x - 1;
  __syncthreads();
  if (!b.flag) return;
  if (get(&a.ctl[C_ERROR]))
    for (int i = threadIdx.x; i < a.M * a.H; i += kThreads) store_y(a, i / a.H, i % a.H, NAN);
  __syncthreads();
  for (int i = threadIdx.x; i < kCtlWords; i += kThreads) put(&a.ctl[i], 0);
}

__global__ void k_moe_clear(int32_t* ctl, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) ctl[i] = 0;
}

// ---- host ------------------------------------------------------------------------

constexpr size_t kAlign = 256;
size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct MoeWs {
  size_t ctl, logits, uniq, uniq_picks, pick_w, h, part, end;
};
MoeWs moe_ws(const sc_moe_config* c) {
  MoeWs o;
  const size_t M = c->max_rows, P = M * c->top_k;
  size_t p = 0;
  o.ctl = p; p = up(p + kCtlWords * 4);
  o.logits = p; p = up(p + M * c->n_experts * 4);
  o.uniq = p; p = up(p + P * 8);
  o.uniq_picks = p; p = up(p + P * 4);
  o.pick_w = p; p = up(p + P * 4);
  o.h = p; p = up(p + (P * c->inter + M * c->shared_inter) * 4);
  o.part = p; p = up(p + (P + M) * c->hidden * 4);
  o.end = p;
  return o;
}

sc_status check_moe(const sc_moe_config* c) {
  if (!c) return fail(SC_E_ARG, "config is NULL");
  if (c->hidden < 64 || c->hidden % 64 || c->hidden > 32768 || c->inter < 64 || c->inter % 64 || c->inter > 32768)
    return fail(SC_E_ARG, "hidden and inter must be multiples of 64 in [64, 32768]");
  if (c->shared_inter < 0 || c->shared_inter % 64 || c->shared_inter > 32768)
    return fail(SC_E_ARG, "shared_inter must be 0 or a multiple of 64 up to 32768");
  if (c->top_k < 1 || c->top_k > kMaxTopK) return fail(SC_E_ARG, "top_k must be in [1, %d]", kMaxTopK);
  if (c->n_experts < c->top_k || c->n_experts > kMaxExperts)
    return fail(SC_E_ARG, "n_experts must be in [top_k, %d]", kMaxExperts);
  if (c->max_rows < 1 || c->max_rows > kMaxTokens) return fail(SC_E_ARG, "max_rows must be in [1, %d]", kMaxTokens);
  if (c->score != SC_SCORE_SOFTMAX && c->score != SC_SCORE_SIGMOID) return fail(SC_E_ARG, "unknown score %d", c->score);
  return SC_OK;
}

template <int MAXR>
hipError_t launch_moe(MoeArgs a, hipStream_t st) {
  constexpr int EB = MAXR == 1 ? 1 : MAXR == 4 ? 2 : 4;
  const int steps_h = (a.H + kStepK - 1) / kStepK, inter = a.I > a.Is ? a.I : a.Is;
  const int steps_i = (inter + kStepK - 1) / kStepK;
  a.router_tiles = (a.E + EB - 1) / EB;
  // LDS: the rows of x whole if they fit, and h of one expert's rows; 64 KB let two blocks share a compute unit
  const int dense = a.M * (steps_h * kStepK * 2 + kPad), hrows = (a.M <= 2 ? a.M : MAXR) * 3 * (steps_i * kStepK * 2 + kPad);
  const int cap = 65536, least = (int)sizeof(RouteLds);
  a.dense = dense <= cap;
  a.lds = (a.dense ? dense : cap) > hrows ? (a.dense ? dense : cap) : hrows;
  if (a.lds > cap) a.lds = cap;
  if (a.lds < least) a.lds = (least + 15) / 16 * 16;
  const long picks = (long)a.M * a.k < a.E ? (long)a.M * a.k : a.E;
  const long tasks = a.router_tiles + (a.shared ? a.Is / kUpRows : 0) + picks * (a.I / kUpRows) +
                     (picks + (a.shared ? 1 : 0)) * (a.H / kDownRows);
  const unsigned blocks = tasks < 1024 ? (unsigned)tasks : 1024u;
  hipLaunchKernelGGL((k_moe_layer<MAXR>), dim3(blocks), dim3(kThreads), a.lds, st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace sc

using namespace sc;

extern "C" {

sc_status moe_layer_workspace_bytes(const sc_moe_config* cfg, size_t* bytes) {
  const sc_status s = check_moe(cfg);
  if (s != SC_OK) return s;
  if (!bytes) return fail(SC_E_ARG, "bytes is NULL");
  *bytes = moe_ws(cfg).end;
  return SC_OK;
}

sc_status moe_layer_prepare(const sc_moe_config* cfg, void* d_workspace, void* stream) {
  const sc_status s = check_moe(cfg);
  if (s != SC_OK) return s;
  if (!d_workspace || (uintptr_t)d_workspace % kAlign) return fail(SC_E_ARG, "the workspace must be 256-byte aligned");
  hipLaunchKernelGGL(k_moe_clear, dim3(1), dim3(256), 0, static_cast<hipStream_t>(stream),
                     reinterpret_cast<int32_t*>(static_cast<uint8_t*>(d_workspace) + moe_ws(cfg).ctl), kCtlWords);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? SC_OK : hip_fail(e, "moe_layer_prepare launch");
}

sc_status moe_layer_forward(const sc_moe_config* c, const sc_moe_weights* w, void* d_workspace, const uint16_t* d_x,
                            int64_t ldx, int32_t M, void* d_y, int32_t y_type, int64_t ldy, int32_t* d_ids,
                            float* d_weights, void* stream) {
  const sc_status s = check_moe(c);
  if (s != SC_OK) return s;
  if (!w || !w->d_router || !w->d_blobs || !w->d_global_scales) return fail(SC_E_ARG, "a weight is NULL");
  if (c->shared_inter && (!w->d_shared_blob || !w->d_shared_scales))
    return fail(SC_E_ARG, "the shared expert's blob or scales are NULL");
  if ((uintptr_t)w->d_router % 16 || (uintptr_t)w->d_blobs % 16 || (uintptr_t)w->d_shared_blob % 16 ||
      (uintptr_t)w->d_global_scales % 4 || (uintptr_t)w->d_shared_scales % 4 || (uintptr_t)w->d_score_bias % 4)
    return fail(SC_E_ARG, "router and blobs must be 16-byte aligned, scales and biases 4-byte");
  if (!d_workspace || (uintptr_t)d_workspace % kAlign) return fail(SC_E_ARG, "the workspace must be 256-byte aligned");
  if (M < 0 || M > c->max_rows) return fail(SC_E_ARG, "M must be in [0, max_rows = %d]", c->max_rows);
  if (y_type != SC_DTYPE_F32 && y_type != SC_DTYPE_BF16) return fail(SC_E_ARG, "y_type must be fp32 or bf16");
  if (M == 0) return SC_OK;
  if (!d_x || !d_y) return fail(SC_E_ARG, "x or y is NULL");
  if ((uintptr_t)d_x % 2 || (uintptr_t)d_y % (y_type == SC_DTYPE_F32 ? 4 : 2) || (uintptr_t)d_ids % 4 ||
      (uintptr_t)d_weights % 4)
    return fail(SC_E_ARG, "x, y, ids or weights are not aligned to their elements");
  if (ldx < c->hidden || ldy < c->hidden) return fail(SC_E_ARG, "row strides must cover the rows");
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  const MoeWs o = moe_ws(c);
  MoeArgs a{};
  a.router = static_cast<const uint16_t*>(w->d_router);
  a.score_bias = c->score == SC_SCORE_SIGMOID ? w->d_score_bias : nullptr;
  a.blobs = static_cast<const uint8_t*>(w->d_blobs);
  a.gs = w->d_global_scales;
  a.shared = c->shared_inter ? static_cast<const uint8_t*>(w->d_shared_blob) : nullptr;
  a.sgs = w->d_shared_scales;
  a.x = d_x;
  a.y = d_y;
  a.ids_out = d_ids;
  a.w_out = d_weights;
  a.ctl = reinterpret_cast<int32_t*>(ws + o.ctl);
  a.logits = reinterpret_cast<float*>(ws + o.logits);
  a.uniq = reinterpret_cast<uint64_t*>(ws + o.uniq);
  a.uniq_picks = reinterpret_cast<uint32_t*>(ws + o.uniq_picks);
  a.pick_w = reinterpret_cast<float*>(ws + o.pick_w);
  a.h = reinterpret_cast<float*>(ws + o.h);
  a.part = reinterpret_cast<float*>(ws + o.part);
  a.ldx = ldx;
  a.ldy = ldy;
  a.blob = make_shape(c->hidden, c->inter, c->n_experts, c->top_k).blob;
  a.M = M;
  a.H = c->hidden;
  a.I = c->inter;
  a.E = c->n_experts;
  a.k = c->top_k;
  a.Is = c->shared_inter;
  a.score = c->score;
  a.out = y_type;
  a.vec = (uintptr_t)d_x % 16 == 0 && ldx % 8 == 0;
  a.scale = c->routed_scale;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = M == 1 ? launch_moe<1>(a, st) : M <= 4 ? launch_moe<4>(a, st) : launch_moe<16>(a, st);
  return e == hipSuccess ? SC_OK : hip_fail(e, "moe_layer_forward launch");
}

}  // extern "C"
