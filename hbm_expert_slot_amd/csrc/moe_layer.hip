// A whole mixture-of-experts layer for 2 to 16 tokens in one launch: router
// product, top-k, gate/up, SiLU, down, weighted combine and the shared expert.
// (One token: moe_one.hip.)
//
// Bound: HBM, by the bytes of the experts picked.  Between the products there
// is nothing to compute, only data to hand over, so the layer is one kernel
// whose blocks go through five phases of tasks:
//   router tiles | picks of a row | shared gate/up tiles | routed gate/up tiles | down tiles
// Blocks take a phase's tasks from counters and go on to the next phase when
// none is left to take.  A task waits for tasks of earlier phases only: a
// row's picks for its logits, a routed gate/up tile for all picks (which every
// block groups by expert for itself), a down tile for all h of its expert.  When a block waits, every
// task of the earlier phases is held by a block that runs, so every wait ends,
// whatever part of the grid is resident.  A down tile starts its weight loads
// before it waits.
//
// The counters are in 16 parts: additions to one address take 11 ns each from
// wherever they come (with a single counter a token's 3500 tickets took longer
// than its weights).
#include "moe_device.h"

namespace sc {
namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
static_assert(kWaves == kTileWaves, "a block does a router tile");
constexpr int kMaxPk = kMaxTokens * kMaxTopK;
constexpr int kUpRows = 16;        // rows of h per gate/up tile: a quad per wavefront
constexpr int kTaskRounds = 2, kTaskTail = 8;   // see Tasks
constexpr int kDownRows = 32;      // output rows per down tile: two quads per wavefront

// Control words, zero between calls: the block that leaves last clears them.
// Counters that many blocks add to, and flags that many blocks poll, lie in
// cache lines of their own, apart from each other: an addition to a line that
// eight L2 caches hold for their pollers is slow, and so is all that waits in
// its channel (a token's layer took 138 us with counters polled in place, 81
// with flags set once).
enum Phase { kRouter = 0, kPick, kShared, kRouted, kDown, kPhases };
constexpr int kExperts = kMaxPk + 1;               // unique experts, then the shared one
constexpr int kTiles = 32768 / kDownRows;
constexpr int C_TICKETS = 0,                                    // [phase][shard]: tasks taken
    C_EXITS = kPhases * kShards * kLine,                        // blocks that left
    C_ERROR = C_EXITS + kLine,                                  // flag: the call was given up
    C_HDONE = C_ERROR + kLine,                                  // [expert]: gate/up tiles done
    C_TILES = C_HDONE + (kExperts + kLine) / kLine * kLine,     // [tile]: experts' down tiles done
    C_HREADY = C_TILES + kTiles,                                // [expert]: flag: all of h is there
    kLayerWords = C_HREADY + kExperts * kLine;                  // whole lines: the one-row kernel's words follow
static_assert(kLayerWords % kLine == 0, "");

// Counts `n` gate/up tiles of an expert in, once all that the block's threads put
// has been performed; who completes them sets the expert's flag.
__device__ __forceinline__ void post_h(const MoeArgs& a, int u, int n, int total) {
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0 && add(&a.ctl[C_HDONE + u], n) == total - n) put(&a.ctl[C_HREADY + u * kLine], 1);
}
// Waits until a flag is set (one thread); false when the call was given up.
__device__ __forceinline__ bool wait_for(const MoeArgs& a, int flag) {
  for (int i = 0; !get(&a.ctl[flag]); ++i)
    if (!poll_on(&a.ctl[C_ERROR], i)) return false;
  return true;
}

// ---- expert products ----------------------------------------------------------

// One expert's rows: routed (its picks) or the shared expert (every row).
struct Work {
  const uint8_t* blob;
  float gs13, gs2;
  int inter;
  int row, n;              // rows row .. row + n - 1 of the expert's
  int first;               // offset in the list of picks, or -1 for the shared expert
  int u;                   // unique index; U for the shared expert
};

// The picks as a block keeps them, grouped by expert (experts ascending, an
// expert's rows ascending).
template <int MAXR>
struct BlockLds {
  static constexpr int kPk = MAXR * kMaxTopK;
  uint32_t uniq[kPk];              // see pack_uniq
  uint16_t pick[kPk];
  uint32_t rows[MAXR == 4 ? kMaxExperts / 2 : 1];   // rows that picked each expert, 16 bits (in the operands' LDS
                                                     // from five rows on)
  int32_t wave[kWaves];
  int32_t tick, flag;
};
// An expert (10 bits), its first pick in the list (9 bits) and its picks (5 bits).
__device__ __forceinline__ uint32_t pack_uniq(int e, int first, int n) {
  return (uint32_t)e << 14 | (uint32_t)first << 5 | (uint32_t)n;
}

// Waits for every pick and groups them; each block does so for itself, which
// saves two hand-overs.  The number of unique experts, or -1.
template <int MAXR>
__device__ __forceinline__ int group_picks(const MoeArgs& a, BlockLds<MAXR>& b, uint32_t* rows) {
  constexpr int N = (BlockLds<MAXR>::kPk + kThreads - 1) / kThreads;
  const int lane = fresh_lane(), wave = threadIdx.x >> 6, P = a.M * a.k;
  if (threadIdx.x == 0) b.flag = 1;
  for (int i = threadIdx.x; i < (a.E + 1) / 2; i += kThreads) rows[i] = 0;
  __syncthreads();
  int id[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int p = threadIdx.x + j * kThreads;
    id[j] = -1;
    if (p >= P) continue;
    uint64_t v;
    for (int i = 0; !(v = get(&a.picks[p])); ++i)
      if (!poll_on(&a.ctl[C_ERROR], i)) {
        b.flag = 0;
        break;
      }
    id[j] = (int)(v >> 32) - 1;
    if (v) atomicOr(&rows[id[j] >> 1], 1u << (p / a.k + (id[j] & 1) * 16));
  }
  __syncthreads();
  if (!b.flag) return -1;
  // a thread's experts in a row; unique experts and picks before them in one scan (high and low half)
  const int per = (a.E + kThreads - 1) / kThreads, e0 = threadIdx.x * per;
  auto mask = [&](int e) { return rows[e >> 1] >> ((e & 1) * 16) & 0xFFFFu; };
  int mine = 0;
  for (int e = e0; e < min(e0 + per, a.E); ++e) {
    const int n = __popc(mask(e));
    mine += n + (n > 0 ? 1 << 16 : 0);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 63) b.wave[wave] = incl;
  __syncthreads();
  int before = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += b.wave[w];
    all += b.wave[w];
  }
  const int U = __builtin_amdgcn_readfirstlane(all >> 16);
  for (int e = e0; e < min(e0 + per, a.E); ++e) {
    const int n = __popc(mask(e));
    if (n > 0) {
      b.uniq[before >> 16] = pack_uniq(e, before & 0xFFFF, n);
      before += n + (1 << 16);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int p = threadIdx.x + j * kThreads;
    if (p >= P) continue;
    int lo = 0, hi = U - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((int)(b.uniq[mid] >> 14) < id[j]) lo = mid + 1;
      else hi = mid;
    }
    b.pick[(b.uniq[lo] >> 5 & 511) + __popc(mask(id[j]) & ((1u << (p / a.k)) - 1))] = (uint16_t)p;
  }
  __syncthreads();
  return U;
}

template <int MAXR>
__device__ __forceinline__ Work work_of(const MoeArgs& a, const BlockLds<MAXR>& b, int u, bool shared) {
  Work w;
  w.u = u;
  w.row = 0;
  if (!shared) {
    const uint32_t d = __builtin_amdgcn_readfirstlane(b.uniq[u]);
    const int e = d >> 14;
    w.first = d >> 5 & 511;
    w.n = d & 31;
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
template <int MAXR>
__device__ __forceinline__ int pick_at(const MoeArgs& a, const BlockLds<MAXR>& b, const Work& w, int c) {
  return w.first < 0 ? a.M * a.k + w.row + c : b.pick[w.first + w.row + c];
}
template <int MAXR>
__device__ __forceinline__ int token_at(const MoeArgs& a, const BlockLds<MAXR>& b, const Work& w, int c) {
  return w.first < 0 ? w.row + c : (int)((uint32_t)b.pick[w.first + w.row + c] / (uint32_t)a.k);
}
// First element of a pick's row of h: picks [P][I], then the shared expert's [M][Is]
__device__ __forceinline__ uint32_t h_at(const MoeArgs& a, int p) {
  const uint32_t P = a.M * a.k;
  return (uint32_t)p < P ? (uint32_t)p * a.I : P * a.I + ((uint32_t)p - P) * a.Is;
}

// K-elements of ROWS operand rows of `parts` bf16 parts that fit in LDS.
__device__ __forceinline__ int lds_range(int lds, int rows, int parts, int K) {
  const int fit = (lds / (rows * parts) - kPad) / 2 / kStepK * kStepK;
  const int need = (K + kStepK - 1) / kStepK * kStepK;
  return fit < need ? fit : need;
}

// `n` rows of x from column kc to kend (rounded up to whole steps, zeros behind
// the end) into LDS; row c is token tok(c).  Four loads in flight per thread.
template <typename F>
__device__ __forceinline__ void stage_x(const MoeArgs& a, uint8_t* lds, int row_lds, int n, int kc, int kend, F tok) {
  const int per_row = (kend - kc + kStepK - 1) / kStepK * (kStepK / 8), total = n * per_row;
  for (int i0 = threadIdx.x; i0 < total; i0 += 4 * kThreads) {
    u32x4 v[4];
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = min(i0 + j * kThreads, total - 1);
      const int c = (int)((uint32_t)i / (uint32_t)per_row), o = (i - c * per_row) * 8;
      at[j] = c * row_lds + o * 2;
      v[j] = load_x8(a, a.x + tok(c) * a.ldx + min(kc + o, kend - 8));
      if (kc + o >= kend) v[j] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * kThreads < total) *reinterpret_cast<u32x4*>(lds + at[j]) = v[j];
  }
}

// h rows of tiles [tile, end) of an expert, 16 each: a wavefront takes a quad of
// gate rows and the quad of up rows that belongs to it.  x_there: all of x lies
// in LDS (dense) and needs no staging.
template <int ROWS, int MAXR>
__device__ __forceinline__ void gateup_task(const MoeArgs& a, const BlockLds<MAXR>& b, const Work& w, int tile, int end,
                                            uint8_t* lds, bool x_there) {
  constexpr int D = 4, NA = (ROWS + 3) / 4;
  const int lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = a.H;
  const Reader<kNv> rd = reader<kNv>(w.blob, w.blob + (int64_t)w.inter * H, 2u * w.inter, H);
  const int r0 = lane & 3;
  const int KC = a.dense ? (H + kStepK - 1) / kStepK * kStepK : lds_range(a.lds, ROWS, 1, H);
  const int row_lds = KC * 2 + kPad;
  const uint8_t* xs[NA];
#pragma unroll
  for (int s = 0; s < NA; ++s) {
    const int c = 4 * s + r0 < w.n ? 4 * s + r0 : 0;
    xs[s] = lds + (a.dense ? token_at(a, b, w, c) : c) * row_lds + rd.klane * 2;
  }
  // Steps are loaded D ahead, on into the next range of K or the next tile.
  // quads: gate rows, then the up rows that belong to them
  Stage<kNv, false, 2> st[D];
  auto load = [&](int d, int part, int kc, int s) {
    const bool in[2] = {part < end, part < end};
    load_stage<kNv, false, 2>(st[d], rd, part * kUpRows + wave * 4, w.inter, kc + s * kStepK, min(H, kc + KC), in);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, tile, 0, d);
  for (int part = tile; part < end; ++part) {
    const int row0 = part * kUpRows + wave * 4;
    float acc[2][ROWS];
#pragma unroll
    for (int c = 0; c < ROWS; ++c) acc[0][c] = acc[1][c] = 0.0f;
    for (int kc = 0; kc < H; kc += KC) {
      const int kend = min(H, kc + KC), steps = (kend - kc + kStepK - 1) / kStepK, padded = (steps + D - 1) / D * D;
      const bool more = kc + KC < H;
      const int part2 = more ? part : part + 1, kc2 = more ? kc + KC : 0;
      if (!x_there) {
        __syncthreads();
        stage_x(a, lds, row_lds, w.n, kc, kend, [&](int c) { return token_at(a, b, w, c); });
        __syncthreads();
        x_there = KC >= H;
      }
      for (int s = 0; s < steps; s += D) {
        const bool on = s + D < padded;
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s + d < steps) use_stage<kNv, false, 2, ROWS, false>(st[d], xs, (s + d) * kStepK * 2, acc);
          load(d, on ? part : part2, on ? kc : kc2, on ? s + d + D : d);
        }
      }
    }
    tile_sum<ROWS>(acc[0]);
    tile_sum<ROWS>(acc[1]);
    if (tile_sum_owner<ROWS>(lane)) {
      const int first = tile_sum_first<ROWS>(lane);
#pragma unroll
      for (int i = 0; i < kTileOut<ROWS>; ++i) {
        const int c = first + i;
        if (c < w.n)
          put(&a.h[h_at(a, pick_at(a, b, w, c)) + row0 + r0], silu(acc[0][i] * w.gs13) * (acc[1][i] * w.gs13));
      }
    }
  }
}

// Output rows of tiles [tile, end), 32 each, of an expert's down product, per
// pick.  h is
// used to its 24 bits, in three bf16 parts: rounded to one part it would put
// 2^-9 of itself into y, more than all fp32 sums together.  False when the call
// was given up.
template <int ROWS, int MAXR>
__device__ __forceinline__ bool down_task(const MoeArgs& a, BlockLds<MAXR>& b, const Work& w, int tile, int end,
                                          uint8_t* lds) {
  constexpr int Q = 2, D = 4, NA = (ROWS + 3) / 4;
  const int lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int I = w.inter;
  const int64_t w13 = (int64_t)I * a.H + (int64_t)I * a.H / 8, codes = (int64_t)a.H * (I / 2);
  const Reader<kNv> rd = reader<kNv>(w.blob + w13, w.blob + w13 + codes, a.H, I);
  const Rsrc rh = make_rsrc(a.h, (uint32_t)(a.M * (a.k * a.I + a.Is)) * 4);
  const int r0 = lane & 3;
  const int KC = lds_range(a.lds, ROWS, 3, I);
  const int part_lds = KC * 2 + kPad, row_lds = 3 * part_lds;
  const uint8_t* xs[NA];
#pragma unroll
  for (int s = 0; s < NA; ++s) {
    // one row: its parts are the rows of the set
    const int c = 4 * s + r0 < w.n ? 4 * s + r0 : 0;
    xs[s] = lds + (ROWS == 1 ? (r0 < 3 ? r0 : 0) * part_lds : c * row_lds) + rd.klane * 2;
  }
  Stage<kNv, false, Q> st[D];
  auto load = [&](int d, int part, int kc, int s) {
    const bool in[Q] = {part < end, part < end};
    load_stage<kNv, false, Q>(st[d], rd, part * kDownRows + wave * 4 * Q, 4, kc + s * kStepK, min(I, kc + KC), in);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, tile, 0, d);
  if (threadIdx.x == 0) b.flag = wait_for(a, C_HREADY + w.u * kLine);
  bool h_there = false;
  for (int part = tile; part < end; ++part) {
    const int row0 = part * kDownRows + wave * 4 * Q;
    float acc[Q][ROWS];
#pragma unroll
    for (int j = 0; j < Q; ++j)
#pragma unroll
      for (int c = 0; c < ROWS; ++c) acc[j][c] = 0.0f;
    for (int kc = 0; kc < I; kc += KC) {
      const int kend = min(I, kc + KC), steps = (kend - kc + kStepK - 1) / kStepK, padded = (steps + D - 1) / D * D;
      const bool more = kc + KC < I;
      const int part2 = more ? part : part + 1, kc2 = more ? kc + KC : 0;
      if (!h_there) {
        __syncthreads();
        if (!b.flag) return false;
        const int per_row = steps * (kStepK / 4), total = w.n * per_row;
        for (int i0 = threadIdx.x; i0 < total; i0 += 2 * kThreads) {
          u32x4 t[2];
          int at[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = min(i0 + j * kThreads, total - 1);
            const int c = (int)((uint32_t)i / (uint32_t)per_row), o = (i - c * per_row) * 4;
            at[j] = c * row_lds + o * 2;
            t[j] = __builtin_amdgcn_raw_buffer_load_b128(
                rh, kc + o < kend ? (int)((h_at(a, pick_at(a, b, w, c)) + kc + o) * 4) : (int)kBeyond, 0, kAgent);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (i0 + j * kThreads < total) split3(__builtin_bit_cast(f32x4, t[j]), lds + at[j], part_lds);
        }
        __syncthreads();
        h_there = KC >= I;
      }
      for (int s = 0; s < steps; s += D) {
        const bool on = s + D < padded;
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s + d < steps)
            use_stage<kNv, false, Q, ROWS, false, true>(st[d], xs, (s + d) * kStepK * 2, acc, part_lds);
          load(d, on ? part : part2, on ? kc : kc2, on ? s + d + D : d);
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

// y of a tile: the picks in rank order, then the shared expert; eight loads in flight.
__device__ __forceinline__ void combine_tile(const MoeArgs& a, int tile) {
  const int P = a.M * a.k;
  const Rsrc rp = make_rsrc(a.part, (uint32_t)(P + (a.shared ? a.M : 0)) * a.H * 4), rw = make_rsrc(a.picks, P * 8);
  for (int i = threadIdx.x; i < a.M * kDownRows; i += kThreads) {
    const int m = i / kDownRows, r = tile * kDownRows + i % kDownRows, p0 = m * a.k;
    const float sh = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        rp, a.shared ? ((P + m) * a.H + r) * 4 : (int)kBeyond, 0, kAgent));
    float s = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      float v[8], w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = j0 + j < a.k;
        v[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rp, in ? ((p0 + j0 + j) * a.H + r) * 4 : (int)kBeyond, 0, kAgent));
        w[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, in ? (p0 + j0 + j) * 8 : (int)kBeyond, 0, kAgent));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < a.k) s = fmaf(w[j], v[j], s);
    }
    if (a.shared) s += sh;
    store_y(a, m, r, s);
  }
}

// More than eight rows (the shared expert's, or those of an expert that many
// tokens picked) are computed eight at a time: sixteen at once need more
// registers than three blocks per compute unit leave, and the second reading of
// a tile comes from the caches.
template <int MAXR>
__device__ __forceinline__ void run_gateup(const MoeArgs& a, const BlockLds<MAXR>& b, Work w, int tile, int end, uint8_t* lds,
                                           bool x_there) {
  if (w.n == 1) return gateup_task<1>(a, b, w, tile, end, lds, x_there);
  if (w.n == 2) return gateup_task<2>(a, b, w, tile, end, lds, x_there);
  if (MAXR == 4 || w.n <= 4) return gateup_task<4>(a, b, w, tile, end, lds, x_there);
  if constexpr (MAXR > 4) {
    const int n = w.n;
    for (w.row = 0; w.row < n; w.row += 8) {
      w.n = min(8, n - w.row);
      gateup_task<8>(a, b, w, tile, end, lds, x_there);
    }
  }
}
template <int MAXR>
__device__ __forceinline__ bool run_down(const MoeArgs& a, BlockLds<MAXR>& b, Work w, int tile, int end, uint8_t* lds) {
  if (w.n == 1) return down_task<1>(a, b, w, tile, end, lds);
  if (w.n == 2) return down_task<2>(a, b, w, tile, end, lds);
  if (MAXR == 4 || w.n <= 4) return down_task<4>(a, b, w, tile, end, lds);
  if constexpr (MAXR > 4) {
    const int n = w.n;
    for (w.row = 0; w.row < n; w.row += 8) {
      w.n = min(8, n - w.row);
      if (!down_task<8>(a, b, w, tile, end, lds)) return false;
    }
  }
  return true;
}

__device__ __forceinline__ Taker taker(const MoeArgs& a, int phase, int n) {
  Taker t{a.ctl + C_TICKETS + phase * kShards * kLine, n, (int)(blockIdx.x % kShards), 0};
  t.ask();
  return t;
}
// The tasks of U experts of `tiles` tiles each.  Several tiles of an expert are a
// task where there are many, since a task stages its rows first; the last experts'
// tasks are single tiles, so that the blocks end together.  8 rows of 8 picks of
// 4096 x 2048 among 288: 225 us with single tiles throughout, 190 like this (170
// with what came later); 16 rows of 6144 x 2048 among 256: no difference to three
// tiles throughout.
struct Tasks {
  int tiles, f, per, many;      // tiles of an expert; of a task; tasks of an expert; experts cut so
  __device__ __forceinline__ Tasks(int U, int tiles_) : tiles(tiles_) {
    const int most = U * tiles / (kTaskRounds * (int)gridDim.x);
    f = most < 1 ? 1 : most > 4 ? 4 : most;
    per = (tiles + f - 1) / f;
    many = f == 1 ? 0 : U - U / kTaskTail;
  }
  __device__ __forceinline__ int count(int U) const { return many * per + (U - many) * tiles; }
  // Task t: its expert, first tile and the one behind its last.
  __device__ __forceinline__ void at(int t, int& u, int& i0, int& i1) const {
    if (t < many * per) {
      u = t / per;
      i0 = (t - u * per) * f;
      i1 = min(i0 + f, tiles);
    } else {
      t -= many * per;
      u = t / tiles;
      i0 = t - u * tiles;
      i1 = i0 + 1;
      u += many;
    }
  }
};

template <int MAXR>
__device__ __forceinline__ void run_phases(const MoeArgs& a, BlockLds<MAXR>& b, uint8_t* lds) {
  const int tu = a.I / kUpRows, td = a.H / kDownRows, ns = a.shared ? 1 : 0;
  const bool x_there = a.dense;
  {
    Taker k = taker(a, kRouter, a.router_tiles);
    for (int t; (t = k.next(&b.tick)) >= 0;) {
      k.ask();
      if constexpr (MAXR > 4) router_tile_mfma(a, t, reinterpret_cast<float*>(lds));
      else router_tile<MAXR>(a, t, reinterpret_cast<float*>(lds));
    }
  }
  {
    // a wavefront per row
    const int n = (a.M + kWaves - 1) / kWaves;
    Taker k = taker(a, kPick, n);
    for (int t; (t = k.next(&b.tick)) >= 0;) {
      k.ask();
      const int wave = threadIdx.x >> 6, m = t * kWaves + wave;
      b.flag = 1;
      __syncthreads();
      if (m < a.M && route_row<MAXR == 16 ? kRouterShares : 1>(a, &a.ctl[C_ERROR], m,
                                                               reinterpret_cast<float*>(lds) + wave * a.E) != kDone)
        b.flag = 0;
      __syncthreads();
      if (!b.flag) return;
    }
  }
  if (a.dense) {
    stage_x(a, lds, (a.H + kStepK - 1) / kStepK * kStepK * 2 + kPad, a.M, 0, a.H, [](int c) { return c; });
    __syncthreads();
  }
  if (ns) {
    Taker k = taker(a, kShared, a.Is / kUpRows);
    for (int t; (t = k.next(&b.tick)) >= 0;) {
      k.ask();
      run_gateup<MAXR>(a, b, work_of(a, b, kMaxPk, true), t, t + 1, lds, x_there);
      post_h(a, kMaxPk, 1, a.Is / kUpRows);
    }
  }
  Taker kr = taker(a, kRouted, 0);
  const int U = group_picks<MAXR>(a, b, MAXR == 4 ? b.rows : reinterpret_cast<uint32_t*>(lds));
  if (U < 0) return;
  {
    const Tasks tasks(U, tu);
    kr.n = tasks.count(U);
    for (int t; (t = kr.next(&b.tick)) >= 0;) {
      kr.ask();
      int u, i0, i1;
      tasks.at(t, u, i0, i1);
      run_gateup<MAXR>(a, b, work_of(a, b, u, false), i0, i1, lds, x_there);
      post_h(a, u, i1 - i0, tu);
    }
  }
  {
    // the shared expert's h is there first
    const Tasks tasks(U, td);
    const int first = ns * td;
    Taker k = taker(a, kDown, first + tasks.count(U));
    for (int t; (t = k.next(&b.tick)) >= 0;) {
      k.ask();
      const bool sh = t < first;
      int u = kMaxPk, i0 = t, i1 = t + 1;
      if (!sh) tasks.at(t - first, u, i0, i1);
      if (!run_down<MAXR>(a, b, work_of(a, b, u, sh), i0, i1, lds)) return;
      stores_done();
      __syncthreads();
      // one lane per tile counts it; the block combines the tiles that it completed
      if (threadIdx.x < 64) {
        const int i = i0 + threadIdx.x;
        const bool last = i < i1 && add(&a.ctl[C_TILES + i], 1) == U + ns - 1;
        const uint64_t m = __ballot(last);
        if (threadIdx.x == 0) b.flag = (int)m;
      }
      __syncthreads();
      for (uint32_t m = (uint32_t)b.flag; m; m &= m - 1) combine_tile(a, i0 + __builtin_ctz(m));
    }
  }
}

template <int MAXR>
__global__ __launch_bounds__(kThreads, 3) void k_moe_layer(MoeArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ BlockLds<MAXR> b;
  run_phases<MAXR>(a, b, lds);
  // the last block out clears the control words; a call that was given up has no result
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0)
    b.flag = add(&a.ctl[C_EXITS], 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!b.flag) return;
  if (get(&a.ctl[C_ERROR])) abandon(a);
  for (int i = threadIdx.x; i < a.M * a.k; i += kThreads) put(&a.picks[i], (uint64_t)0);
  __syncthreads();
  for (int i = threadIdx.x; i < C_HREADY; i += kThreads) put(&a.ctl[i], 0);
  for (int i = threadIdx.x; i < min(a.M * a.k, a.E); i += kThreads) put(&a.ctl[C_HREADY + i * kLine], 0);
  if (threadIdx.x == 0) put(&a.ctl[C_HREADY + kMaxPk * kLine], 0);
}

// A workspace as it is between calls.
__global__ void k_moe_clear(MoeArgs a, int ctl_words, int picks) {
  const int i0 = blockIdx.x * blockDim.x + threadIdx.x, n = gridDim.x * blockDim.x;
  for (int i = i0; i < ctl_words; i += n) a.ctl[i] = 0;
  for (int i = i0; i < picks; i += n) a.picks[i] = 0;
  for (int i = i0; i < a.logit_words; i += n) a.logits[i] = kNoLogit;
}

// ---- host ------------------------------------------------------------------------

constexpr int kCtlWords = kLayerWords + kOneWords;
constexpr size_t kAlign = 256;
size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct MoeWs {
  size_t ctl, logits, picks, h, part, end;
  int logit_words;
};
MoeWs moe_ws(const sc_moe_config* c) {
  MoeWs o;
  const size_t M = c->max_rows, P = M * c->top_k;
  o.logit_words = (M > 4 ? kRouterShares : 1) * M * c->n_experts;
  size_t p = 0;
  o.ctl = p; p = up(p + kCtlWords * 4);
  o.logits = p; p = up(p + (size_t)o.logit_words * 4);
  o.picks = p; p = up(p + P * 8);
  o.h = p; p = up(p + (P * c->inter + M * c->shared_inter) * 4);
  o.part = p; p = up(p + (P + M) * c->hidden * 4);
  o.end = p;
  return o;
}
// The parts of a workspace.
MoeArgs bind(const sc_moe_config* c, void* d_workspace) {
  uint8_t* ws = static_cast<uint8_t*>(d_workspace);
  const MoeWs o = moe_ws(c);
  MoeArgs a{};
  a.ctl = reinterpret_cast<int32_t*>(ws + o.ctl);
  a.logits = reinterpret_cast<uint32_t*>(ws + o.logits);
  a.picks = reinterpret_cast<uint64_t*>(ws + o.picks);
  a.h = reinterpret_cast<float*>(ws + o.h);
  a.part = reinterpret_cast<float*>(ws + o.part);
  a.logit_words = o.logit_words;
  return a;
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
  const int steps_h = (a.H + kStepK - 1) / kStepK, inter = a.I > a.Is ? a.I : a.Is;
  const int steps_i = (inter + kStepK - 1) / kStepK;
  a.ks = MAXR == 16 ? kRouterShares : 1;
  a.router_tiles = MAXR == 16 ? (a.E + 15) / 16 * a.ks : (a.E + 3) / 4;
  // LDS: the rows of x whole if they fit, and h of one expert's rows; three blocks share a compute unit's 160 KB
  constexpr int most = MAXR == 16 ? 8 : MAXR;   // rows of one expert at a time
  const int dense = a.M * (steps_h * kStepK * 2 + kPad), hrows = (a.M <= 2 ? a.M : most) * 3 * (steps_i * kStepK * 2 + kPad);
  constexpr int cap = 49920;
  static_assert((cap / (most * 3) - kPad) / 2 >= kStepK, "one step of the largest row count must fit");
  const int least = kWaves * a.E * 4 > 4096 ? kWaves * a.E * 4 : 4096;   // routing: scores; router tiles: sums
  a.dense = MAXR == 4 && dense <= cap;
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
  hipLaunchKernelGGL(k_moe_clear, dim3(32), dim3(256), 0, static_cast<hipStream_t>(stream), bind(cfg, d_workspace),
                     kCtlWords, cfg->max_rows * cfg->top_k);
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
  MoeArgs a = bind(c, d_workspace);
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
  hipError_t e;
  bool done = false;
  if (M == 1) {
    MoeArgs one = a;
    one.ctl += kLayerWords;
    e = launch_moe_one(one, st, &done);
  }
  if (!done) e = M <= 4 ? launch_moe<4>(a, st) : launch_moe<16>(a, st);
  return e == hipSuccess ? SC_OK : hip_fail(e, "moe_layer_forward launch");
}

}  // extern "C"
