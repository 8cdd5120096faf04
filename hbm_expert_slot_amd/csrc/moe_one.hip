// One token through a whole mixture-of-experts layer, in one launch.
//
// Bound: HBM, by the bytes of k + 1 experts, and the waits between its products
// (router, picks, h), of a few microseconds each.  Every row of every matrix is
// used once, so the work is cut evenly in advance: one block of 12 wavefronts
// per compute unit takes a share of the router's experts, of the h rows and of
// the output rows, and its wavefronts split the share's 512-element steps
// evenly, wherever in a row that cuts (the pieces of a row are added in LDS, in
// wavefront order).  All of h lies in LDS for the down product, so an output row
// is summed over all experts in one block and there is nothing to combine
// between blocks.  The weights of the next product are on their way while a
// block waits for its operand.
//
// Against the tiles of moe_layer.hip with one row: 54 us, those 74 (8 of 256
// experts of 6144 x 2048 and a shared one: 191 MB, 3.5 TB/s).
//
// Block b takes share b.  A wait that lasts looks for a share that no block has
// claimed and does it too, so that it ends even if some blocks never start (two
// such layers at once may each hold half of the machine).  A pair of calls at the
// size above: 104 us on two streams (up to 169 seen), 107 on one; a call beside
// 4096 x 4096 x 4096 products on another stream 149 us, alone 57.
//
// Loads return in order within a wavefront, so whoever polls or fetches h must
// have no weights on their way: the first four wavefronts do that, the other
// eight the down product.
#include "moe_device.h"

#include <atomic>

namespace sc {
namespace moe {
namespace {

constexpr int kThreads = 768, kWaves = kThreads / 64;
constexpr int kPatience = 4096;     // polls (about a millisecond) before a waiting block takes another share
constexpr int kMaxLate = kMaxPolls / kPatience;      // such waits of a block after which the call is given up
constexpr int kMaxShares = 1024;
constexpr int kService = 4, kDownWaves = kWaves - kService;   // see above

// Control words, each group in cache lines of its own; zero between calls.
constexpr int O_CLAIM = 0,                              // [share]: taken
    O_HDONE = O_CLAIM + kMaxShares,                     // [part]: wavefronts that have put their part of a share's h
    O_EXITS = O_HDONE + kShards * kLine,                // [part]: blocks that left
    O_HROOT = O_EXITS + kShards * kLine,                // parts of O_HDONE that are complete
    O_EROOT = O_HROOT + kLine,                          // parts of O_EXITS that are complete
    O_ERROR = O_EROOT + kLine;                          // flag: the call was given up
static_assert(O_ERROR + kLine == kOneWords, "");

struct Plan {
  int x_bytes, h_steps, part_h;      // LDS: x; steps of h at a time and the bytes of one of its three parts
  int slots_up;                      // pieces of h rows per wavefront
  int putters;                       // wavefronts that add a share's pieces and put its h
};

struct OneLds {
  uint64_t pick[kMaxTopK];
  float gs13[kMaxTopK];              // matrix scale of each pick's gate and up
  float coef[kMaxTopK + 1];          // weight times matrix scale of the down product
  float sval[kMaxExperts];
  float red[kWaves * 4];
  int32_t from[kWaves + 1], head[kWaves];   // first unit of each wavefront, and its first row quad
  int32_t state[kService];
  uint16_t list[kMaxShares];         // the block's shares
  int32_t n, flag, taken;
  MoeArgs args;                      // for take_over
  Plan plan;
};

struct Range {
  int lo, hi;
  __device__ __forceinline__ int size() const { return hi - lo; }
};
// Part `i` of n things cut into `of` parts (n * of < 2^31).
__device__ __forceinline__ Range cut(int n, int i, int of) {
  return {(int)((uint32_t)(n * i) / (uint32_t)of), (int)((uint32_t)(n * (i + 1)) / (uint32_t)of)};
}

// ---- router ------------------------------------------------------------------------

// A thread's first loads of the router product: four experts' elements 8 tid .. + 7.
struct RouterLoads {
  u32x4 w[4], x;
  __device__ __forceinline__ void start(const MoeArgs& a, int share) {
    const int c = fresh_thread() * 8;
    const Range ex = cut(a.E, share, gridDim.x);
    x = u32x4{0, 0, 0, 0};
    if (c < a.H) x = load_x8(a, a.x + c);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c < a.H && ex.lo + e < ex.hi) w[e] = *reinterpret_cast<const u32x4*>(a.router + (int64_t)(ex.lo + e) * a.H + c);
  }
};

// Logits of a share's experts: the wavefronts split H.  `lost` (thread 0): somebody
// else has claimed the share; nothing is stored then and the result is false.
// loaded(): called when the last loads have been used.
template <typename F>
__device__ __forceinline__ bool router_share(const MoeArgs& a, OneLds& s, int share, int lost, RouterLoads& ld, F loaded) {
  const int tid = fresh_thread(), lane = tid & 63, wave = tid >> 6;
  const Range ex = cut(a.E, share, gridDim.x);
  for (int e0 = ex.lo; e0 < ex.hi || e0 == ex.lo; e0 += 4) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = tid * 8; c < a.H; c += kThreads * 8) {
      if (e0 > ex.lo || c >= kThreads * 8) {
        ld.x = load_x8(a, a.x + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e0 + e < ex.hi) ld.w[e] = *reinterpret_cast<const u32x4*>(a.router + (int64_t)(e0 + e) * a.H + c);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e0 + e < ex.hi)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (uint32_t)ld.w[e][i]),
                                                     __builtin_bit_cast(bf16x2, (uint32_t)ld.x[i]), acc[e], false);
    }
    tile_sum<4>(acc);
    float z = acc[0];
    z += dpp<0x4E>(z);
    z += dpp<0xB1>(z);
    if (e0 + 4 >= ex.hi) loaded();
    if (tile_sum_owner<4>(lane) && (lane & 3) == 0) s.red[wave * 4 + tile_sum_first<4>(lane)] = z;
    if (tid == 0) s.flag = !lost;
    __syncthreads();
    if (!s.flag) return false;
    if (tid < 4 && e0 + tid < ex.hi) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) t += s.red[w * 4 + tid];
      put_logit(&a.logits[e0 + tid], t);
    }
    __syncthreads();
  }
  return true;
}

// A row quad's pieces, lying `width` floats apart from slot to slot, in wavefront
// order: f(piece).  The units are cut among `nw` wavefronts.
template <typename F>
__device__ __forceinline__ void for_pieces(const OneLds& s, const float* part, int slots, int width, int quad, int T,
                                           int nw, F f) {
  const int lo = quad * T, hi = lo + T, units = s.from[nw];
  int w = (int)((uint32_t)(lo * nw) / (uint32_t)units);      // at or before the first
  while (s.from[w + 1] <= lo) ++w;
  for (; w < nw && s.from[w] < hi; ++w)
    if (s.from[w] < s.from[w + 1]) f(part + (w * slots + quad - s.head[w]) * width);
}
// Notes a wavefront's units for for_pieces.
__device__ __forceinline__ void note_units(OneLds& s, int wave, int nw, Range u, int T, int units) {
  if (fresh_lane() == 0) {
    s.from[wave] = u.lo;
    s.head[wave] = u.lo / T;
    if (wave == nw - 1) s.from[nw] = units;
  }
}

// Where a wavefront's units lie: lane i holds unit i of a window of 64, so that
// the arithmetic of expert, row and step is done once for all of them, and a load
// reads its unit's place out of a lane.
struct Places {
  uint32_t code_lo, code_hi, scale_lo, scale_hi;
  int left;            // elements from the step to the end of the row; 0 behind the last unit
  uint32_t code, scale;         // the lane's own offsets within a quad: row lane % 4, element 32 (lane / 4)
  int klane;

  __device__ __forceinline__ void own(int lane, int K) {
    klane = (lane >> 2) * 32;
    code = (lane & 3) * (uint32_t)(K / 2) + klane / 2;
    scale = (lane & 3) * (uint32_t)(K / 16) + klane / 16;
  }
  // matrix of rows of K elements, codes at `codes` and scales `after` bytes on
  __device__ __forceinline__ void set(const uint8_t* codes, int64_t after, int64_t row, int K, int k, bool in) {
    const uint64_t c = (uint64_t)codes + row * (K / 2) + k / 2;
    const uint64_t t = (uint64_t)codes + after + row * (K / 16) + k / 16;
    code_lo = (uint32_t)c;
    code_hi = (uint32_t)(c >> 32);
    scale_lo = (uint32_t)t;
    scale_hi = (uint32_t)(t >> 32);
    left = in ? K - k : 0;
  }
  static __device__ __forceinline__ const void* at(uint32_t lo, uint32_t hi, int i) {
    return (const void*)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, i) << 32 |
                         (uint32_t)__builtin_amdgcn_readlane((int)lo, i));
  }
  // Unit i; its Q quads lie apart_c and apart_s bytes apart.
  template <int Q>
  __device__ __forceinline__ void load(Stage<kNv, false, Q>& st, int i, uint32_t apart_c, uint32_t apart_s) const {
    const Rsrc rc = make_rsrc(at(code_lo, code_hi, i), kBeyond - 1), rs = make_rsrc(at(scale_lo, scale_hi, i), kBeyond - 1);
    const bool on = klane < __builtin_amdgcn_readlane(left, i);
    const uint32_t lc = on ? code : kBeyond, ls = on ? scale : kBeyond;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      st.q[j] = load16(rc, lc, j * apart_c);
      st.s[j] = load2(rs, ls, j * apart_s);
    }
  }
};
constexpr int kWindow = 32;     // units after which the window moves on (loads run ahead of it)

// ---- gate and up --------------------------------------------------------------------

// h rows of quads [q.lo, q.hi) of the routed picks (quad = pick * I/4 + row / 4)
// or of the shared expert.
template <bool SHARED>
struct UpShare {
  static constexpr int D = 4;      // steps in flight per wavefront, gate and up
  Places pl;
  Stage<kNv, false, 2> st[D];
  Range q, u;
  int T, inter;

  __device__ __forceinline__ void window(const MoeArgs& a, const OneLds& s, int n) {
    const int v = u.lo + n + fresh_lane(), quad = (int)((uint32_t)v / (uint32_t)T), t = v - quad * T;
    const bool in = v < u.hi;
    int row = (q.lo + quad) * 4;
    const int j = SHARED ? 0 : (int)((uint32_t)row / (uint32_t)inter);
    row -= j * inter;
    const int e = SHARED || !in ? 0 : (int)(s.pick[j] >> 32) - 1;
    pl.set(SHARED ? a.shared : a.blobs + e * a.blob, (int64_t)inter * a.H, row, a.H, t * kStepK, in);
  }
  __device__ __forceinline__ void load(const MoeArgs& a, int d, int i) {
    pl.load(st[d], i, (uint32_t)inter * (a.H / 2), (uint32_t)inter * (a.H / 16));
  }
  __device__ __forceinline__ void start(const MoeArgs& a, const OneLds& s, Range quads) {
    const int wave = wave_index();
    q = quads;
    T = (a.H + kStepK - 1) / kStepK;
    inter = SHARED ? a.Is : a.I;
    u = cut(q.size() * T, wave, kWaves);
    if (u.size() == 0) return;
    pl.own(fresh_lane(), a.H);
    window(a, s, 0);
#pragma unroll
    for (int d = 0; d < D; ++d) load(a, d, d);
  }
  // x lies in LDS.  The first wavefronts add the pieces and put h; their stores
  // need not have been performed yet.
  __device__ __forceinline__ void finish(const MoeArgs& a, OneLds& s, const uint8_t* x, float* part, const Plan& p);
};

template <bool SHARED>
__device__ __forceinline__ void UpShare<SHARED>::finish(const MoeArgs& a, OneLds& s, const uint8_t* x, float* part,
                                                        const Plan& p) {
  const int lane = fresh_lane(), wave = wave_index();
  const int units = q.size() * T;
  if (units == 0) return;
  note_units(s, wave, kWaves, u, T, units);
  const uint8_t* xs[1] = {x + (lane >> 2) * 64};
  float acc[2][1] = {{0.0f}, {0.0f}};
  int tu = u.lo % T, w0 = 0;
  float* out = part + wave * p.slots_up * 8;
  for (int i = 0; i < u.size(); i += D) {
    if (i - w0 >= kWindow) {
      w0 = i;
      window(a, s, w0);
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i + d < u.size()) {
        use_stage<kNv, false, 2, 1, false>(st[d], xs, tu * kStepK * 2, acc);
        load(a, d, i - w0 + d + D);
        if (++tu == T || i + d == u.size() - 1) {
          tile_sum<1>(acc[0]);
          tile_sum<1>(acc[1]);
          if (lane < 4) {
            out[lane] = acc[0][0];
            out[4 + lane] = acc[1][0];
          }
          out += 8;
          acc[0][0] = acc[1][0] = 0.0f;
          tu = 0;
        }
      }
    }
  }
  __syncthreads();
  if (wave < p.putters) {
    for (int i = fresh_thread(); i < q.size() * 4; i += p.putters * 64) {
      float g = 0.0f, up = 0.0f;
      for_pieces(s, part, p.slots_up, 8, i >> 2, T, kWaves, [&](const float* v) {
        g += v[i & 3];
        up += v[4 + (i & 3)];
      });
      const int row = q.lo * 4 + i;
      const float gs = SHARED ? a.sgs[0] : s.gs13[row / inter];
      put(&a.h[(SHARED ? a.k * a.I : 0) + row], silu(g * gs) * (up * gs));
    }
  }
}

// ---- down -----------------------------------------------------------------------------

// The K axis of the down product: the picks' h one after the other, each padded
// to whole steps, then the shared expert's.
struct Axis {
  int per, total;      // steps of a pick and of all
};
__device__ __forceinline__ Axis axis(const MoeArgs& a) {
  const int per = (a.I + kStepK - 1) / kStepK, sh = a.shared ? (a.Is + kStepK - 1) / kStepK : 0;
  return {per, a.k * per + sh};
}

// The down product of a share: each of its eight wavefronts takes a run of
// steps (all of them a part of every output row), or, where there are fewer
// steps than wavefronts, a step and a part of the rows.  A slab is one step of
// kSlab row quads; a wavefront keeps two of them in flight.
constexpr int kSlab = 6, kSlabs = 2, kEarly = 2;

struct DownWave {
  Range steps;      // of the axis
  Range quads;      // of the share
  int slice, slices;      // which of the runs of steps, and how many there are
  int count;        // slabs

  __device__ __forceinline__ DownWave(int wave, Range all, Range rows) {
    const int T = all.size();
    slices = min(T, kDownWaves);
    const int groups = kDownWaves / slices, group = wave / slices;
    slice = wave - group * slices;
    const Range t = cut(T, slice, slices), r = cut(rows.size(), min(group, groups - 1), groups);
    steps = {all.lo + t.lo, all.lo + t.hi};
    quads = {rows.lo + r.lo, rows.lo + r.hi};
    count = group < groups ? (r.size() + kSlab - 1) / kSlab * t.size() : 0;
  }
  // Slab i: all steps of the first kSlab quads, then of the next.
  __device__ __forceinline__ void load(const MoeArgs& a, const OneLds& s, const Axis& ax, Stage<kNv, false, kSlab>& st,
                                       int i) const {
    const int g = (int)((uint32_t)i / (uint32_t)steps.size()), t = steps.lo + i - g * steps.size();
    const int j = min((int)((uint32_t)t / (uint32_t)ax.per), a.k);
    const bool sh = j == a.k;
    const int e = sh ? 0 : __builtin_amdgcn_readfirstlane((int)(s.pick[j] >> 32)) - 1, K = sh ? a.Is : a.I;
    const uint8_t* w2 = (sh ? a.shared : a.blobs + e * a.blob) + (int64_t)K * a.H + (int64_t)K * a.H / 8;
    const Reader<kNv> rd = reader<kNv>(w2, w2 + (int64_t)a.H * (K / 2), a.H, K);
    const int q = quads.lo + g * kSlab;
    bool in[kSlab];
#pragma unroll
    for (int n = 0; n < kSlab; ++n) in[n] = i < count && q + n < quads.hi;
    load_stage<kNv, false, kSlab>(st, rd, q * 4, 4, (t - j * ax.per) * kStepK, K, in);
  }
};

// h of the steps into LDS, times its pick's weight and scale, in three bf16
// parts; by the service wavefronts.
__device__ __forceinline__ void stage_h(const MoeArgs& a, const OneLds& s, const Axis& ax, Range steps, uint8_t* h,
                                        int part_h) {
  constexpr int N = 18, kThr = kService * 64;     // all of it in flight where there are eight picks of 2048 and a shared expert
  const Rsrc rh = make_rsrc(a.h, (uint32_t)(a.k * a.I + a.Is) * 4);
  const int total = steps.size() * (kStepK / 4);
  for (int i0 = fresh_thread(); i0 < total; i0 += N * kThr) {
    u32x4 v[N];
    float c[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = min(i0 + n * kThr, total - 1);
      const int t = steps.lo + i / (kStepK / 4), j = min(t / ax.per, a.k);
      const int kk = (t - j * ax.per) * kStepK + i % (kStepK / 4) * 4;
      v[n] = __builtin_amdgcn_raw_buffer_load_b128(rh, kk < (j == a.k ? a.Is : a.I) ? (j * a.I + kk) * 4 : (int)kBeyond, 0,
                                                   kAgent);
      c[n] = s.coef[j];
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (i0 + n * kThr < total) split3(__builtin_bit_cast(f32x4, v[n]) * c[n], h + (i0 + n * kThr) * 8, part_h);
  }
}

// A wavefront's slabs: its part of each output row, part[slice][quad of the share][4].
__device__ __forceinline__ void down_slabs(const MoeArgs& a, const OneLds& s, const Axis& ax, const DownWave& d, Range all,
                                           Range rows, const uint8_t* h, int part_h, float* part,
                                           Stage<kNv, false, kSlab> (&st)[kSlabs]) {
  const int lane = fresh_lane(), r0 = lane & 3;
  const uint8_t* xs[1] = {h + (r0 < 3 ? r0 : 0) * part_h + (lane >> 2) * 64};
  float acc[kSlab][1];
#pragma unroll
  for (int n = 0; n < kSlab; ++n) acc[n][0] = 0.0f;
  int t = d.steps.lo, q = d.quads.lo;
  for (int i = 0; i < d.count; i += kSlabs) {
#pragma unroll
    for (int b = 0; b < kSlabs; ++b) {
      if (i + b < d.count) {
        use_stage<kNv, false, kSlab, 1, false, true>(st[b], xs, (t - all.lo) * kStepK * 2, acc);
        if (i + b + kSlabs < d.count) d.load(a, s, ax, st[b], i + b + kSlabs);
        if (++t == d.steps.hi) {
          t = d.steps.lo;
#pragma unroll
          for (int n = 0; n < kSlab; ++n) {
            tile_sum<1>(acc[n]);
            if (lane < 4 && q + n < d.quads.hi) part[(d.slice * rows.size() + q + n - rows.lo) * 4 + lane] = acc[n][0];
            acc[n][0] = 0.0f;
          }
          q += kSlab;
        }
      }
    }
  }
}

// ---- the kernel -------------------------------------------------------------------------

// The shared expert's quads of a share.  The block that makes the picks (share 0)
// has none.
__device__ __forceinline__ Range shared_quads(const MoeArgs& a, int share, int B) {
  if (B == 1) return {0, a.Is / 4};
  return share == 0 ? Range{0, 0} : cut(a.Is / 4, share - 1, B - 1);
}

// A share's routed h, counted in (part by part: additions to one address take 11 ns each).
__device__ __forceinline__ void up_routed(const MoeArgs& a, OneLds& s, const uint8_t* x, float* part, const Plan& p,
                                          int share) {
  const int B = gridDim.x, shard = share % kShards, tid = fresh_thread();
  UpShare<false> up;
  up.start(a, s, cut(a.k * a.I / 4, share, B));
  up.finish(a, s, x, part, p);
  if (tid < p.putters * 64) {
    stores_done();     // of the shared expert's h too
    if ((tid & 63) == 0 &&
        add(&a.ctl[O_HDONE + shard * kLine], 1) == (B - shard + kShards - 1) / kShards * p.putters - 1)
      add(&a.ctl[O_HROOT], 1);
  }
}

// A wait has lasted: takes a share that no block has claimed, if there is one,
// and does its part so far.  Not inlined, and with its arguments in LDS: it
// hardly ever runs, and costs the kernel no registers.
__device__ __noinline__ void take_over(OneLds* ps, uint8_t* lds, bool picks) {
  OneLds& s = *ps;
  const MoeArgs& a = s.args;
  const uint8_t* x = lds;
  float* part = reinterpret_cast<float*>(lds + s.plan.x_bytes + 3 * s.plan.part_h);
  const int B = gridDim.x, lane = fresh_lane();
  __syncthreads();
  if (threadIdx.x < 64) {
    int t = -1;
    for (int t0 = 0; t0 < B && t < 0; t0 += 64) {
      const uint64_t m = __ballot(t0 + lane < B && !get(&a.ctl[O_CLAIM + t0 + lane]));
      if (!m) continue;
      const int c = t0 + __builtin_ctzll(m);
      int was = 0;
      if (lane == 0) was = __hip_atomic_exchange(&a.ctl[O_CLAIM + c], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (!__builtin_amdgcn_readfirstlane(was)) t = c;
    }
    if (lane == 0) {
      s.taken = t;
      if (t >= 0) s.list[s.n++] = (uint16_t)t;
    }
  }
  __syncthreads();
  const int t = __builtin_amdgcn_readfirstlane(s.taken);
  if (t < 0) return;
  RouterLoads rl;
  rl.start(a, t);
  router_share(a, s, t, 0, rl, []() {});
  if (a.shared) {
    UpShare<true> up;
    up.start(a, s, shared_quads(a, t, B));
    up.finish(a, s, x, part, s.plan);
  }
  __syncthreads();
  if (picks) up_routed(a, s, x, part, s.plan, t);
  __syncthreads();
}

// Polls until ready() is true on every lane, for a while.
template <typename F>
__device__ __forceinline__ int poll(int32_t* error, F ready) {
  for (int i = 0;; ++i) {
    if (!__ballot(!ready())) return kDone;
    if (i >= kPatience) return kLate;
    if (!poll_on(error, i)) return kGivenUp;
  }
}

__global__ __launch_bounds__(kThreads) void k_moe_one(MoeArgs a, Plan p) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ OneLds s;
  uint8_t* x = lds;
  uint8_t* h = lds + p.x_bytes;
  float* part = reinterpret_cast<float*>(h + 3 * p.part_h);
  int32_t* error = &a.ctl[O_ERROR];
  const int B = gridDim.x, wave = wave_index(), lane = fresh_lane();

  int lost = 0, late = 0;
  if (threadIdx.x == 0) {
    s.n = 1;
    s.list[0] = (uint16_t)blockIdx.x;
    s.args = a;
    s.plan = p;
    lost = __hip_atomic_exchange(&a.ctl[O_CLAIM + blockIdx.x], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // the shared expert's weights follow the router's: ahead of them they would hold up the picks
  RouterLoads rl;
  rl.start(a, blockIdx.x);
  const u32x4 x0 = rl.x;
  UpShare<true> sh;
  // false: another block has taken the share over
  bool ok = router_share(a, s, blockIdx.x, lost, rl, [&]() {
    if (a.shared) sh.start(a, s, shared_quads(a, blockIdx.x, B));
  });
  if (ok) {
    // x into LDS, zero behind the end
    const int tid = fresh_thread();
    if (tid * 16 < p.x_bytes) *reinterpret_cast<u32x4*>(x + tid * 16) = x0;
    for (int c = (tid + kThreads) * 8; c < p.x_bytes / 2; c += kThreads * 8) {
      u32x4 v = {0, 0, 0, 0};
      if (c < a.H) v = load_x8(a, a.x + c);
      *reinterpret_cast<u32x4*>(x + c * 2) = v;
    }
    __syncthreads();
    if (a.shared) sh.finish(a, s, x, part, p);
    // the picks: made by the first wavefront of the block that holds share 0, waited for by every block's
    bool routed = false;      // by this block
    for (;;) {
      if (wave == 0) {
        int r = kDone;
        for (int i = 0; i < s.n && r == kDone; ++i)
          if (s.list[i] == 0 && !routed) {
            r = route_row<1>(a, error, 0, s.sval, kPatience);
            routed = r == kDone;
          }
        uint64_t v = 1;
        if (r == kDone) r = poll(error, [&]() { return lane >= a.k || (v = get(&a.picks[lane])) != 0; });
        if (r == kDone && lane < a.k) {
          const int e = (int)(v >> 32) - 1;
          s.pick[lane] = v;
          s.gs13[lane] = a.gs[2 * e];
          s.coef[lane] = __uint_as_float((uint32_t)v) * a.gs[2 * e + 1];
        }
        if (lane == 0) {
          s.coef[a.k] = a.shared ? a.sgs[1] : 0.0f;
          s.flag = r;
        }
      }
      __syncthreads();
      const int r = s.flag;
      if (r == kDone) break;
      if (r == kGivenUp) {
        ok = false;
        break;
      }
      if (++late == kMaxLate && threadIdx.x == 0) put(error, 1);
      take_over(&s, lds, false);
    }
  }
  if (ok) {
    for (int i = 0; i < s.n; ++i) {
      up_routed(a, s, x, part, p, s.list[i]);
      if (i + 1 < s.n) __syncthreads();
    }
    // All of h.  The wavefronts part here, and meet at as many barriers on either way.
    const Axis ax = axis(a);
    const Range head{0, min(ax.total, p.h_steps)};
    for (;;) {
      int r = kDone;
      auto meet = [&]() {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kService; ++i) r = max(r, s.state[i]);
        return r == kDone;
      };
      if (wave >= kService) {
        Stage<kNv, false, kSlab> st[kSlabs];
        const Range rows0 = cut(a.H / 4, s.list[0], B);
        DownWave d(wave - kService, head, rows0);
        auto start = [&](int from, int to) {
#pragma unroll
          for (int b = 0; b < kSlabs; ++b)
            if (b >= from && b < to) d.load(a, s, ax, st[b], b);
        };
        start(0, kEarly);
        if (meet()) {
          start(kEarly, kSlabs);
          for (int i = 0; i < s.n; ++i) {
            const Range rows = cut(a.H / 4, s.list[i], B);
            for (int t0 = 0; t0 < ax.total; t0 += p.h_steps) {
              const Range steps{t0, min(ax.total, t0 + p.h_steps)};
              if (i > 0 || t0 > 0) {
                d = DownWave(wave - kService, steps, rows);
                start(0, kSlabs);
                __syncthreads();
              }
              down_slabs(a, s, ax, d, steps, rows, h, p.part_h, part, st);
              __syncthreads();
              __syncthreads();
            }
          }
        }
      } else {
        int mine = poll(error, [&]() { return get(&a.ctl[O_HROOT]) >= min(B, kShards); });
        if (mine == kDone) stage_h(a, s, ax, head, h, p.part_h);
        if (lane == 0) s.state[wave] = mine;
        if (meet()) {
          for (int i = 0; i < s.n; ++i) {
            const Range rows = cut(a.H / 4, s.list[i], B);
            const int tid = fresh_thread();
            float y = 0.0f;      // of the thread's output row
            for (int t0 = 0; t0 < ax.total; t0 += p.h_steps) {
              const Range steps{t0, min(ax.total, t0 + p.h_steps)};
              if (i > 0 || t0 > 0) {
                if (p.h_steps < ax.total) stage_h(a, s, ax, steps, h, p.part_h);
                __syncthreads();
              }
              __syncthreads();
              if (tid < rows.size() * 4)
                for (int w = 0; w < min(steps.size(), kDownWaves); ++w) y += part[w * rows.size() * 4 + tid];
              __syncthreads();
            }
            if (tid < rows.size() * 4) store_y(a, 0, rows.lo * 4 + tid, y);
          }
        }
      }
      if (r != kLate) break;
      if (++late == kMaxLate && threadIdx.x == 0) put(error, 1);
      take_over(&s, lds, true);
    }
  }

  // the last block out clears what was handed over; a call that was given up has no result
  stores_done();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int part16 = blockIdx.x % kShards;
    s.flag = add(&a.ctl[O_EXITS + part16 * kLine], 1) == (B - part16 + kShards - 1) / kShards - 1 &&
             add(&a.ctl[O_EROOT], 1) == min(B, kShards) - 1;
  }
  __syncthreads();
  if (!s.flag) return;
  if (get(error)) abandon(a);
  if ((int)threadIdx.x < a.k) put(&a.picks[threadIdx.x], (uint64_t)0);
  __syncthreads();
  for (int i = threadIdx.x; i < kOneWords; i += kThreads) put(&a.ctl[i], 0);
}

}  // namespace

hipError_t launch_moe_one(const MoeArgs& a, hipStream_t st, bool* fits) {
  *fits = true;
  static std::atomic<int> units[64];
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  int cus = units[dev % 64].load(std::memory_order_relaxed);
  if (!cus) {
    e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    units[dev % 64].store(cus, std::memory_order_relaxed);
  }
  // one block per compute unit; fewer where a block would have less than 16 rows
  const int most = a.k * a.I > a.H ? a.k * a.I : a.H;
  int B = (most + 15) / 16;
  if (B > cus) B = cus;
  if (B > kMaxShares) B = kMaxShares;
  Plan p;
  const int steps = (a.H + kStepK - 1) / kStepK;
  p.x_bytes = steps * kStepK * 2;
  auto share = [](int n, int of) { return (n + of - 1) / of; };
  const int up = share(a.k * a.I / 4, B), ups = share(a.Is / 4, B > 1 ? B - 1 : 1), down = share(a.H / 4, B);
  // a wavefront's steps are a run: it touches its part of the quads and one more at either end
  p.slots_up = ((up > ups ? up : ups) + kWaves - 1) / kWaves + 2;
  p.putters = up <= 16 && ups <= 16 ? 1 : kService;      // quads of four rows: one wavefront adds up to 64 rows
  const int pu = kWaves * p.slots_up * 32, pd = kDownWaves * down * 16, parts = pu > pd ? pu : pd;
  const int total = a.k * ((a.I + kStepK - 1) / kStepK) + (a.shared ? (a.Is + kStepK - 1) / kStepK : 0);
  const int room = 163840 - (int)sizeof(OneLds) - 1280 - p.x_bytes - parts;
  const int fit = (room / 3 - kPad) / (kStepK * 2);
  p.h_steps = fit < total ? fit : total;
  p.part_h = p.h_steps * kStepK * 2 + kPad;
  // on a device of few compute units a share can be too large for a block
  *fits = p.h_steps >= 1 && down * 4 <= kService * 64;
  if (!*fits) return hipSuccess;
  hipLaunchKernelGGL(k_moe_one, dim3(B), dim3(kThreads), p.x_bytes + 3 * p.part_h + parts, st, a, p);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace sc
