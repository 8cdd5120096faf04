// One token through a whole mixture-of-experts layer, in one launch.
//
// Bound: HBM, by the bytes of k + 1 experts, and the waits between its products
// (router, picks, h), of a few microseconds each.  Every row of every matrix is
// used once, so the work is cut evenly in advance: one block of 16 wavefronts
// per compute unit takes a share of the router's experts, of the h rows and of
// the output rows, and its wavefronts split the share's 512-element steps
// evenly, wherever in a row that cuts (the pieces of a row are added in LDS, in
// wavefront order).  All of h lies in LDS for the down product, so an output row
// is summed over all experts in one block and there is nothing to combine
// between blocks.  The weights of the next product are on their way while a
// block waits for its operand.
//
// Against the tiles of moe_layer.hip with one row: MI355X_FIGURES
//
// Shares are taken from a counter, one per block.  A wait that lasts takes
// further shares, so that it ends even if some blocks never start (two such
// layers at once may each hold half of the machine).
#include "moe_device.h"

#include <atomic>

namespace sc {
namespace moe {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kPatience = 4096;     // polls (about a millisecond) before a waiting block takes another share
constexpr int kMaxShares = 1024;

// Control words, each group in cache lines of its own; zero between calls.
constexpr int O_SHARES = 0,                             // [part]: shares taken
    O_HDONE = O_SHARES + kShards * kLine,               // [part]: shares whose h is done
    O_EXITS = O_HDONE + kShards * kLine,                // [part]: blocks that left
    O_HROOT = O_EXITS + kShards * kLine,                // parts of O_HDONE that are complete
    O_EROOT = O_HROOT + kLine,                          // parts of O_EXITS that are complete
    O_HREADY = O_EROOT + kLine,                         // flag: all of h is there
    O_ERROR = O_HREADY + kLine;                         // flag: the call was given up
static_assert(O_ERROR + kLine == kOneWords, "");

struct Plan {
  int x_bytes, h_steps, part_h;      // LDS: x; steps of h at a time and the bytes of one of its three parts
  int slots_up, slots_down;          // pieces of rows per wavefront
};

struct OneLds {
  uint64_t pick[kMaxTopK];
  float coef[kMaxTopK + 1];          // weight times matrix scale of the down product
  float sval[kMaxExperts];
  float red[kWaves * 4];
  int32_t from[kWaves + 1], head[kWaves];   // first unit of each wavefront, and its first row quad
  uint16_t list[kMaxShares];         // the block's shares
  int32_t n, tick, flag;
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

// Logits of a share's experts: the wavefronts split H; x lies in LDS.
__device__ __forceinline__ void router_share(const MoeArgs& a, OneLds& s, const uint8_t* x, int share) {
  const int lane = fresh_lane(), wave = threadIdx.x >> 6;
  const Range ex = cut(a.E, share, gridDim.x);
  for (int e0 = ex.lo; e0 < ex.hi; e0 += 4) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = (wave * 64 + lane) * 8; c < a.H; c += kThreads * 8) {
      u32x4 w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e0 + e < ex.hi) w[e] = *reinterpret_cast<const u32x4*>(a.router + (int64_t)(e0 + e) * a.H + c);
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + c * 2);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e0 + e < ex.hi)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[e] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, (uint32_t)w[e][i]),
                                                     __builtin_bit_cast(bf16x2, (uint32_t)v[i]), acc[e], false);
    }
    tile_sum<4>(acc);
    float z = acc[0];
    z += dpp<0x4E>(z);
    z += dpp<0xB1>(z);
    if (tile_sum_owner<4>(lane) && (lane & 3) == 0) s.red[wave * 4 + tile_sum_first<4>(lane)] = z;
    __syncthreads();
    if ((int)threadIdx.x < 4 && e0 + (int)threadIdx.x < ex.hi) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) t += s.red[w * 4 + threadIdx.x];
      put_logit(&a.logits[e0 + threadIdx.x], t);
    }
    __syncthreads();
  }
}

// A row quad's pieces, lying `width` floats apart from slot to slot, in wavefront
// order: f(piece).
template <typename F>
__device__ __forceinline__ void for_pieces(const OneLds& s, const float* part, int slots, int width, int quad, int T, F f) {
  const int lo = quad * T, hi = lo + T;
  for (int w = 0; w < kWaves; ++w)
    if (s.from[w] < s.from[w + 1] && s.from[w] < hi && s.from[w + 1] > lo) f(part + (w * slots + quad - s.head[w]) * width);
}

// ---- gate and up --------------------------------------------------------------------

// h rows of quads [q.lo, q.hi) of the routed picks (quad = pick * I/4 + row / 4)
// or of the shared expert, by wavefronts FIRST .. kWaves - 1.
template <int FIRST>
__device__ __forceinline__ void up_share(const MoeArgs& a, OneLds& s, const uint8_t* x, float* part, int slots, bool shared,
                                         Range q) {
  constexpr int D = 4;
  const int lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int T = (a.H + kStepK - 1) / kStepK, inter = shared ? a.Is : a.I;
  const int units = q.size() * T;
  if (units == 0) return;
  const Range u = wave >= FIRST ? cut(units, wave - FIRST, kWaves - FIRST) : Range{0, 0};
  if (lane == 0) {
    s.from[wave] = u.lo;
    s.head[wave] = u.lo / T;
    if (wave == 0) s.from[kWaves] = units;
  }
  if (u.size() > 0) {
    const uint8_t* xs[1] = {x + (lane >> 2) * 64};
    // where the loads are: pick, row of the pick, step
    int row = (q.lo + u.lo / T) * 4, j = shared ? 0 : row / inter, t = u.lo % T, left = u.size();
    row -= j * inter;
    auto open = [&](int pick) {
      const int e = shared ? 0 : __builtin_amdgcn_readfirstlane((int)(s.pick[pick] >> 32)) - 1;
      const uint8_t* blob = shared ? a.shared : a.blobs + e * a.blob;
      return reader<kNv>(blob, blob + (int64_t)inter * a.H, 2u * inter, a.H);
    };
    Reader<kNv> rd = open(j);
    Stage<kNv, false, 2> st[D];
    auto load = [&](int d) {
      const bool in[2] = {left > 0, left > 0};
      load_stage<kNv, false, 2>(st[d], rd, row, inter, t * kStepK, a.H, in);
      --left;
      if (++t == T) {
        t = 0;
        row += 4;
        if (row == inter && left > 0) {
          row = 0;
          rd = open(++j);
        }
      }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d);
    float acc[2][1] = {{0.0f}, {0.0f}};
    int tu = u.lo % T;
    float* out = part + wave * slots * 8;
    for (int i = 0; i < u.size(); i += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i + d < u.size()) {
          use_stage<kNv, false, 2, 1, false>(st[d], xs, tu * kStepK * 2, acc);
          load(d);
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
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.size() * 4; i += kThreads) {
    float g = 0.0f, up = 0.0f;
    for_pieces(s, part, slots, 8, i >> 2, T, [&](const float* p) {
      g += p[i & 3];
      up += p[4 + (i & 3)];
    });
    const int row = q.lo * 4 + i;
    const int j = shared ? 0 : row / inter;
    const int e = shared ? 0 : (int)(s.pick[j] >> 32) - 1;
    const float gs = shared ? a.sgs[0] : a.gs[2 * e];
    put(&a.h[(shared ? a.k * a.I : 0) + row], silu(g * gs) * (up * gs));
  }
  __syncthreads();
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

// The loads of a wavefront's part of the down product.
struct DownLoads {
  Reader<kNv> rd;
  int row, t, left;      // output row, step on the axis, units to go
  int j, K;              // pick (k: the shared expert) and its inner size
  Range steps;           // of the axis

  __device__ __forceinline__ void open(const MoeArgs& a, const OneLds& s, const Axis& ax) {
    j = t / ax.per;
    if (j > a.k) j = a.k;
    const bool sh = j == a.k;
    const int e = sh ? 0 : __builtin_amdgcn_readfirstlane((int)(s.pick[j] >> 32)) - 1;
    K = sh ? a.Is : a.I;
    const uint8_t* w2 = (sh ? a.shared : a.blobs + e * a.blob) + (int64_t)K * a.H + (int64_t)K * a.H / 8;
    rd = reader<kNv>(w2, w2 + (int64_t)a.H * (K / 2), a.H, K);
  }
  __device__ __forceinline__ void load(const MoeArgs& a, const OneLds& s, const Axis& ax, Stage<kNv, false, 1>& st) {
    const bool in[1] = {left > 0};
    load_stage<kNv, false, 1>(st, rd, row, 4, (t - j * ax.per) * kStepK, K, in);
    --left;
    if (++t == steps.hi) {
      t = steps.lo;
      row += 4;
    }
    // the shared expert's steps may be more than a pick's
    if (left > 0 && (t == steps.lo || (t - j * ax.per == ax.per && j < a.k))) open(a, s, ax);
  }
};

constexpr int kAhead = 8;      // steps in flight per wavefront

__device__ __forceinline__ void down_start(const MoeArgs& a, const OneLds& s, const Axis& ax, Range rows, Range steps,
                                           DownLoads& ld, Stage<kNv, false, 1> (&st)[kAhead]) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), T = steps.size();
  const Range u = cut(rows.size() * T, wave, kWaves);
  ld.steps = steps;
  ld.left = u.size();
  ld.row = (rows.lo + u.lo / T) * 4;
  ld.t = steps.lo + u.lo % T;
  ld.open(a, s, ax);
#pragma unroll
  for (int d = 0; d < kAhead; ++d) ld.load(a, s, ax, st[d]);
}

// h of the steps into LDS, times its pick's weight and scale, in three bf16 parts.
__device__ __forceinline__ void stage_h(const MoeArgs& a, const OneLds& s, const Axis& ax, Range steps, uint8_t* h,
                                        int part_h) {
  const Rsrc rh = make_rsrc(a.h, (uint32_t)(a.k * a.I + a.Is) * 4);
  const int total = steps.size() * (kStepK / 4);
  for (int i0 = threadIdx.x; i0 < total; i0 += 5 * kThreads) {
    u32x4 v[5];
    float c[5];
#pragma unroll
    for (int n = 0; n < 5; ++n) {
      const int i = min(i0 + n * kThreads, total - 1);
      const int t = steps.lo + i / (kStepK / 4), j = min(t / ax.per, a.k);
      const int kk = (t - j * ax.per) * kStepK + i % (kStepK / 4) * 4;
      v[n] = __builtin_amdgcn_raw_buffer_load_b128(rh, kk < (j == a.k ? a.Is : a.I) ? (j * a.I + kk) * 4 : (int)kBeyond, 0,
                                                   kAgent);
      c[n] = s.coef[j];
    }
#pragma unroll
    for (int n = 0; n < 5; ++n)
      if (i0 + n * kThreads < total) split3(__builtin_bit_cast(f32x4, v[n]) * c[n], h + (i0 + n * kThreads) * 8, part_h);
  }
}

// ---- the kernel -------------------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void k_moe_one(MoeArgs a, Plan p) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ OneLds s;
  uint8_t* x = lds;
  uint8_t* h = lds + p.x_bytes;
  float* part = reinterpret_cast<float*>(h + 3 * p.part_h);
  int32_t* error = &a.ctl[O_ERROR];
  const int B = gridDim.x, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;

  Taker shares{a.ctl + O_SHARES, B, (int)(blockIdx.x % kShards), 0};
  shares.ask();
  // x into LDS meanwhile, zero behind the end
  for (int c = threadIdx.x * 8; c < p.x_bytes / 2; c += kThreads * 8) {
    u32x4 v = {0, 0, 0, 0};
    if (c < a.H) v = load_x8(a, a.x + c);
    *reinterpret_cast<u32x4*>(x + c * 2) = v;
  }
  if (threadIdx.x == 0) s.n = 0;
  // takes a share and does its router part; false when there is none left
  auto take = [&]() {
    const int t = shares.next(&s.tick);
    if (t < 0) return false;
    if (threadIdx.x == 0) s.list[s.n++] = (uint16_t)t;
    router_share(a, s, x, t);
    __syncthreads();
    return true;
  };
  auto up_shared = [&](int share, int first) {
    if (!a.shared) return;
    if (first) up_share<1>(a, s, x, part, p.slots_up, true, cut(a.Is / 4, share, B));
    else up_share<0>(a, s, x, part, p.slots_up, true, cut(a.Is / 4, share, B));
  };
  auto up_routed = [&](int share) {
    up_share<0>(a, s, x, part, p.slots_up, false, cut(a.k * a.I / 4, share, B));
    // counted in, part by part: additions to one address take 11 ns each
    stores_done();
    __syncthreads();
    if (threadIdx.x == 0 && add(&a.ctl[O_HDONE + share % kShards * kLine], 1) == (B - share % kShards + kShards - 1) / kShards - 1 &&
        add(&a.ctl[O_HROOT], 1) == min(B, kShards) - 1)
      put(&a.ctl[O_HREADY], 1);
  };

  bool ok = take();
  if (ok) {
    // The block that holds share 0 makes the picks, with its first wavefront; the
    // others go on to the shared expert's h.
    const int own = s.list[0];
    if (own == 0) {
      for (;;) {
        if (wave == 0) {
          const int r = route_row<1>(a, error, 0, s.sval, kPatience);
          if (lane == 0) s.flag = r;
        }
        if (a.shared && s.n == 1) up_shared(0, 1);
        __syncthreads();
        const int r = s.flag;
        __syncthreads();
        if (r == kDone) break;
        if (r == kGivenUp) {
          ok = false;
          break;
        }
        // late: some share has not been taken yet
        if (take()) up_shared(s.list[s.n - 1], 0);
      }
    } else {
      up_shared(own, 0);
    }
    // the picks
    while (ok) {
      if (wave == 0) {
        int r = kDone;
        uint64_t v = 1;
        for (int i = 0;; ++i) {
          if (lane < a.k) v = get(&a.picks[lane]);
          if (!__ballot(v == 0)) break;
          if (i >= kPatience) {
            r = kLate;
            break;
          }
          if (!poll_on(error, i)) {
            r = kGivenUp;
            break;
          }
        }
        if (lane < a.k) s.pick[lane] = v;
        if (lane == 0) s.flag = r;
      }
      __syncthreads();
      const int r = s.flag;
      __syncthreads();
      if (r == kDone) break;
      if (r == kGivenUp) ok = false;
      else if (take()) up_shared(s.list[s.n - 1], 0);
    }
  }
  if (ok) {
    for (int i = threadIdx.x; i <= a.k; i += kThreads)
      s.coef[i] = i < a.k ? __uint_as_float((uint32_t)s.pick[i]) * a.gs[2 * ((int)(s.pick[i] >> 32) - 1) + 1]
                          : a.shared ? a.sgs[1] : 0.0f;
    for (int i = 0; i < s.n; ++i) up_routed(s.list[i]);
    const Axis ax = axis(a);
    const Range head{0, min(ax.total, p.h_steps)};
    DownLoads ld;
    Stage<kNv, false, 1> st[kAhead];
    down_start(a, s, ax, cut(a.H / 4, s.list[0], B), head, ld, st);
    while (ok) {
      if (threadIdx.x == 0) {
        int r = kDone;
        for (int i = 0; !get(&a.ctl[O_HREADY]); ++i) {
          if (i >= kPatience) {
            r = kLate;
            break;
          }
          if (!poll_on(error, i)) {
            r = kGivenUp;
            break;
          }
        }
        s.flag = r;
      }
      __syncthreads();
      const int r = s.flag;
      __syncthreads();
      if (r == kDone) break;
      if (r == kGivenUp) ok = false;
      else if (take()) {
        const int t = s.list[s.n - 1];
        up_shared(t, 0);
        up_routed(t);
        down_start(a, s, ax, cut(a.H / 4, s.list[0], B), head, ld, st);
      }
    }
    for (int i = 0; ok && i < s.n; ++i) {
      const Range rows = cut(a.H / 4, s.list[i], B);
      const int fl = fresh_lane(), r0 = fl & 3;
      const uint8_t* xs[1] = {h + (r0 < 3 ? r0 : 0) * p.part_h + (fl >> 2) * 64};
      float y = 0.0f;      // of the thread's output row
      for (int t0 = 0; t0 < ax.total; t0 += p.h_steps) {
        const Range steps{t0, min(ax.total, t0 + p.h_steps)};
        if (i > 0 || t0 > 0) {
          down_start(a, s, ax, rows, steps, ld, st);
          __syncthreads();
        }
        if (i == 0 || p.h_steps < ax.total) stage_h(a, s, ax, steps, h, p.part_h);
        __syncthreads();
        const int w0 = __builtin_amdgcn_readfirstlane(wave), T = steps.size(), units = rows.size() * T;
        const Range u = cut(units, w0, kWaves);
        float* out = part + w0 * p.slots_down * 4;
        if (lane == 0) {
          s.from[w0] = u.lo;
          s.head[w0] = u.lo / T;
          if (w0 == 0) s.from[kWaves] = units;
        }
        float acc[1][1] = {{0.0f}};
        int tu = T ? u.lo % T : 0;
        for (int n = 0; n < u.size(); n += kAhead) {
#pragma unroll
          for (int d = 0; d < kAhead; ++d) {
            if (n + d < u.size()) {
              use_stage<kNv, false, 1, 1, false, true>(st[d], xs, tu * kStepK * 2, acc);
              ld.load(a, s, ax, st[d]);
              if (++tu == T || n + d == u.size() - 1) {
                tile_sum<1>(acc[0]);
                if (lane < 4) out[lane] = acc[0][0];
                out += 4;
                acc[0][0] = 0.0f;
                tu = 0;
              }
            }
          }
        }
        __syncthreads();
        if ((int)threadIdx.x < rows.size() * 4) {
          for_pieces(s, part, p.slots_down, 4, threadIdx.x >> 2, T, [&](const float* v) { y += v[threadIdx.x & 3]; });
        }
        __syncthreads();
      }
      if ((int)threadIdx.x < rows.size() * 4) store_y(a, 0, rows.lo * 4 + threadIdx.x, y);
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

hipError_t launch_moe_one(const MoeArgs& a, hipStream_t st) {
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
  auto share = [&](int n) { return (n + B - 1) / B; };
  const int up = share(a.k * a.I / 4), ups = share(a.Is / 4), down = share(a.H / 4);
  // a wavefront's steps are a run: it touches its part of the quads and one more at either end; the shared
  // expert's are split among one wavefront less in one block
  p.slots_up = ((up + kWaves - 1) / kWaves > (ups + kWaves - 2) / (kWaves - 1) ? (up + kWaves - 1) / kWaves
                                                                              : (ups + kWaves - 2) / (kWaves - 1)) + 2;
  p.slots_down = (down + kWaves - 1) / kWaves + 2;
  const int pu = kWaves * p.slots_up * 32, pd = kWaves * p.slots_down * 16, parts = pu > pd ? pu : pd;
  const int total = a.k * ((a.I + kStepK - 1) / kStepK) + (a.shared ? (a.Is + kStepK - 1) / kStepK : 0);
  const int room = 163840 - (int)sizeof(OneLds) - 1280 - p.x_bytes - parts;
  const int fit = (room / 3 - kPad) / (kStepK * 2);
  p.h_steps = fit < total ? fit : total;
  p.part_h = p.h_steps * kStepK * 2 + kPad;
  if (p.h_steps < 1) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k_moe_one, dim3(B), dim3(kThreads), p.x_bytes + 3 * p.part_h + parts, st, a, p);
  return hipGetLastError();
}

}  // namespace moe
}  // namespace sc
