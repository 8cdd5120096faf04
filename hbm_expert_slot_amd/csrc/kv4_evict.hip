// Eviction from the 4-bit key/value cache by accumulated attention weight.
//
// Of each sequence and head the `keep` tokens with the largest keys stay: tokens
// of the first and last positions before all others, the others by weight, equal
// ones by place.  Attention does not depend on the order of cached tokens (their
// rotary positions are in the keys), so only tokens behind the first `keep` places
// move, into the places that became free: sources and targets never overlap, and
// only what has to move is moved.
//
// 122835 tokens of 8 sequences and 8 heads of 128, NVFP4, cut down to 12000 each: the
// choice 38 us (64 blocks, one per sequence and head: bound by its passes over 32
// tokens per lane and their counters in LDS), the moves 43 us (24300 tokens of each head;
// bound by the scattered pieces of a token, 30 MB read and 42 MB written in all), where
// weights, positions and moved tokens need 13.  Sequences of at most 700 tokens: 13 us,
// for clearing and searching 6144 bins; 131069 tokens of one sequence and 8 heads: 367 us.
#include "kv4_device.h"

#include <type_traits>

namespace sc {
namespace kv4 {
namespace {

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / 64;

struct EvictArgs {
  Pool pool;
  Seqs seqs;
  int32_t keep, recent, sinks;
  int32_t most;             // moves that the lists have room for
  int32_t* count;           // [sequence][head] moves
  int32_t* from;            // [sequence][head][most]
  int32_t* to;              // [sequence][head][most]
  int32_t* new_lens;        // [sequence]
};

// Whole numbers that order like the weights: NaN above infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFEu;
  return b >> 31 ? ~b : b | 0x80000000u;
}

// One block per sequence and head: the keep-th largest key by three rounds of
// counting 11, 11 and 10 bits, then the places that become free and the tokens that
// move there.  A wavefront has consecutive places, 64 at a time, so that places are
// ranked by ballots within it and one sum over the wavefronts.  Up to kHeld rounds
// of places the keys stay in registers; more are formed again in every pass (32768
// tokens: 39 us; 65536: 187).
constexpr int kHeld = 32, kBins = 2048;

__global__ __launch_bounds__(kSelectThreads) void k_kv4_select(EvictArgs a) {
  // of each pass; four counters of a bin side by side, for lanes that meet in it
  __shared__ __align__(16) uint32_t hist[3][kBins][4];
  __shared__ int s_top[kSelectWaves], s_bad[kSelectWaves];
  __shared__ uint32_t s_key[3], s_need[3];
  __shared__ int s_count[6][kSelectWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_index();
  const int b = blockIdx.x / a.pool.heads, head = blockIdx.x % a.pool.heads;
  const int n = length_of(a.seqs, b), np = (n + kPage - 1) / kPage;
  const auto leave = [&]() {
    if (tid != 0) return;
    a.count[blockIdx.x] = 0;
    if (head == 0) a.new_lens[b] = a.seqs.lens[b];
  };
  if (n <= a.keep) return leave();
  const int rounds = (np + kSelectWaves - 1) / kSelectWaves, first = wave * rounds;      // pages of a wavefront
  const int mine = min(rounds, np - first);
  const bool held = rounds <= kHeld;
  // the table's entries of the wavefront's pages are in its lanes, 64 at a time
  int entries = 0, group = -1;
  bool bad = false;                           // a page that is none: the sequence stays as it is
  const auto at_of = [&](int i) -> int64_t {
    if (i >> 6 != group) {
      group = i >> 6;
      const int p = (i & ~63) + lane;
      entries = p < mine ? page_at(a.pool, a.seqs, b, first + p) : 0;
      bad |= __any(entries < 0);
    }
    return ((int64_t)max(__builtin_amdgcn_readlane(entries, i & 63), 0) * a.pool.heads + head) * kPage + lane;
  };
  const auto in = [&](int i) { return (first + i) * kPage + lane < n; };
  uint32_t key[kHeld];
  int pos[kHeld];
  int top = INT32_MIN;
  if (held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < mine && in(i)) {
        pos[i] = a.pool.positions[at_of(i)];
        key[i] = __float_as_uint(a.pool.weights[at_of(i)]);
      }
  }
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) *reinterpret_cast<u32x4*>(hist[0][i]) = u32x4{0, 0, 0, 0};
  if (held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < mine && in(i)) top = max(top, pos[i]);
  } else {
    for (int i = 0; i < mine; ++i) {
      const int64_t at = at_of(i);
      if (in(i)) top = max(top, a.pool.positions[at]);
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, __shfl_xor(top, o));
  if (lane == 0) {
    s_top[wave] = top;
    s_bad[wave] = bad;
  }
  __syncthreads();
  // what each wavefront has, in its first sixteen lanes
  const auto of_waves = [&](const int* s, int otherwise) { return lane < kSelectWaves ? s[lane] : otherwise; };
  if (__any(of_waves(s_bad, 0) != 0)) return leave();
  if (head == 0 && tid == 0) a.new_lens[b] = a.keep;
  top = of_waves(s_top, INT32_MIN);
#pragma unroll
  for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor(top, o));
  const int64_t last = (int64_t)__builtin_amdgcn_readfirstlane(top) - a.recent;
  const auto key_from = [&](int p, float w) { return p < a.sinks || p > last ? 0xFFFFFFFFu : order_of(w); };
  if (held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < mine && in(i)) key[i] = key_from(pos[i], __uint_as_float(key[i]));
  }
  // f(i, key) for the wavefront's rounds of places; a place behind the last has no key
  const auto each = [&](auto&& f) {
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < mine) f(i, in(i), key[i]);
    } else {
      for (int i = 0; i < mine; ++i) {
        const int64_t at = at_of(i);
        const bool is = in(i);
        f(i, is, is ? key_from(a.pool.positions[at], a.pool.weights[at]) : 0u);
      }
    }
  };
  // counts of the wavefronts before this one
  const auto before = [&](int which, int count) {
    if (lane == 0) s_count[which][wave] = count;
    __syncthreads();
    const int upto = wave_scan(of_waves(s_count[which], 0));
    return wave ? __builtin_amdgcn_readlane(upto, wave - 1) : 0;
  };
  uint32_t prefix = 0, need = (uint32_t)a.keep;       // of the tokens whose key begins with prefix
  constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = kShift[pass], bits = pass == 2 ? 10 : 11;
    each([&](int, bool is, uint32_t k) {
      if (is && (pass == 0 || k >> (shift + bits) == prefix)) atomicAdd(&hist[pass][k >> shift & ((1u << bits) - 1)][lane & 3], 1u);
    });
    __syncthreads();
    // the largest bin that the tokens from the top down to it reach `need` in: a thread has two bins, descending
    const int d = kBins - 1 - 2 * tid;
    const u32x4 h0 = *reinterpret_cast<const u32x4*>(hist[pass][d]), h1 = *reinterpret_cast<const u32x4*>(hist[pass][d - 1]);
    const uint32_t c0 = h0.x + h0.y + h0.z + h0.w, c1 = h1.x + h1.y + h1.z + h1.w;
    const int own = wave_scan((int)(c0 + c1));
    const uint32_t upto = (uint32_t)(own + before(pass, __builtin_amdgcn_readlane(own, 63))), above = upto - c0 - c1;
    if (above < need && upto >= need) {
      const bool second = above + c0 < need;
      s_key[pass] = prefix << bits | (uint32_t)(second ? d - 1 : d);
      s_need[pass] = need - above - (second ? c0 : 0);
    }
    __syncthreads();
    prefix = s_key[pass];
    need = s_need[pass];
  }
  // prefix is the keep-th largest key, need the number of its tokens that stay: the first ones
  const uint64_t below = (1ull << lane) - 1;
  // larger keys and equal ones, in front of place `keep` and behind
  int more[2] = {0, 0}, same[2] = {0, 0}, front = 0;
  each([&](int i, bool is, uint32_t k) {
    const uint64_t g = __ballot(is && k > prefix), e = __ballot(is && k == prefix);
    const int left = a.keep - (first + i) * kPage;           // places in front
    const uint64_t f = left >= 64 ? ~0ull : left > 0 ? (1ull << left) - 1 : 0;
    more[0] += __popcll(g & f);
    more[1] += __popcll(g & ~f);
    same[0] += __popcll(e & f);
    same[1] += __popcll(e & ~f);
    front += __popcll(__ballot(is) & f);
  });
  const int equal = before(3, same[0] + same[1]);
  const auto places = [&](auto&& f) {                   // f(i, is, stays)
    int e = equal;
    each([&](int i, bool is, uint32_t k) {
      const uint64_t m = __ballot(is && k == prefix);
      f(i, is, is && (k > prefix || (k == prefix && e + __popcll(m & below) < (int)need)));
      e += __popcll(m);
    });
  };
  // equal ones stay as long as there is need: front ones first
  const int stay = max(0, min((int)need - equal, same[0] + same[1])), stay_front = min(stay, same[0]);
  int nfree = front - more[0] - stay_front, nmove = more[1] + stay - stay_front;
  const int all = nmove;
  nfree = before(4, nfree);
  nmove = before(5, nmove);
  if (wave == kSelectWaves - 1 && lane == 0) a.count[blockIdx.x] = min(nmove + all, a.most);
  int32_t* from = a.from + (int64_t)blockIdx.x * a.most;
  int32_t* to = a.to + (int64_t)blockIdx.x * a.most;
  places([&](int i, bool is, bool stays) {
    const int place = (first + i) * kPage + lane;
    const bool front = place < a.keep, f = is && front && !stays, m = is && !front && stays;
    const uint64_t fs = __ballot(f), ms = __ballot(m);
    const int fi = nfree + __popcll(fs & below), mi = nmove + __popcll(ms & below);
    if (f && fi < a.most) to[fi] = place;
    if (m && mi < a.most) from[mi] = place;
    nfree += __popcll(fs);
    nmove += __popcll(ms);
  });
}

// Sixteen lanes move a token: its pieces of codes, scales, weight and position.  A
// block has 64 consecutive moves, whose tokens share lines on both sides (a wavefront
// per token: 224 us where this takes 43; 32 or 128 moves per block: no difference).
constexpr int kMoves = 64;
template <int D, int FMT>
__global__ __launch_bounds__(256) void k_kv4_move(EvictArgs a) {
  typedef Layout<D, FMT> L;
  constexpr int B = D / 32, U = kMoves / 16;       // bytes of keys and of values per lane; moves of a lane
  typedef std::conditional_t<B == 2, uint16_t, std::conditional_t<B == 4, uint32_t, u32x2>> Key;
  typedef std::conditional_t<L::VDims == 8, uint32_t, uint16_t> Value;
  const int which = blockIdx.x, j = threadIdx.x & 15;
  const int b = which / a.pool.heads, head = which % a.pool.heads, n = a.count[which];
  for (int i0 = blockIdx.y * kMoves; i0 < n; i0 += gridDim.y * kMoves) {
    int f[U], t[U];
    int64_t uf[U], ut[U];
    Key kc[U];
    Value vc[U][L::C];
    uint8_t ks[U], vs[U];
    uint32_t mark[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int64_t i = (int64_t)which * a.most + min(i0 + x * 16 + (int)(threadIdx.x >> 4), n - 1);
      f[x] = a.from[i];
      t[x] = a.to[i];
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      uf[x] = (int64_t)a.seqs.table[b * a.seqs.ld + f[x] / kPage] * a.pool.heads + head;
      ut[x] = (int64_t)a.seqs.table[b * a.seqs.ld + t[x] / kPage] * a.pool.heads + head;
      f[x] %= kPage;
      t[x] %= kPage;
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const uint8_t* s = a.pool.pages + uf[x] * L::kHead;
      kc[x] = *reinterpret_cast<const Key*>(s + f[x] * (D / 2) + j * B);
#pragma unroll
      for (int c = 0; c < L::C; ++c) vc[x][c] = *reinterpret_cast<const Value*>(s + L::kSide + L::value_codes(f[x], c, j));
      if (j < L::NS) {
        ks[x] = s[L::key_scale(f[x], j)];
        vs[x] = s[L::kSide + L::value_scale(f[x], j)];
      }
      if (j < 2) mark[x] = (j ? (const uint32_t*)a.pool.positions : (const uint32_t*)a.pool.weights)[uf[x] * kPage + f[x]];
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      if (i0 + x * 16 + (int)(threadIdx.x >> 4) >= n) continue;
      uint8_t* d = a.pool.pages + ut[x] * L::kHead;
      *reinterpret_cast<Key*>(d + t[x] * (D / 2) + j * B) = kc[x];
#pragma unroll
      for (int c = 0; c < L::C; ++c) *reinterpret_cast<Value*>(d + L::kSide + L::value_codes(t[x], c, j)) = vc[x][c];
      if (j < L::NS) {
        d[L::key_scale(t[x], j)] = ks[x];
        d[L::kSide + L::value_scale(t[x], j)] = vs[x];
      }
      if (j < 2) (j ? (uint32_t*)a.pool.positions : (uint32_t*)a.pool.weights)[ut[x] * kPage + t[x]] = mark[x];
    }
  }
}

sc_status check_evict(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t keep) {
  sc_status s = check_cache(cache);
  if (s == SC_OK) s = check_seqs(seqs);
  if (s != SC_OK) return s;
  if (!cache->d_weights) return fail(SC_E_ARG, "the cache keeps no weights");
  if (keep < 1) return fail(SC_E_ARG, "keep must be positive");
  if ((int64_t)seqs->n_seqs * cache->kv_heads > (1 << 17)) return fail(SC_E_ARG, "too many sequences for one call");
  return SC_OK;
}

int most_moves(const sc_kv4_seqs* seqs, int keep) {
  const int64_t behind = (int64_t)seqs->width * kPage - keep;
  return (int)(behind <= 0 ? 0 : behind < keep ? behind : keep);
}

}  // namespace
}  // namespace kv4
}  // namespace sc

using namespace sc;
using namespace sc::kv4;

extern "C" {

sc_status kv4_evict_workspace_bytes(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t keep, size_t* bytes) {
  if (!bytes) return fail(SC_E_ARG, "bytes is NULL");
  const sc_status s = check_evict(cache, seqs, keep);
  if (s != SC_OK) return s;
  const size_t n = (size_t)seqs->n_seqs * cache->kv_heads;
  *bytes = 4 * n * (1 + 2 * (size_t)most_moves(seqs, keep));
  return SC_OK;
}

sc_status kv4_evict(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, int32_t keep, int32_t recent, int32_t sinks,
                    int32_t* d_new_lens, void* d_workspace, void* stream) {
  const sc_status s = check_evict(cache, seqs, keep);
  if (s != SC_OK) return s;
  if (recent < 0 || sinks < 0 || (int64_t)recent + sinks > keep)
    return fail(SC_E_ARG, "recent and sinks must be >= 0 and together at most keep");
  if (seqs->n_seqs == 0) return SC_OK;
  if (!d_new_lens || (uintptr_t)d_new_lens % 4) return fail(SC_E_ARG, "new lengths are NULL or not 4-byte aligned");
  // every head reads the lengths, one of them writes the new ones
  const uintptr_t old = (uintptr_t)seqs->d_lens, now = (uintptr_t)d_new_lens, bytes = 4 * (uintptr_t)seqs->n_seqs;
  if (now < old + bytes && old < now + bytes) return fail(SC_E_ARG, "new lengths must not overlap the lengths");
  if (!d_workspace || (uintptr_t)d_workspace % 4) return fail(SC_E_ARG, "workspace is NULL or not 4-byte aligned");
  EvictArgs a{};
  a.pool = pool_of(cache);
  a.seqs = seqs_of(seqs);
  a.keep = keep;
  a.recent = recent;
  a.sinks = sinks;
  a.most = most_moves(seqs, keep);
  const int units = seqs->n_seqs * cache->kv_heads;
  a.count = static_cast<int32_t*>(d_workspace);
  a.from = a.count + units;
  a.to = a.from + (int64_t)units * a.most;
  a.new_lens = d_new_lens;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(k_kv4_select, dim3(units), dim3(kSelectThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.most > 0)
    e = by_layout(cache->head_dim, cache->format, [&](auto d, auto f) {
      const int blocks = (a.most + kMoves - 1) / kMoves;
      hipLaunchKernelGGL((k_kv4_move<d(), f()>), dim3(units, blocks < 64 ? blocks : 64), dim3(256), 0, st, a);
      return hipGetLastError();
    });
  if (e != hipSuccess) return hip_fail(e, "kv4_evict launch");
  return SC_OK;
}

}  // extern "C"
