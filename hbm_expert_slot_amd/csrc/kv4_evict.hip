// Eviction from the 4-bit key/value cache by accumulated attention weight.
//
// Of each sequence and head the `keep` tokens with the largest keys stay: tokens
// of the first and last positions before all others, the others by weight, equal
// ones by place.  Attention does not depend on the order of cached tokens (their
// rotary positions are in the keys), so only tokens behind the first `keep` places
// move, into the places that became free: sources and targets never overlap.
#include "kv4_device.h"

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

// One block per sequence and head: the keep-th largest key by four rounds of
// counting bytes, then the places that become free and the tokens that move there.
__global__ __launch_bounds__(kSelectThreads) void k_kv4_select(EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ int s_top, s_bad;
  __shared__ uint32_t s_key, s_need;
  __shared__ int s_wave[kSelectWaves], s_equal, s_free, s_move;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x / a.pool.heads, head = blockIdx.x % a.pool.heads;
  const int n = length_of(a.seqs, b);
  const auto unit_of = [&](int place) -> int64_t {
    return ((int64_t)page_at(a.pool, a.seqs, b, place / kPage) * a.pool.heads + head) * kPage + place % kPage;
  };
  if (tid == 0) {
    s_top = INT32_MIN;
    s_bad = 0;
  }
  __syncthreads();
  if (n > a.keep) {
    // a page that is none: the sequence stays as it is
    for (int i = tid; i < (n + kPage - 1) / kPage; i += kSelectThreads)
      if (page_at(a.pool, a.seqs, b, i) < 0) s_bad = 1;
  }
  __syncthreads();
  const bool leave = n <= a.keep || s_bad;
  if (head == 0 && tid == 0) a.new_lens[b] = leave ? a.seqs.lens[b] : a.keep;
  if (leave) {
    if (tid == 0) a.count[blockIdx.x] = 0;
    return;
  }
  int top = INT32_MIN;
  for (int i = tid; i < n; i += kSelectThreads) top = max(top, a.pool.positions[unit_of(i)]);
  atomicMax(&s_top, top);
  __syncthreads();
  const int64_t last = (int64_t)s_top - a.recent;
  const auto key_of = [&](int place) -> uint32_t {
    const int64_t u = unit_of(place);
    const int p = a.pool.positions[u];
    return p < a.sinks || p > last ? 0xFFFFFFFFu : order_of(a.pool.weights[u]);
  };
  uint32_t prefix = 0, need = (uint32_t)a.keep;       // of the tokens whose key begins with prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelectThreads) {
      const uint32_t k = key_of(i);
      if (shift == 24 || k >> (shift + 8) == prefix) atomicAdd(&hist[k >> shift & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int d = 255;
      for (; d > 0 && above + hist[d] < need; --d) above += hist[d];
      s_key = prefix << 8 | (uint32_t)d;
      s_need = need - above;
    }
    __syncthreads();
    prefix = s_key;
    need = s_need;
    __syncthreads();
  }
  // prefix is the keep-th largest key, need the number of its tokens that stay
  if (tid == 0) s_equal = s_free = s_move = 0;
  int32_t* from = a.from + (int64_t)blockIdx.x * a.most;
  int32_t* to = a.to + (int64_t)blockIdx.x * a.most;
  const auto before = [&](bool mine, int& running) -> int {     // of the places before mine, in order
    const uint64_t m = __ballot(mine);
    __syncthreads();
    if (lane == 0) s_wave[wave] = __popcll(m);
    __syncthreads();
    int sum = running + __popcll(m & ((1ull << lane) - 1)), all = 0;
    for (int w = 0; w < kSelectWaves; ++w) {
      if (w < wave) sum += s_wave[w];
      all += s_wave[w];
    }
    running += all;
    return sum;
  };
  int equal = 0, nfree = 0, nmove = 0;
  for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? key_of(i) : 0u;
    const bool same = i < n && k == prefix;
    const int rank = before(same, equal);
    const bool stays = i < n && (k > prefix || (same && rank < (int)need));
    const int f = before(i < a.keep && !stays, nfree);
    const int v = before(i >= a.keep && stays, nmove);
    if (i < a.keep && !stays && f < a.most) to[f] = i;
    if (i >= a.keep && stays && v < a.most) from[v] = i;
  }
  if (tid == 0) a.count[blockIdx.x] = min(nmove, a.most);
}

// A wavefront moves one token at a time: its pieces of codes, scales, weight and position.
template <int D, int FMT>
__global__ __launch_bounds__(256) void k_kv4_move(EvictArgs a) {
  typedef Layout<D, FMT> L;
  const int which = blockIdx.x, lane = threadIdx.x & 63;
  const int b = which / a.pool.heads, head = which % a.pool.heads, n = a.count[which];
  for (int i = blockIdx.y * 4 + (threadIdx.x >> 6); i < n; i += gridDim.y * 4) {
    const int pf = a.from[(int64_t)which * a.most + i], pt = a.to[(int64_t)which * a.most + i];
    const int64_t uf = (int64_t)page_at(a.pool, a.seqs, b, pf / kPage) * a.pool.heads + head;
    const int64_t ut = (int64_t)page_at(a.pool, a.seqs, b, pt / kPage) * a.pool.heads + head;
    const int f = pf % kPage, t = pt % kPage;
    const uint8_t* src = a.pool.pages + uf * L::kHead;
    uint8_t* dst = a.pool.pages + ut * L::kHead;
    constexpr int B = L::VDims / 2;
    for (int j = lane; j < D / 8; j += 64)
      *reinterpret_cast<uint32_t*>(dst + L::key_codes(t, 8 * j)) = *reinterpret_cast<const uint32_t*>(src + L::key_codes(f, 8 * j));
    for (int j = lane; j < 16 * L::C; j += 64) {
      const uint8_t* s = src + L::kSide + L::value_codes(f, j / 16, j % 16);
      uint8_t* d = dst + L::kSide + L::value_codes(t, j / 16, j % 16);
      if constexpr (B == 4) *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(s);
      else *reinterpret_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(s);
    }
    for (int j = lane; j < L::NS; j += 64) {
      dst[L::key_scale(t, j)] = src[L::key_scale(f, j)];
      dst[L::kSide + L::value_scale(t, j)] = src[L::kSide + L::value_scale(f, j)];
    }
    if (lane == 0) a.pool.weights[ut * kPage + t] = a.pool.weights[uf * kPage + f];
    if (lane == 1) a.pool.positions[ut * kPage + t] = a.pool.positions[uf * kPage + f];
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
      const int blocks = (a.most + 3) / 4;
      hipLaunchKernelGGL((k_kv4_move<d(), f()>), dim3(units, blocks < 64 ? blocks : 64), dim3(256), 0, st, a);
      return hipGetLastError();
    });
  if (e != hipSuccess) return hip_fail(e, "kv4_evict launch");
  return SC_OK;
}

}  // extern "C"
