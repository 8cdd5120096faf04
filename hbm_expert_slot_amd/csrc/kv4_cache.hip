// The 4-bit key/value cache: writing tokens into its pages, and reading them back.
//
// Codes and scales follow the rule of fp4_quantize with a given scale: a group's
// scale is the nearest to max / (6 scale) (NVFP4) or 2^(floor(log2 max) - 2)
// (MXFP4), a code the nearest to the exact quotient.
//
// What bounds them: HBM, and for writing the vector instructions of the rounding
// (about 100 for 16 elements).  17417 tokens of 8 heads of 128: fp16 to MXFP4 27 us (90
// MB, 3.3 TB/s), back to fp32 29 us (162 MB, 5.5 TB/s).  With the values written past the
// caches both together take 54.6 us, through them 61.
#include "fp4_round.h"
#include "kv4_device.h"

namespace sc {
namespace kv4 {
namespace {

constexpr int kThreads = 256;

constexpr int kMaxTokens = 64;   // of a block

struct RowArgs {
  Pool pool;
  Seqs seqs;
  const int32_t* starts;     // [n + 1], or null: tokens are dealt out evenly
  const int32_t* given;      // positions [tokens], or null: the places
  const float* gs[2];
  void* rows[2];             // keys, values
  int64_t token[2], head[2]; // strides
  int32_t tokens;
  int32_t block_tokens;
  int32_t per;               // threads that a token's rows take
  bool write;
};

// Sequence and place of a token of the packed rows; place -1: it is not there, -2:
// it belongs to no sequence.  starts: a.starts, or a copy of them.
__device__ __forceinline__ int place_of(const RowArgs& a, const int32_t* starts, int t, int& b) {
  int end;
  if (a.starts) {
    int lo = 0, hi = a.seqs.n;           // starts[lo] <= t < starts[hi]
    if (t < starts[0] || t >= starts[hi]) return -2;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    end = starts[lo + 1];
  } else {
    const int each = a.tokens / a.seqs.n;
    b = t / each;
    end = (b + 1) * each;
  }
  const int64_t p = (int64_t)a.seqs.lens[b] - (end - t);
  return p >= 0 && p < (int64_t)a.seqs.width * kPage ? (int)p : -1;
}

// Where the tokens of a block lie, found once for all of their rows: offset of the
// page (-1: none, -2: the token belongs to no sequence), and the places of a token's
// codes and scales in a head's keys and values.
struct Places {
  int64_t page[kMaxTokens];
  uint32_t codes[2][kMaxTokens], scales[2][kMaxTokens];
  int32_t starts[kThreads];
};
template <int D, int FMT>
__device__ __forceinline__ int find_places(const RowArgs& a, Places& p, int t0) {
  typedef Layout<D, FMT> L;
  const int n = min(a.block_tokens, a.tokens - t0), i = threadIdx.x;
  // a search in LDS waits for memory once, not at every step
  const bool copied = a.starts && a.seqs.n < kThreads;
  if (copied) {
    if (i <= a.seqs.n) p.starts[i] = a.starts[i];
    __syncthreads();
  }
  if (i < n) {
    int b;
    const int place = copied ? place_of(a, p.starts, t0 + i, b) : place_of(a, a.starts, t0 + i, b), t = place & (kPage - 1);
    const int page = place < 0 ? place : page_at(a.pool, a.seqs, b, place / kPage);
    p.page[i] = page < 0 ? page : (int64_t)page * a.pool.heads;
    p.codes[0][i] = L::key_codes(t, 0);
    p.codes[1][i] = L::value_codes(t, 0, 0);
    p.scales[0][i] = L::key_scale(t, 0);
    p.scales[1][i] = L::value_scale(t, 0);
    if (blockIdx.y == 0 && page >= 0 && a.pool.weights && a.write) {
      const int at = a.given ? a.given[t0 + i] : place;
      for (int h = 0; h < a.pool.heads; ++h) {
        const int64_t m = (p.page[i] + h) * kPage + t;
        a.pool.weights[m] = 0.0f;
        a.pool.positions[m] = at;
      }
    }
  }
  __syncthreads();
  return n;
}

// A thread has one piece of a token's rows (keys of all heads, then values) and goes
// through the block's tokens with it; small rows leave threads for several tokens at
// a time.
struct Work {
  int piece, side, head, first, last;      // tokens of the block
};
template <int N>
__device__ __forceinline__ Work work_of(const RowArgs& a, int n) {
  Work w;
  const int at_once = max(1, kThreads / a.per), each = (n + at_once - 1) / at_once;
  const int mine = a.per >= kThreads ? 0 : threadIdx.x / a.per;
  const int i = a.per >= kThreads ? blockIdx.y * kThreads + threadIdx.x : threadIdx.x - mine * a.per;
  w.piece = i % N;
  const int row = i / N;
  w.side = row >= a.pool.heads;
  w.head = row - (w.side ? a.pool.heads : 0);
  w.first = mine * each;
  w.last = i < a.per && mine < at_once ? min(n, w.first + each) : 0;
  return w;
}

// A thread takes 16 elements of a token at a time; the next ones are on their way
// while it works on these.
template <typename T, int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_kv4_append(RowArgs a) {
  typedef Layout<D, FMT> L;
  constexpr int N = D / 16;
  struct Raw {
    T v[16];
  };
  __shared__ Places places;
  const int t0 = blockIdx.x * a.block_tokens, n = find_places<D, FMT>(a, places, t0);
  const Work w = work_of<N>(a, n);
  const int s16 = w.piece, sg = FMT == kNv ? s16 : s16 / 2;
  const int64_t step = a.token[w.side];
  const T* src = static_cast<const T*>(a.rows[w.side]) + (t0 + w.first) * step + w.head * a.head[w.side] + s16 * 16;
  const float gs = FMT == kNv && a.gs[w.side] ? *a.gs[w.side] : 1.0f;
  // of token 0 of a page
  uint8_t* at0 = a.pool.pages + w.head * (int64_t)L::kHead + w.side * L::kSide;
  const uint32_t code = w.side ? L::value_codes(0, D >= 128 ? s16 / 8 : 0, D >= 128 ? s16 % 8 * 2 : s16 * 4) : s16 * 8;
  const uint32_t scale = w.side ? L::value_scale(0, sg) - L::value_scale(0, 0) : L::key_scale(0, sg) - L::key_scale(0, 0);
  constexpr int U = sizeof(T) == 4 ? 1 : 2;      // tokens whose loads are under way together
  Raw raw[U];
  const auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < w.last) __builtin_memcpy(&raw[u], src + (i0 + u - w.first) * step, sizeof(Raw));
  };
  load(w.first);
  for (int i0 = w.first; i0 < w.last; i0 += U) {
    Raw now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = raw[u];
    load(i0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= w.last) break;
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = (float)now[u].v[e];
      uint32_t sbyte;
      u32x2 codes;
      round16<FMT, sizeof(T) == 2>(v, gs, sbyte, codes);
      const int64_t page = places.page[i];
      if (page < 0) continue;
      uint8_t* at = at0 + page * L::kHead;
      if (FMT == kNv || (s16 & 1) == 0) at[scale + places.scales[w.side][i]] = (uint8_t)sbyte;
      at += code + places.codes[w.side][i];
      if (w.side == 0) {
        *reinterpret_cast<u32x2*>(at) = codes;
      } else if constexpr (D >= 128) {
        *reinterpret_cast<uint32_t*>(at) = codes.x;
        *reinterpret_cast<uint32_t*>(at + 16) = codes.y;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint16_t*>(at + j * 8) = (uint16_t)(codes[j / 2] >> (j % 2 * 16));
      }
    }
  }
}

// A thread writes 16 bytes of a token at a time, so that a wavefront's stores are one piece.
template <typename T, int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_kv4_read(RowArgs a) {
  typedef Layout<D, FMT> L;
  constexpr int E = 16 / sizeof(T), N = D / E;
  __shared__ Places places;
  const int t0 = blockIdx.x * a.block_tokens, n = find_places<D, FMT>(a, places, t0);
  const Work w = work_of<N>(a, n);
  const int dim = w.piece * E, sg = dim / L::G;
  const int64_t step = a.token[w.side];
  T* dst = static_cast<T*>(a.rows[w.side]) + (t0 + w.first) * step + w.head * a.head[w.side] + dim;
  const float gs = FMT == kNv && a.gs[w.side] ? *a.gs[w.side] : 1.0f;
  const uint8_t* at0 = a.pool.pages + w.head * (int64_t)L::kHead + w.side * L::kSide;
  const uint32_t code = w.side ? L::value_codes(0, D >= 128 ? dim / 128 : 0, dim % (16 * L::VDims) / L::VDims) + dim % L::VDims / 2
                               : dim / 2;
  const uint32_t scale = w.side ? L::value_scale(0, sg) - L::value_scale(0, 0) : L::key_scale(0, sg) - L::key_scale(0, 0);
  constexpr int U = 4;               // tokens whose loads are under way together
  typedef __attribute__((ext_vector_type(E), aligned(sizeof(T)))) T V;
  struct Batch {
    uint32_t codes[U], sb[U];
  };
  const auto load = [&](Batch& x, int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u, w.last - 1);
      const uint8_t* at = at0 + max(places.page[i], (int64_t)0) * L::kHead;
      x.sb[u] = at[scale + places.scales[w.side][i]];
      at += code + places.codes[w.side][i];
      if constexpr (E == 4) {
        x.codes[u] = *reinterpret_cast<const uint16_t*>(at);
      } else if constexpr (D >= 128) {
        x.codes[u] = *reinterpret_cast<const uint32_t*>(at);
      } else {           // values: eight dimensions are of two lanes
        x.codes[u] = *reinterpret_cast<const uint16_t*>(at) |
                     (uint32_t)*reinterpret_cast<const uint16_t*>(at + (w.side ? 8 : 2)) << 16;
      }
    }
  };
  if (w.first >= w.last) return;
  Batch next;
  load(next, w.first);
  for (int i0 = w.first; i0 < w.last; i0 += U) {
    const Batch x = next;
    load(next, i0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t page = places.page[min(i0 + u, w.last - 1)];
      float s = FMT == kNv ? __builtin_amdgcn_cvt_pk_f32_fp8((int)x.sb[u], false)[0] : e8m0(x.sb[u]);
      if (page < 0) s = NAN;
      V out;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const f32x2 y = e == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.codes[u], 1.0f, 0)
                        : e == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.codes[u], 1.0f, 1)
                        : e == 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.codes[u], 1.0f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(x.codes[u], 1.0f, 3);
        // code times group scale is exact; one rounding by the scale of all
        out[e] = (T)(y.x * s * gs);
        out[e + 1] = (T)(y.y * s * gs);
      }
      // past the caches: what is read back is many times what was read
      if (i0 + u < w.last && page != -2) __builtin_nontemporal_store(out, reinterpret_cast<V*>(dst + (i0 + u - w.first) * step));
    }
  }
}

int type_size(int t) { return t == SC_DTYPE_F32 ? 4 : 2; }

template <bool WRITE, typename T>
hipError_t run(RowArgs a, int dim, int fmt, hipStream_t st) {
  a.write = WRITE;
  a.per = 2 * a.pool.heads * (WRITE ? dim / 16 : dim * (int)sizeof(T) / 16);
  const int groups = (a.per + kThreads - 1) / kThreads, at_once = a.per < kThreads ? kThreads / a.per : 1;
  // twelve tokens for each thread, fewer where that leaves compute units idle
  const int64_t even = ((int64_t)a.tokens * groups + 1023) / 1024, full = 12 * at_once;
  const int64_t n = full < even ? full : even;
  a.block_tokens = (int)(n < 1 ? 1 : n < kMaxTokens ? n : kMaxTokens);
  const unsigned grid = (unsigned)((a.tokens + a.block_tokens - 1) / a.block_tokens);
  return by_layout(dim, fmt, [&](auto d, auto f) {
    if constexpr (WRITE) hipLaunchKernelGGL((k_kv4_append<T, d(), f()>), dim3(grid, groups), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_kv4_read<T, d(), f()>), dim3(grid, groups), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  });
}

template <bool WRITE>
sc_status rows(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_rows* r, int32_t tokens,
               const int32_t* starts, const int32_t* positions, void* stream) {
  sc_status s = check_cache(cache);
  if (s == SC_OK) s = check_seqs(seqs);
  if (s != SC_OK) return s;
  if (!r) return fail(SC_E_ARG, "rows are NULL");
  if (r->type != SC_DTYPE_BF16 && r->type != SC_DTYPE_F16 && r->type != SC_DTYPE_F32)
    return fail(SC_E_ARG, "unknown type %d", r->type);
  if (tokens < 0) return fail(SC_E_ARG, "tokens must be >= 0");
  if ((uintptr_t)starts % 4 || (uintptr_t)positions % 4) return fail(SC_E_ARG, "starts or positions are not aligned");
  if (tokens == 0 || seqs->n_seqs == 0) return SC_OK;
  if (!starts && tokens % seqs->n_seqs)
    return fail(SC_E_ARG, "%d tokens cannot be dealt out evenly to %d sequences", tokens, seqs->n_seqs);
  // a launch has less than 2^32 threads: with less than 2^32 elements per side never over 0.26 of that, as a thread
  // has at least 8 elements of a token and a block 12 tokens (but for about 1024 blocks, where there are fewer)
  if ((int64_t)tokens * cache->kv_heads * cache->head_dim >= (int64_t)1 << 32)
    return fail(SC_E_ARG, "too many tokens for one call");
  const int size = type_size(r->type);
  if (!r->d_k || !r->d_v || (uintptr_t)r->d_k % size || (uintptr_t)r->d_v % size)
    return fail(SC_E_ARG, "k or v is NULL or not aligned to its elements");
  if (r->k_token < 0 || r->v_token < 0 || r->k_head < 0 || r->v_head < 0)
    return fail(SC_E_ARG, "strides must be >= 0");
  RowArgs a{};
  a.pool = pool_of(cache);
  a.seqs = seqs_of(seqs);
  a.starts = starts;
  a.given = positions;
  a.gs[0] = cache->d_k_scale;
  a.gs[1] = cache->d_v_scale;
  a.rows[0] = r->d_k;
  a.rows[1] = r->d_v;
  a.token[0] = r->k_token;
  a.token[1] = r->v_token;
  a.head[0] = r->k_head;
  a.head[1] = r->v_head;
  a.tokens = tokens;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int d = cache->head_dim, f = cache->format;
  const hipError_t e = r->type == SC_DTYPE_F32   ? run<WRITE, float>(a, d, f, st)
                       : r->type == SC_DTYPE_F16 ? run<WRITE, _Float16>(a, d, f, st)
                                                 : run<WRITE, __bf16>(a, d, f, st);
  if (e != hipSuccess) return hip_fail(e, WRITE ? "kv4_append launch" : "kv4_read launch");
  return SC_OK;
}

}  // namespace

sc_status check_cache(const sc_kv4_cache* c) {
  if (!c) return fail(SC_E_ARG, "cache is NULL");
  if (c->format != SC_FP4_NV && c->format != SC_FP4_MX) return fail(SC_E_ARG, "unknown format %d", c->format);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(SC_E_ARG, "head_dim must be 64, 128 or 256");
  if (c->kv_heads < 1 || c->kv_heads > SC_KV4_MAX_HEADS)
    return fail(SC_E_ARG, "kv_heads must be in [1, %d]", SC_KV4_MAX_HEADS);
  if (c->n_pages < 1) return fail(SC_E_ARG, "n_pages must be positive");
  if (!c->d_pages || (uintptr_t)c->d_pages % 16) return fail(SC_E_ARG, "pages are NULL or not 16-byte aligned");
  if (!c->d_weights != !c->d_positions) return fail(SC_E_ARG, "weights and positions belong together");
  if ((uintptr_t)c->d_weights % 16 || (uintptr_t)c->d_positions % 16)
    return fail(SC_E_ARG, "weights and positions must be 16-byte aligned");
  if ((uintptr_t)c->d_k_scale % 4 || (uintptr_t)c->d_v_scale % 4) return fail(SC_E_ARG, "scales must be 4-byte aligned");
  if (c->format == SC_FP4_MX && (c->d_k_scale || c->d_v_scale)) return fail(SC_E_ARG, "only NVFP4 has a global scale");
  return SC_OK;
}

sc_status check_seqs(const sc_kv4_seqs* s) {
  if (!s) return fail(SC_E_ARG, "sequences are NULL");
  if (s->n_seqs < 0 || s->n_seqs > SC_KV4_MAX_SEQS) return fail(SC_E_ARG, "n_seqs must be in [0, %d]", SC_KV4_MAX_SEQS);
  if (s->width < 1 || s->width > SC_KV4_MAX_WIDTH) return fail(SC_E_ARG, "width must be in [1, %d]", SC_KV4_MAX_WIDTH);
  if (s->n_seqs == 0) return SC_OK;
  if (s->ld_table < s->width && s->n_seqs > 1) return fail(SC_E_ARG, "the table's rows overlap");
  if (!s->d_table || !s->d_lens || (uintptr_t)s->d_table % 4 || (uintptr_t)s->d_lens % 4)
    return fail(SC_E_ARG, "table or lengths are NULL or not 4-byte aligned");
  return SC_OK;
}

}  // namespace kv4
}  // namespace sc

using namespace sc;

extern "C" {

sc_status kv4_page_bytes(int32_t format, int32_t head_dim, size_t* bytes) {
  if (!bytes) return fail(SC_E_ARG, "bytes is NULL");
  if (format != SC_FP4_NV && format != SC_FP4_MX) return fail(SC_E_ARG, "unknown format %d", format);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return fail(SC_E_ARG, "head_dim must be 64, 128 or 256");
  *bytes = kv4::by_layout(head_dim, format, [](auto d, auto f) { return (size_t)kv4::Layout<d(), f()>::kHead; });
  return SC_OK;
}

sc_status kv4_append(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_rows* rows, int32_t tokens,
                     const int32_t* d_starts, const int32_t* d_positions, void* stream) {
  return kv4::rows<true>(cache, seqs, rows, tokens, d_starts, d_positions, stream);
}

sc_status kv4_read(const sc_kv4_cache* cache, const sc_kv4_seqs* seqs, const sc_kv4_rows* rows, int32_t tokens,
                   const int32_t* d_starts, void* stream) {
  return kv4::rows<false>(cache, seqs, rows, tokens, d_starts, nullptr, stream);
}

}  // extern "C"
