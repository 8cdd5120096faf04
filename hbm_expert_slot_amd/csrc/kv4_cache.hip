// The 4-bit key/value cache: writing tokens into its pages, and reading them back.
//
// Codes and scales follow the rule of fp4_quantize with a given scale: a group's
// scale is the nearest to max / (6 scale) (NVFP4) or 2^(floor(log2 max) - 2)
// (MXFP4), a code the nearest to the exact quotient.
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
  uint32_t per_magic;        // x / (2 heads) is the upper half of x times this
};

// Sequence and place of a token of the packed rows; place -1: it is not there, -2:
// it belongs to no sequence.
__device__ __forceinline__ int place_of(const RowArgs& a, int t, int& b) {
  int end;
  if (a.starts) {
    int lo = 0, hi = a.seqs.n;           // starts[lo] <= t < starts[hi]
    if (t < a.starts[0] || t >= a.starts[hi]) return -2;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    end = a.starts[lo + 1];
  } else {
    const int each = a.tokens / a.seqs.n;
    b = t / each;
    end = (b + 1) * each;
  }
  const int64_t p = (int64_t)a.seqs.lens[b] - (end - t);
  return p >= 0 && p < (int64_t)a.seqs.width * kPage ? (int)p : -1;
}

// Where the tokens of a block lie: found once for all of their rows.
struct Places {
  int page[kMaxTokens], place[kMaxTokens];
};
__device__ __forceinline__ int find_places(const RowArgs& a, Places& p, int t0) {
  const int n = min(a.block_tokens, a.tokens - t0);
  if ((int)threadIdx.x < n) {
    int b;
    const int place = place_of(a, t0 + threadIdx.x, b);
    p.place[threadIdx.x] = place;
    p.page[threadIdx.x] = place < 0 ? -1 : page_at(a.pool, a.seqs, b, place / kPage);
  }
  __syncthreads();
  return n;
}

// Row r of a block's tokens: keys of all heads, then values, token after token.
struct Row {
  int token, side, head;
};
__device__ __forceinline__ Row row_of(const RowArgs& a, int r) {
  Row w;
  w.token = (int)__umulhi((uint32_t)r, a.per_magic);
  const int in = r - w.token * 2 * a.pool.heads;
  w.side = in >= a.pool.heads;
  w.head = in - (w.side ? a.pool.heads : 0);
  return w;
}

// A thread takes 16 elements of a row at a time; the next ones are on their way
// while it works on these.
template <typename T, int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_kv4_append(RowArgs a) {
  typedef Layout<D, FMT> L;
  constexpr int N = D / 16, R = kThreads / N;      // threads of a row, rows at a time
  struct Raw {
    T v[16];
  };
  __shared__ Places places;
  const int t0 = blockIdx.x * a.block_tokens, s16 = threadIdx.x % N;
  const int rows = find_places(a, places, t0) * 2 * a.pool.heads;
  const auto load = [&](int r) {
    const Row w = row_of(a, min(r, rows - 1));
    Raw x;
    __builtin_memcpy(&x, static_cast<const T*>(a.rows[w.side]) + (t0 + w.token) * a.token[w.side] + w.head * a.head[w.side] +
                             s16 * 16, sizeof x);
    return x;
  };
  int r = threadIdx.x / N;
  Raw raw = load(r);
  for (; r < rows; r += R) {
    const Raw next = load(r + R);
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = (float)raw.v[e];
    raw = next;
    const Row w = row_of(a, r);
    uint32_t sbyte;
    u32x2 codes;
    round16<FMT>(v, FMT == kNv && a.gs[w.side] ? *a.gs[w.side] : 1.0f, sbyte, codes);
    const int page = places.page[w.token], place = places.place[w.token];
    if (page < 0) continue;
    const int t = place % kPage;
    const int64_t unit = (int64_t)page * a.pool.heads + w.head;
    uint8_t* at = a.pool.pages + unit * L::kHead + w.side * L::kSide;
    const int sg = FMT == kNv ? s16 : s16 / 2;
    if (FMT == kNv || (s16 & 1) == 0) at[w.side ? L::value_scale(t, sg) : L::key_scale(t, sg)] = (uint8_t)sbyte;
    if (w.side == 0) {
      *reinterpret_cast<u32x2*>(at + L::key_codes(t, s16 * 16)) = codes;
      if (s16 == 0 && a.pool.weights) {
        a.pool.weights[unit * kPage + t] = 0.0f;
        a.pool.positions[unit * kPage + t] = a.given ? a.given[t0 + w.token] : place;
      }
    } else if constexpr (D >= 128) {
      const int c = s16 / 8, ln = s16 % 8 * 2;
      *reinterpret_cast<uint32_t*>(at + L::value_codes(t, c, ln)) = codes.x;
      *reinterpret_cast<uint32_t*>(at + L::value_codes(t, c, ln + 1)) = codes.y;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint16_t*>(at + L::value_codes(t, 0, s16 * 4 + j)) = (uint16_t)(codes[j / 2] >> (j % 2 * 16));
    }
  }
}

// A thread writes 16 bytes of a row at a time, so that a wavefront's stores are one piece.
template <typename T, int D, int FMT>
__global__ __launch_bounds__(kThreads) void k_kv4_read(RowArgs a) {
  typedef Layout<D, FMT> L;
  constexpr int E = 16 / sizeof(T), N = D / E, R = kThreads / N;
  __shared__ Places places;
  const int t0 = blockIdx.x * a.block_tokens, p = threadIdx.x % N, dim = p * E;
  const int rows = find_places(a, places, t0) * 2 * a.pool.heads;
#pragma unroll 2
  for (int r = threadIdx.x / N; r < rows; r += R) {
    const Row w = row_of(a, r);
    const int page = places.page[w.token], place = places.place[w.token];
    if (place == -2) continue;
    typedef __attribute__((ext_vector_type(E))) T V;
    V out;
    if (page < 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) out[e] = (T)__builtin_nanf("");
    } else {
      const int t = place % kPage, sg = dim / L::G;
      const uint8_t* at = a.pool.pages + ((int64_t)page * a.pool.heads + w.head) * L::kHead + w.side * L::kSide;
      const uint32_t sb = at[w.side ? L::value_scale(t, sg) : L::key_scale(t, sg)];
      const auto two = [&](uint32_t off) { return (uint32_t)*reinterpret_cast<const uint16_t*>(at + off); };
      uint32_t codes;
      if constexpr (E == 4) {
        codes = two(w.side == 0 ? L::key_codes(t, dim) : L::value_codes(t, dim / 128, dim % 128 / L::VDims) + dim % L::VDims / 2);
      } else if constexpr (D >= 128) {
        codes = *reinterpret_cast<const uint32_t*>(at + (w.side == 0 ? L::key_codes(t, dim) : L::value_codes(t, dim / 128, dim % 128 / 8)));
      } else {
        codes = w.side == 0 ? *reinterpret_cast<const uint32_t*>(at + L::key_codes(t, dim))
                            : two(L::value_codes(t, 0, 2 * p)) | two(L::value_codes(t, 0, 2 * p + 1)) << 16;
      }
      const float s = FMT == kNv ? __builtin_amdgcn_cvt_pk_f32_fp8((int)sb, false)[0] : e8m0(sb);
      const float gs = FMT == kNv && a.gs[w.side] ? *a.gs[w.side] : 1.0f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const f32x2 x = e == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0)
                        : e == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1)
                        : e == 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
        // code times group scale is exact; one rounding by the scale of all
        out[e] = (T)(x.x * s * gs);
        out[e + 1] = (T)(x.y * s * gs);
      }
    }
    T* dst = static_cast<T*>(a.rows[w.side]) + (t0 + w.token) * a.token[w.side] + w.head * a.head[w.side] + dim;
    __builtin_memcpy(dst, &out, sizeof out);
  }
}

int type_size(int t) { return t == SC_DTYPE_F32 ? 4 : 2; }

template <bool WRITE, typename T>
hipError_t run(RowArgs a, int dim, int fmt, hipStream_t st) {
  // a block has work for four rounds of its threads, unless that leaves compute units idle
  const int per = 2 * a.pool.heads, threads = WRITE ? dim / 16 : dim * (int)sizeof(T) / 16;
  const int full = (4 * kThreads / threads + per - 1) / per, even = (a.tokens + 511) / 512;
  const int n = full < even ? full : even;
  a.block_tokens = n < kMaxTokens ? n : kMaxTokens;
  a.per_magic = (uint32_t)((1ull << 32) / per + 1);      // exact: rows of a block times heads are below 2^32
  const unsigned grid = (unsigned)((a.tokens + a.block_tokens - 1) / a.block_tokens);
  return by_layout(dim, fmt, [&](auto d, auto f) {
    if constexpr (WRITE) hipLaunchKernelGGL((k_kv4_append<T, d(), f()>), dim3(grid), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_kv4_read<T, d(), f()>), dim3(grid), dim3(kThreads), 0, st, a);
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
  if (tokens >= 1 << 24) return fail(SC_E_ARG, "too many tokens for one call");     // a launch has less than 2^32 threads
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
