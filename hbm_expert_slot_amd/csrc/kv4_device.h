// Layout of the 4-bit key/value cache, and what its kernels share.
//
// A page holds 64 tokens.  Of every page, each head has its keys and its values
// side by side: 64 D / 2 bytes of codes, then 64 D / G group scales.  The order
// inside is the one in which the attention kernel's lanes take them, so that a
// wavefront fetches a page straight into the operands of its matrix
// instructions, by loads of 16 bytes per lane that cover whole kilobytes, with
// no transposition through LDS:
//
//   keys     codes of token t: D/2 contiguous bytes, tokens one after the other.
//            scales: for lane (r = t % 16, g) those of its share of the tokens r,
//            16 + r, 32 + r, 48 + r side by side (one load for four tiles).
//   values   four tokens side by side, so that a lane gets four tokens of its own
//            few dimensions: [t/4][chunk of 128 dims][16 lanes][t % 4][codes].
//            scales: [g][group][16 tokens of that g].
#pragma once

#include "fp4_device.h"
#include "internal.h"

namespace sc {
namespace kv4 {

using namespace fp4;

constexpr int kPage = SC_KV4_PAGE;

template <int D, int FMT>
struct Layout {
  static constexpr int G = FMT == kNv ? 16 : 32;
  static constexpr int C = D >= 128 ? D / 128 : 1;       // chunks of (up to) 128 dimensions
  static constexpr int NS = D / G;                       // scales per token
  static constexpr int kCodes = kPage * D / 2, kScales = kPage * NS, kSide = kCodes + kScales, kHead = 2 * kSide;
  static constexpr int LaneDims = D >= 128 ? 32 : 16;    // a lane's share of a key per chunk
  static constexpr int VDims = D >= 128 ? 8 : 4;         // a lane's dimensions of a value per chunk
  // lanes (of the four along a key) with scales of their own, and their scales per token
  static constexpr int SL = LaneDims >= G ? 4 : 2, SP = NS / SL;

  // offsets inside a side
  static __device__ __forceinline__ uint32_t key_codes(int t, int dim) { return (uint32_t)(t * (D / 2) + dim / 2); }
  static __device__ __forceinline__ uint32_t key_scale(int t, int s) {
    constexpr int W = 128 / G;                           // scales of a chunk
    const int c = D >= 128 ? s / W : 0, in = D >= 128 ? s % W : s;
    constexpr int E = SP / C;                            // a lane's scales per chunk
    const int gl = in / E, e = c * E + in % E;
    return (uint32_t)(kCodes + (((t % 16) * SL + gl) * 4 + t / 16) * SP + e);
  }
  // first of the codes of VDims dimensions of lane n in chunk c
  static __device__ __forceinline__ uint32_t value_codes(int t, int c, int n) {
    constexpr int B = VDims / 2;
    return (uint32_t)((((t / 4) * C + c) * 16 + n) * 4 * B + (t % 4) * B);
  }
  // tokens of g: those with t / 4 % 4 == g, ascending
  static __device__ __forceinline__ uint32_t value_scale(int t, int s) {
    return (uint32_t)(kCodes + ((t / 4 % 4) * NS + s) * 16 + t / 16 * 4 + t % 4);
  }
};

// A batch of sequences as the kernels see it.
struct Seqs {
  const int32_t* table;      // [n][ld]
  const int32_t* lens;       // [n]
  int64_t ld;
  int32_t n, width;
};

struct Pool {
  uint8_t* pages;
  float* weights;
  int32_t* positions;
  int32_t n_pages, heads;
};

// The page of a place, or -1 where the table has none.
__device__ __forceinline__ int page_at(const Pool& p, const Seqs& s, int b, int index) {
  if (index < 0 || index >= s.width) return -1;
  const int page = s.table[b * s.ld + index];
  return page >= 0 && page < p.n_pages ? page : -1;
}

// A sequence's length; -1 where it is none that the table can hold.
__device__ __forceinline__ int length_of(const Seqs& s, int b) {
  const int n = s.lens[b];
  return n >= 0 && n <= s.width * kPage ? n : -1;
}

sc_status check_cache(const sc_kv4_cache* c);
sc_status check_seqs(const sc_kv4_seqs* s);
inline Seqs seqs_of(const sc_kv4_seqs* s) { return Seqs{s->d_table, s->d_lens, s->ld_table, s->n_seqs, s->width}; }
inline Pool pool_of(const sc_kv4_cache* c) {
  return Pool{static_cast<uint8_t*>(c->d_pages), c->d_weights, c->d_positions, c->n_pages, c->kv_heads};
}

// f<D, FMT>() for the cache's head size and format
template <typename F>
auto by_layout(int dim, int fmt, F&& f) {
  if (fmt == SC_FP4_NV) {
    if (dim == 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, kNv>{});
    if (dim == 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, kNv>{});
    return f(std::integral_constant<int, 256>{}, std::integral_constant<int, kNv>{});
  }
  if (dim == 64) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, kMx>{});
  if (dim == 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, kMx>{});
  return f(std::integral_constant<int, 256>{}, std::integral_constant<int, kMx>{});
}

}  // namespace kv4
}  // namespace sc
