// Shared by the tensor-core kernels of the window attention with visible first
// tokens: which tokens a pair of CTAs takes, the slots of their keys, and the
// loads of key rows.
#pragma once

#include <algorithm>

#include "hs_device.cuh"
#include "hs_internal.h"
#include "tc_host.h"
#include "tc_pair.cuh"

namespace hs {
namespace first {

constexpr int kH = 64;
constexpr int kMaxQC = 9;            // Dk <= 576
constexpr int kQChunk = kH * 128;    // 64 heads x 64 columns bf16
constexpr int kPPanel = kH * 128;    // 64 rows x 64 keys bf16

struct Docs {
  const int32_t* cu;
  int num_docs, T, max_seqlen;
  int window, first;
};

__device__ __forceinline__ uint32_t low_bits(int n) {  // the lowest n, n >= 1
  return n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// Bits lo .. hi (clipped to 0 .. 31).
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
  if (hi < 0 || lo > 31 || lo > hi) return 0u;
  return (lo <= 0 ? 0xffffffffu : 0xffffffffu << lo) & low_bits(hi + 1);
}

// Slots a token sees: lo .. hi of the window's and f0 .. f0 + nf - 1.
struct Mask {
  int lo, hi, f0, nf;
  // of the 32 slots from s
  __device__ __forceinline__ uint32_t bits(int s) const {
    return range_bits(lo - s, hi - s) | range_bits(f0 - s, f0 + nf - 1 - s);
  }
};

// One pass of a pair: tokens t0 and t0 + 1 of one document, or a single token
// (mode 0 or 1: which CTA's) where its neighbour is in another document.
// Key slots: the window's keys from wlo in slots 0 .. nw - 1, then from nwp (nw
// up to a multiple of 16) the nf first tokens that lie before wlo.
struct Pass {
  int t0, mode;  // mode 2: both
  int bos, wlo, nw, nwp, nf, ntile;
  __device__ __forceinline__ int token(int rank) const { return mode == 2 ? t0 + rank : t0; }
  __device__ __forceinline__ bool active(int rank) const { return mode == 2 || mode == rank; }
  __device__ __forceinline__ int keys(int tile) const {  // a multiple of 32
    const int left = nwp + nf - 256 * tile;
    return left >= 256 ? 256 : (left + 31) & ~31;
  }
  __device__ __forceinline__ Mask mask(int rank, int window, int first) const {
    const int t = token(rank);
    // wlo is t0's; t0 + 1's own window may begin one key later
    const int own = max(bos, t - window + 1);
    return {wlo - bos < first ? 0 : own - wlo, t - wlo, nwp, nf};
  }
  // First row of the 16 slots from s (a multiple of 16).
  __device__ __forceinline__ int row(int s) const {
    return s < nwp ? wlo + s : s < nwp + nf ? bos + (s - nwp) : bos;
  }
};

// The passes of one pair, in order; every role walks them alike.
struct Walk {
  const Docs& d;
  int pair, step, half;  // half 1: the second token of a split pair is next
  __device__ __forceinline__ Walk(const Docs& docs, int first_pair, int pairs)
      : d(docs), pair(first_pair), step(pairs), half(0) {}
  __device__ __forceinline__ bool next(Pass& p, int* status) {
    return next(p, status, [](int) {});
  }
  // bad(t): for a token in no (valid) document, which no pass has.
  template <typename Bad>
  __device__ __forceinline__ bool next(Pass& p, int* status, Bad bad) {
    while (2 * pair + half < d.T) {
      const int t = 2 * pair + half;
      int bos, eos;
      const bool ok = find_doc(d.cu, d.num_docs, d.T, d.max_seqlen, t, bos, eos, status);
      const bool both = half == 0 && ok && t + 1 < eos;
      p.t0 = t;
      p.mode = both ? 2 : half;
      if (both || half == 1) {
        half = 0;
        pair += step;
      } else {
        half = 1;
      }
      if (!ok) {
        bad(t);
        continue;
      }
      p.bos = bos;
      p.wlo = max(bos, t - d.window + 1);
      p.nw = t + (both ? 1 : 0) - p.wlo + 1;
      p.nwp = (p.nw + 15) & ~15;
      p.nf = min(d.first, p.wlo - bos);
      if (p.nf == 0) p.nwp = p.nw;
      p.ntile = (p.nwp + p.nf + 255) / 256;
      return true;
    }
    return false;
  }
};

// `rows` (a multiple of 16) key rows of slots s0 .., `panels` panels of 64
// columns from col, `pitch` bytes apart; a row's 128 bytes are swizzled.
// One box where 128 rows are consecutive keys, else boxes of 16 rows spread
// over the lanes.
__device__ __forceinline__ void load_rows(const Pass& ps, const CUtensorMap* big,
                                          const CUtensorMap* small, uint8_t* dst, uint32_t bar,
                                          int s0, int rows, int col, int lane, int panels,
                                          int pitch) {
  if (rows == 128 && s0 + 128 <= ps.nwp) {
    if (lane < panels)
      tc::tma_pair_2d(dst + lane * pitch, big, bar, col + 64 * lane, ps.wlo + s0);
  } else {
    const int boxes = rows / 16;
    for (int e = lane; e < boxes * panels; e += 32) {
      const int pn = e / boxes, bx = e - pn * boxes;
      tc::tma_pair_2d(dst + pn * pitch + bx * 2048, small, bar, col + 64 * pn,
                      ps.row(s0 + 16 * bx));
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------- host
inline Docs docs_of(const Problem& p, int window, int first) {
  return {p.cu_seqlens, p.num_docs, p.total_tokens, p.max_seqlen, window, first};
}
inline bool row_map(CUtensorMap* m, const void* base, int width, int rows, int64_t stride, int box) {
  const uint64_t dims[2] = {(uint64_t)width, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)stride * 2};
  const uint32_t b[2] = {64, (uint32_t)box};
  return tc::encode_bf16_map(m, base, 2, dims, strides, b);
}
inline bool head_map(CUtensorMap* m, const void* base, int width, int rows, int64_t row_stride,
                     int64_t head_stride) {
  const uint64_t dims[3] = {(uint64_t)width, (uint64_t)kH, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)head_stride * 2, (uint64_t)row_stride * 2};
  const uint32_t b[3] = {64, (uint32_t)kH, 1};
  return tc::encode_bf16_map(m, base, 3, dims, strides, b);
}
// CTAs of a persistent grid of pairs.
inline int pair_grid(int tokens) {
  const int pairs = (tokens + 1) / 2, most = tc::sm_count() / 2;
  return 2 * std::max(1, std::min(pairs, most));
}

}  // namespace first
}  // namespace hs
