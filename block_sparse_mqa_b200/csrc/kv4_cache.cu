// hs_kv4_append and hs_kv4_read: rows into the 4-bit paged cache and back.
//
// Quantisation of a group of 32 elements x_i (format: kv4.cuh):
//   s   = the smallest representable scale with 7 s >= max_i |x_i|
//   n_i = 8 + clamp(rint(x_i / s), -7, 7)         value (n_i - 8) s
// A group with a NaN or an infinity gets the NaN scale, so that it reads as
// NaN and is not hidden; a scale past the format's range saturates.
//
// An element is read once and its code written once; what bounds both is the
// issue of the conversions (append) and the look-up's chain of loads.  20147
// rows of 576 in a graph: append 19.9 us (1.5 TB/s), read 8.9 us (3.3 TB/s).
// A block takes 8 consecutive rows, looks up where they live once (32 rows a
// block: 35.2 us for 31.3, append and read of those rows, and 14.9 for 7.4 with
// 1256), and its 8 warps take the groups: four lanes share a group (8 elements,
// 16 bytes of bf16, one word of codes each), eight rows side by side, so that a
// warp reads eight runs of 64 bytes and writes one of 128 (the codes of a group
// of consecutive rows are contiguous).

#include "kv4.cuh"

namespace hs {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;   // of a block
constexpr int kBatch = 3;  // groups of a thread whose loads go together

// A block's rows: where each lives (page -1: nowhere).
struct Rows {
  int page[kRows], slot[kRows];
};

// Row i of the packed rows belongs to sequence s with cu[s] <= i < cu[s+1] and
// is its cached position seq_lens[s] - (cu[s+1] - i).  The block counts the
// sequences that end at or before its first row (one round of loads for up to
// 256 of them, where a search would wait for each of its steps), and each row
// steps on from there.  Rows behind the last sequence are padding (silent); a
// malformed input is recorded.
__device__ __forceinline__ void locate_rows(const Kv4Rows& a, int64_t row0, Rows& sh) {
  int before = 0;
  for (int s0 = 0; s0 < a.num_seqs; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    before += __syncthreads_count(s < a.num_seqs && __ldg(a.cu + s + 1) <= row0);
  }
  if (threadIdx.x < kRows) {
    const int64_t i = row0 + threadIdx.x;
    int page = -1, slot = 0;
    if (i < a.total_tokens && i < __ldg(a.cu + a.num_seqs)) {
      int s = before;
      while (s < a.num_seqs && __ldg(a.cu + s + 1) <= i) ++s;
      const int bos = s < a.num_seqs ? __ldg(a.cu + s) : -1;
      const int eos = s < a.num_seqs ? __ldg(a.cu + s + 1) : -1;
      const int len = s < a.num_seqs ? __ldg(a.seq_lens + s) : 0;
      if (bos < 0 || i < bos || eos > a.total_tokens || len < eos - bos) {
        record_status(a.status, HS_ERR_INVALID_ARG);
      } else {
        const int pos = len - (int)(eos - i);
        slot = pos & ((1 << a.ps_log2) - 1);
        page = kv4::page_of(a.table + (int64_t)s * a.table_stride, a.table_width, a.num_pages, pos,
                            a.ps_log2, a.status);
      }
    }
    sh.page[threadIdx.x] = page;
    sh.slot[threadIdx.x] = slot;
  }
  __syncthreads();
}

template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if (kVec) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int u = 0; u < 8 / kPer; ++u) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + u);
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[u * kPer + j] = to_f32<T>(e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(p[j]);
  }
}

// Groups of the k rows and, behind them, of the v rows.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Rows a, const Kv4Append w) {
  __shared__ Rows sh;
  const int64_t row0 = (int64_t)blockIdx.x * kRows;
  locate_rows(a, row0, sh);
  const int gk = kv4::groups(w.dk), G = gk + kv4::groups(w.dv), ps = 1 << a.ps_log2;
  const int lane = threadIdx.x & 31, part = lane & 3;
  constexpr int kStep = kThreads / 32;
  const int per = ((G + kBatch * kStep - 1) / (kBatch * kStep));  // batches of a row
  for (int it = 0; it < per * (kRows / 8); ++it) {
    const int g0 = (threadIdx.x >> 5) + it % per * kBatch * kStep;
    const int r = (lane >> 2) + 8 * (it / per);
    const int page = sh.page[r], slot = sh.slot[r];
    // the batch's loads before its first store
    float x[kBatch][8];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int gg = g0 + u * kStep;
      if (page < 0 || gg >= G) continue;
      const T* src = gg >= gk ? static_cast<const T*>(w.v) + (row0 + r) * w.v_row_stride + (gg - gk) * 32
                              : static_cast<const T*>(w.k) + (row0 + r) * w.k_row_stride + gg * 32;
      load8<T, kVec>(src + 8 * part, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int gg = g0 + u * kStep;
      if (gg >= G) break;
      const bool is_v = gg >= gk;
      const int g = is_v ? gg - gk : gg, width = is_v ? w.dv : w.dk;
      // the largest magnitude by its bits, where NaN and infinity come on top
      uint32_t top = 0u;
      if (page >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[u][j]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (page < 0) continue;
      uint32_t word = 0x88888888u, byte = 0u;
      if (top >= 0x7f800000u) {
        byte = kv4::kNanScale;
      } else if (top != 0u) {
        const float amax = __uint_as_float(top);
        const float s = kv4::group_scale(amax), inv = __frcp_rn(s);
        byte = kv4::scale_byte(s);
        if (amax > 7.f * s) {  // past the largest scale
#pragma unroll
          for (int j = 0; j < 8; ++j) x[u][j] = fminf(fmaxf(x[u][j], -7.f * s), 7.f * s);
        }
        word = kv4::code_word(x[u], s, inv);
      }
      uint8_t* pg = static_cast<uint8_t*>(is_v ? w.v_cache : w.k_cache) +
                    (int64_t)page * kv4::page_bytes(width, ps);
      *reinterpret_cast<uint32_t*>(pg + kv4::code_off(g, slot, ps) + 4 * part) = word;
      if (part == 0) pg[kv4::scale_off(g, slot, ps, kv4::groups(width))] = (uint8_t)byte;
    }
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4Rows a, const uint8_t* __restrict__ cache, int width, T* out,
                int64_t out_row_stride) {
  __shared__ Rows sh;
  const int64_t row0 = (int64_t)blockIdx.x * kRows;
  locate_rows(a, row0, sh);
  const int G = kv4::groups(width), ps = 1 << a.ps_log2;
  const int lane = threadIdx.x & 31, part = lane & 3;
  constexpr int kStep = kThreads / 32;
  const int per = ((G + kBatch * kStep - 1) / (kBatch * kStep));  // batches of a row
  for (int it = 0; it < per * (kRows / 8); ++it) {
    const int g0 = (threadIdx.x >> 5) + it % per * kBatch * kStep;
    const int r = (lane >> 2) + 8 * (it / per);
    const int page = sh.page[r], slot = sh.slot[r];
    if (page < 0) continue;
    const uint8_t* pg = cache + (int64_t)page * kv4::page_bytes(width, ps);
    uint32_t word[kBatch], byte[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = g0 + u * kStep;
      if (g >= G) continue;
      word[u] = __ldg(reinterpret_cast<const uint32_t*>(pg + kv4::code_off(g, slot, ps) + 4 * part));
      byte[u] = __ldg(pg + kv4::scale_off(g, slot, ps, G));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int g = g0 + u * kStep;
      if (g >= G) break;
      const float s = kv4::scale_value(byte[u]);
      alignas(16) T v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int n = (int)((word[u] >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - 8;
        v[e] = from_f32<T>((float)n * s);  // exact in bf16 and fp32
      }
      T* dst = out + (row0 + r) * out_row_stride + g * 32 + 8 * part;
      if (kVec) {
#pragma unroll
        for (int q = 0; q < (int)(8 * sizeof(T) / 16); ++q)
          reinterpret_cast<uint4*>(dst)[q] = reinterpret_cast<const uint4*>(v)[q];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = v[e];
      }
    }
  }
}

unsigned grid_for(int64_t rows) { return (unsigned)((rows + kRows - 1) / kRows); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T>
cudaError_t append_typed(const Kv4Rows& a, const Kv4Append& w, cudaStream_t s) {
  constexpr int kPer = 16 / sizeof(T);
  const bool vec = aligned16(w.k) && w.k_row_stride % kPer == 0 &&
                   (w.dv == 0 || (aligned16(w.v) && w.v_row_stride % kPer == 0));
  auto kern = vec ? kv4_append_kernel<T, true> : kv4_append_kernel<T, false>;
  kern<<<grid_for(a.total_tokens), kThreads, 0, s>>>(a, w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read_typed(const Kv4Rows& a, const void* cache, int width, void* out, int64_t ors,
                       cudaStream_t s) {
  const bool vec = aligned16(out) && ors % (16 / (int)sizeof(T)) == 0;
  const uint8_t* c = static_cast<const uint8_t*>(cache);
  T* o = static_cast<T*>(out);
  auto kern = vec ? kv4_read_kernel<T, true> : kv4_read_kernel<T, false>;
  kern<<<grid_for(a.total_tokens), kThreads, 0, s>>>(a, c, width, o, ors);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Rows& a, const Kv4Append& w, cudaStream_t s) {
  return w.dtype == HS_BF16 ? append_typed<__nv_bfloat16>(a, w, s) : append_typed<float>(a, w, s);
}

cudaError_t launch_kv4_read(const Kv4Rows& a, const void* cache, int width, void* out,
                            int64_t out_row_stride, hs_dtype dtype, cudaStream_t s) {
  return dtype == HS_BF16 ? read_typed<__nv_bfloat16>(a, cache, width, out, out_row_stride, s)
                          : read_typed<float>(a, cache, width, out, out_row_stride, s);
}

}  // namespace hs
