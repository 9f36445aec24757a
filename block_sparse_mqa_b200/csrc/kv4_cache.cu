// hs_kv4_append and hs_kv4_read: rows into the 4-bit paged cache and back.
//
// Quantisation of a group of 32 elements x_i (format: kv4.cuh):
//   s   = the smallest representable scale with 7 s >= max_i |x_i|
//   n_i = 8 + clamp(rint(x_i / s), -7, 7)         value (n_i - 8) s
// A group with a NaN or an infinity gets the NaN scale, so that it reads as
// NaN and is not hidden; a scale past the format's range saturates.
//
// Both are bound by memory: one thread owns one group of one row, reads its 64
// bytes (bf16) or 16 bytes of codes once and writes the other form once.
// Neighbouring threads take neighbouring groups of a row, whose elements are
// contiguous.

#include "kv4.cuh"

namespace hs {
namespace {

constexpr int kThreads = 256;

// Where row i of the packed rows lives: sequence s with cu[s] <= i < cu[s+1],
// cached position seq_lens[s] - (cu[s+1] - i).  False: a padding row behind
// the last sequence (silent) or a malformed input (recorded).
__device__ __forceinline__ bool locate(const Kv4Rows& a, int64_t i, int& page, int& slot) {
  if (i >= __ldg(a.cu + a.num_seqs)) return false;  // behind the last sequence
  int lo = 0, hi = a.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid) <= i) lo = mid; else hi = mid;
  }
  const int bos = __ldg(a.cu + lo), eos = __ldg(a.cu + lo + 1);
  const int len = __ldg(a.seq_lens + lo);
  if (bos < 0 || i < bos || i >= eos || eos > a.total_tokens || len < eos - bos) {
    record_status(a.status, HS_ERR_INVALID_ARG);
    return false;
  }
  const int pos = len - (int)(eos - i);
  slot = pos & ((1 << a.ps_log2) - 1);
  page = kv4::page_of(a.table + (int64_t)lo * a.table_stride, a.table_width, a.num_pages, pos,
                      a.ps_log2, a.status);
  return page >= 0;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load_group(const T* p, float (&x)[32]) {
  if (kVec) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int u = 0; u < 32 / kPer; ++u) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + u);
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[u * kPer + j] = to_f32<T>(e[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = to_f32<T>(p[j]);
  }
}

// Groups of the k rows and, behind them, of the v rows: item = row * (Gk + Gv) + group.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4Rows a, const Kv4Append w) {
  const int gk = kv4::groups(w.dk), gv = kv4::groups(w.dv), G = gk + gv;
  const int ps = 1 << a.ps_log2;
  const int64_t total = (int64_t)a.total_tokens * G;
  for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < total;
       it += (int64_t)gridDim.x * kThreads) {
    const int64_t i = it / G;
    const int gg = (int)(it - i * G);
    int page, slot;
    if (!locate(a, i, page, slot)) continue;
    const bool is_v = gg >= gk;
    const int g = is_v ? gg - gk : gg;
    const T* src = is_v ? static_cast<const T*>(w.v) + i * w.v_row_stride
                        : static_cast<const T*>(w.k) + i * w.k_row_stride;
    float x[32];
    load_group<T, kVec>(src + g * 32, x);
    float amax = 0.f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      amax = fmaxf(amax, fabsf(x[j]));
      finite = finite && fabsf(x[j]) <= FLT_MAX;
    }
    uint32_t code[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
    uint32_t byte = 0;
    if (!finite) {
      byte = kv4::kNanScale;
    } else if (amax > 0.f) {
      const float s = kv4::group_scale(amax);
      byte = kv4::scale_byte(s);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          word |= kv4::code_of(x[8 * q + e], s) << (4 * (e >> 1) + 16 * (e & 1));
        code[q] = word;
      }
    }
    uint8_t* pg = static_cast<uint8_t*>(is_v ? w.v_cache : w.k_cache) +
                  (int64_t)page * kv4::page_bytes(is_v ? w.dv : w.dk, ps);
    *reinterpret_cast<uint4*>(pg + kv4::code_off(g, slot, ps)) =
        make_uint4(code[0], code[1], code[2], code[3]);
    pg[kv4::scale_off(g, slot, ps, is_v ? gv : gk)] = (uint8_t)byte;
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
kv4_read_kernel(const Kv4Rows a, const uint8_t* __restrict__ cache, int width, T* out,
                int64_t out_row_stride) {
  const int G = kv4::groups(width), ps = 1 << a.ps_log2;
  const int64_t total = (int64_t)a.total_tokens * G;
  for (int64_t it = (int64_t)blockIdx.x * kThreads + threadIdx.x; it < total;
       it += (int64_t)gridDim.x * kThreads) {
    const int64_t i = it / G;
    const int g = (int)(it - i * G);
    int page, slot;
    if (!locate(a, i, page, slot)) continue;
    const uint8_t* pg = cache + (int64_t)page * kv4::page_bytes(width, ps);
    const uint4 c = *reinterpret_cast<const uint4*>(pg + kv4::code_off(g, slot, ps));
    const float s = kv4::scale_value(pg[kv4::scale_off(g, slot, ps, G)]);
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
    T v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int e = j & 7;
      const int n = (int)((word[j >> 3] >> (4 * (e >> 1) + 16 * (e & 1))) & 15u) - 8;
      v[j] = from_f32<T>((float)n * s);  // exact in bf16 and fp32
    }
    T* dst = out + i * out_row_stride + g * 32;
    if (kVec) {
#pragma unroll
      for (int u = 0; u < (int)(32 * sizeof(T) / 16); ++u)
        reinterpret_cast<uint4*>(dst)[u] = reinterpret_cast<const uint4*>(v)[u];
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) dst[j] = v[j];
    }
  }
}

int grid_for(int64_t items) {
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  return (int)(blocks < 148 * 16 ? blocks : 148 * 16);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T>
cudaError_t append_typed(const Kv4Rows& a, const Kv4Append& w, cudaStream_t s) {
  const int64_t items = (int64_t)a.total_tokens * (kv4::groups(w.dk) + kv4::groups(w.dv));
  constexpr int kPer = 16 / sizeof(T);
  const bool vec = aligned16(w.k) && w.k_row_stride % kPer == 0 &&
                   (w.dv == 0 || (aligned16(w.v) && w.v_row_stride % kPer == 0));
  if (vec) kv4_append_kernel<T, true><<<grid_for(items), kThreads, 0, s>>>(a, w);
  else kv4_append_kernel<T, false><<<grid_for(items), kThreads, 0, s>>>(a, w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t read_typed(const Kv4Rows& a, const void* cache, int width, void* out, int64_t ors,
                       cudaStream_t s) {
  const int64_t items = (int64_t)a.total_tokens * kv4::groups(width);
  const bool vec = aligned16(out) && ors % (16 / (int)sizeof(T)) == 0;
  const uint8_t* c = static_cast<const uint8_t*>(cache);
  T* o = static_cast<T*>(out);
  if (vec) kv4_read_kernel<T, true><<<grid_for(items), kThreads, 0, s>>>(a, c, width, o, ors);
  else kv4_read_kernel<T, false><<<grid_for(items), kThreads, 0, s>>>(a, c, width, o, ors);
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
