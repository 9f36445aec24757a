// hs_kv4_mqa_decode on CUDA cores (fp32 arithmetic): fp32 queries and widths
// the tensor-core kernel does not take.
//
// With s_j = scale <q[b,h], k_j> over the attended cached positions j,
//   lse[b,h] = log(exp(sink_h) + sum_j exp(s_j)),  out[b,h] = sum_j exp(s_j - lse) v_j.
// One CTA per (split of the key list, 4 heads, sequence) walks its keys in
// tiles of 32 rows staged in shared memory as fp32, with a running maximum and
// sum per head; a second kernel joins the splits in their order and adds the
// sink.  A lone split is finished by its CTA, without a workspace, so that many
// sequences need none (partials of every sequence would take 9 GB for 70000 with
// 64 heads, Dv 512).  Every sum has a fixed order.

#include <math.h>

#include "kv4.cuh"

namespace hs {
namespace {

constexpr int kThreads = 256;
constexpr int kHB = 4;    // heads per CTA
constexpr int kKT = 32;   // keys per tile
constexpr int kMaxCols = 4;  // value columns per thread (dv <= 1024)

// Splits of each sequence's keys: enough CTAs for two per SM, at least 64 keys
// each.  A function of the sizes alone (the workspace depends on it).
int num_splits(int num_seqs, int num_heads, int max_keys) {
  const int64_t ctas = (int64_t)num_seqs * ((num_heads + kHB - 1) / kHB);
  int64_t n = (2 * 148 + ctas - 1) / ctas;
  const int64_t most = ((int64_t)max_keys + 63) / 64;
  if (n > most) n = most;
  return n < 1 ? 1 : n > 256 ? 256 : (int)n;
}

// Rows x0 .. x0 + cnt - 1 of the key list, `width` columns of `cache`, as fp32
// rows of stride `ld` in shared memory; a row without a page is zero.
__device__ __forceinline__ void stage_rows(const Kv4Decode& a, const uint8_t* cache, int width,
                                           int plane_width, const int* pages, const int* slots,
                                           int cnt, float* buf, int ld) {
  const int G = kv4::groups(width), ps = 1 << a.ps_log2;
  const int64_t pb = kv4::page_bytes(plane_width, ps);
  for (int e = threadIdx.x; e < cnt * G; e += kThreads) {
    const int r = e % cnt, g = e / cnt;
    float* dst = buf + r * ld + g * 32;
    if (pages[r] < 0) {
      for (int j = 0; j < 32; ++j) dst[j] = 0.f;
      continue;
    }
    const uint8_t* pg = cache + (int64_t)pages[r] * pb;
    const uint4 c = *reinterpret_cast<const uint4*>(pg + kv4::code_off(g, slots[r], ps));
    const float s =
        kv4::scale_value(pg[kv4::scale_off(g, slots[r], ps, kv4::groups(plane_width))]);
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int el = j & 7;
      const int n = (int)((word[j >> 3] >> (4 * (el >> 1) + 16 * (el & 1))) & 15u) - 8;
      dst[j] = (float)n * s;
    }
  }
}

// Sequence length, or 0 (recorded) where it is out of range.
__device__ __forceinline__ int seq_len(const Kv4Decode& a, int b) {
  const int len = __ldg(a.seq_lens + b);
  if (len < 0 || len > a.max_seqlen) {
    record_status(a.status, HS_ERR_INVALID_ARG);
    return 0;
  }
  return len;
}

// 1 / den and the lse, for a sum den of exponentials over exp(Ms).
__device__ __forceinline__ float2 inv_and_lse(float den, float Ms) {
  return make_float2(den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den),  // NaN stays NaN
                     den == 0.f ? -INFINITY : Ms + logf(den));
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
simt_kv4_decode_kernel(const Kv4Decode a, int nsplit, float* part_o, float2* part_ml) {
  extern __shared__ float sm[];
  const int split = blockIdx.x, h0 = blockIdx.y * kHB, tid = threadIdx.x;
  const int dk = a.dk, dv = a.dv, H = a.num_heads;
  const int hn = min(kHB, H - h0);
  const int ldk = dk + 1, ldv = dv + 1;
  float* qs = sm;                                   // [kHB][dk]
  float* buf = qs + kHB * dk;                       // [kKT][max(dk, dv) + 1]
  float* sc = buf + kKT * (max(dk, dv) + 1);        // [kHB][kKT] logits, then exponentials
  float* mrun = sc + kHB * kKT;                     // [kHB]
  float* lrun = mrun + kHB;                         // [kHB]
  float* alpha = lrun + kHB;                        // [kHB]
  int* pages = reinterpret_cast<int*>(alpha + kHB);  // [kKT]
  int* slots = pages + kKT;                         // [kKT]
  for (int b = blockIdx.z; b < a.num_seqs; b += gridDim.z) {
    const kv4::KeyList kl = kv4::key_list(seq_len(a, b), a.window, a.first);
    const int per = (kl.n + nsplit - 1) / nsplit;
    const int x0 = min(kl.n, split * per), x1 = min(kl.n, x0 + per);
    __syncthreads();
    for (int e = tid; e < hn * dk; e += kThreads) {
      const int h = e / dk, d = e - h * dk;
      qs[e] = to_f32<T>(static_cast<const T*>(
          a.q)[(int64_t)b * a.q_row_stride + (int64_t)(h0 + h) * a.q_head_stride + d]);
    }
    if (tid < kHB) {
      mrun[tid] = -INFINITY;
      lrun[tid] = 0.f;
    }
    float acc[kHB][kMaxCols];
#pragma unroll
    for (int h = 0; h < kHB; ++h)
#pragma unroll
      for (int c = 0; c < kMaxCols; ++c) acc[h][c] = 0.f;
    const uint8_t* vc = a.v_cache ? a.v_cache : a.k_cache;
    const int vplane = a.v_cache ? dv : dk;
    for (int x = x0; x < x1; x += kKT) {
      const int cnt = min(kKT, x1 - x);
      __syncthreads();
      if (tid < cnt) {
        const int pos = kl.pos(x + tid);
        pages[tid] = kv4::page_of(a.table + (int64_t)b * a.table_stride, a.table_width,
                                  a.num_pages, pos, a.ps_log2, a.status);
        slots[tid] = pos & ((1 << a.ps_log2) - 1);
      }
      __syncthreads();
      stage_rows(a, a.k_cache, dk, dk, pages, slots, cnt, buf, ldk);
      __syncthreads();
      {  // two threads per (head, key) dot product
        const int i = tid >> 1, h = i / kKT, j = i - h * kKT;
        float s = 0.f;
        if (h < hn && j < cnt) {
          const float* qr = qs + h * dk;
          const float* kr = buf + j * ldk;
          for (int d = tid & 1; d < dk; d += 2) s = fmaf(qr[d], kr[d], s);
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        if ((tid & 1) == 0) sc[i] = h < hn && j < cnt ? s * a.scale : -INFINITY;
      }
      __syncthreads();
      const int warp = tid >> 5, lane = tid & 31;
      if (warp < hn) {
        const float s = sc[warp * kKT + lane];
        const float mo = mrun[warp], mn = fmaxf(mo, warp_max(s));
        const float ms = mn == -INFINITY ? 0.f : mn;  // every logit so far is -inf
        const float e = expf(s - ms);
        const float l = warp_sum(e);
        sc[warp * kKT + lane] = e;
        __syncwarp();
        if (lane == 0) {
          const float al = expf(mo - ms);
          alpha[warp] = al;
          mrun[warp] = mn;
          lrun[warp] = lrun[warp] * al + l;
        }
      }
      __syncthreads();
      stage_rows(a, vc, dv, vplane, pages, slots, cnt, buf, ldv);
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kMaxCols; ++c) {
        const int d = tid + c * kThreads;
        if (d >= dv) continue;
#pragma unroll
        for (int h = 0; h < kHB; ++h) {
          if (h >= hn) continue;
          float o = acc[h][c] * alpha[h];
          for (int j = 0; j < cnt; ++j) o = fmaf(sc[h * kKT + j], buf[j * ldv + d], o);
          acc[h][c] = o;
        }
      }
    }
    __syncthreads();
    for (int h = 0; h < hn; ++h) {
      const int64_t slot = ((int64_t)b * H + h0 + h) * nsplit + split;
      // a lone split: what the join below would do with it, rounded alike
      float w = 1.f, inv = 1.f;
      if (nsplit == 1) {
        const float sk = a.sink ? __ldg(a.sink + h0 + h) : -INFINITY;
        const float M = fmaxf(sk, mrun[h]), Ms = M == -INFINITY ? 0.f : M;
        w = expf(mrun[h] - Ms);
        const float2 r = inv_and_lse(__fmul_rn(lrun[h], w) + expf(sk - Ms), Ms);
        inv = r.x;
        if (tid == 0) a.lse[slot] = r.y;
      }
#pragma unroll
      for (int c = 0; c < kMaxCols; ++c) {
        const int d = tid + c * kThreads;
        if (d < dv) {
          float v = 0.f;
#pragma unroll
          for (int hh = 0; hh < kHB; ++hh)
            if (hh == h) v = acc[hh][c];
          if (nsplit == 1)
            static_cast<T*>(a.out)[slot * dv + d] = from_f32<T>(__fmul_rn(v, w) * inv);
          else
            part_o[slot * dv + d] = v;
        }
      }
      if (nsplit > 1 && tid == 0) part_ml[slot] = make_float2(mrun[h], lrun[h]);
    }
  }
}

// Joins the splits of one (sequence, head) and the sink.
template <typename T>
__global__ void __launch_bounds__(kThreads)
simt_kv4_join_kernel(const Kv4Decode a, int nsplit, const float* part_o, const float2* part_ml) {
  const int64_t bh = blockIdx.x;  // b * H + h
  const int h = (int)(bh % a.num_heads);
  const float sk = a.sink ? __ldg(a.sink + h) : -INFINITY;
  float M = sk;
  for (int i = 0; i < nsplit; ++i) M = fmaxf(M, part_ml[bh * nsplit + i].x);
  float den = 0.f;
  const float Ms = M == -INFINITY ? 0.f : M;
  for (int i = 0; i < nsplit; ++i) {
    const float2 ml = part_ml[bh * nsplit + i];
    den += ml.y * expf(ml.x - Ms);
  }
  den += expf(sk - Ms);
  const float2 r = inv_and_lse(den, Ms);
  for (int d = threadIdx.x; d < a.dv; d += kThreads) {
    float o = 0.f;
    for (int i = 0; i < nsplit; ++i)
      o = fmaf(part_o[(bh * nsplit + i) * a.dv + d], expf(part_ml[bh * nsplit + i].x - Ms), o);
    static_cast<T*>(a.out)[bh * a.dv + d] = from_f32<T>(o * r.x);
  }
  if (threadIdx.x == 0) a.lse[bh] = r.y;
}

size_t smem_bytes(int dk, int dv) {
  return sizeof(float) * ((size_t)kHB * dk + (size_t)kKT * ((dk > dv ? dk : dv) + 1) +
                          (size_t)kHB * kKT + 3 * kHB + 2 * kKT);
}

template <typename T>
cudaError_t launch_typed(const Kv4Decode& a, cudaStream_t s) {
  const int nsplit = num_splits(a.num_seqs, a.num_heads, a.max_seqlen);
  const int64_t slots = (int64_t)a.num_seqs * a.num_heads * nsplit;
  float2* ml = static_cast<float2*>(a.workspace);
  float* po = reinterpret_cast<float*>(ml + slots);
  auto kern = simt_kv4_decode_kernel<T>;
  const size_t bytes = smem_bytes(a.dk, a.dv);
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(nsplit, (a.num_heads + kHB - 1) / kHB, a.num_seqs < 65535 ? a.num_seqs : 65535);
  kern<<<grid, kThreads, bytes, s>>>(a, nsplit, po, ml);
  e = cudaGetLastError();
  if (e != cudaSuccess || nsplit == 1) return e;
  simt_kv4_join_kernel<T><<<(unsigned)((int64_t)a.num_seqs * a.num_heads), kThreads, 0, s>>>(
      a, nsplit, po, ml);
  return cudaGetLastError();
}

}  // namespace

size_t simt_kv4_decode_workspace(int num_seqs, int num_heads, int max_seqlen, int dv) {
  const int nsplit = num_splits(num_seqs, num_heads, max_seqlen);
  if (nsplit == 1) return 0;
  return (size_t)num_seqs * num_heads * nsplit * (sizeof(float2) + (size_t)dv * sizeof(float));
}

cudaError_t launch_simt_kv4_decode(const Kv4Decode& a, cudaStream_t s) {
  return a.dtype == HS_BF16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace hs
