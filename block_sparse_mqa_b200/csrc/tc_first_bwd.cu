// hs_swa_first_mqa_bwd on tcgen05 tensor cores (bf16 in, fp32 accumulate), 64
// query heads over one KV head, pairs of CTAs (tc_pair.cuh).
//
// With S_t the key set of tc_first_fwd.cu, p = exp(scale <q, k_j> - lse) and
// ds = p (<dout, v_j> - delta), delta = <dout, out>:
//   dq[t,h] = scale sum_j ds k_j,   dk[j] = scale sum_{t,h} ds q[t,h],
//   dv[j] = sum_{t,h} p dout[t,h].
//
// What bounds it: 2 * 64 * |S_t| (3 Dk + 2 Dv) operations per token, and the
// operands' way from L2.  dq wants a token's heads as rows, dk and dv want a
// key's (token, head) pairs as the summed dimension; p and ds serve both, so
// they are computed once, in the query-major pass, and written as bf16 (the
// rounding the products need anyway) into a band in the workspace:
//   band[t][h][c] is key base(t) + c, base(t) = (t & ~7) - Wp, c < bw
// (Wp: window - 1 up to a multiple of 8; bw: Wp + 8 up to one of 16), and behind
// it the first tokens' columns, key bos + c - bw.  Everything outside a token's
// key set is written as 0, and so is the whole row of a token in no valid document:
// the key pass takes every token of a chunk.
// The key-major pass is then a plain product over the band: a tile's 256 keys
// are columns base-shifted per token, which a TMA box fetches for any token;
// columns left or right of the band read as 0, so documents and window edges
// need no case of their own.
//   pass A  per pair of tokens, tiles of 128 keys: S = Q K^T, dP = dO V^T,
//           P and dS to the band, dQ += dS K                   (M = 128); where
//           the keys are many, delta of the next pair beside it
//   pass B  per (tok tokens, up to 256 of the keys that their windows reach,
//           512 columns of dk or dv): partial
//           dV^T += dO^T P or dK^T += Q^T dS                   (M = 256, N = 256)
//           and the same per (tok tokens of a document, its first tokens).
//           Items go by their tokens, so that the ones running together read
//           the same q and dout from L2.
//   reduce  adds a key's partial sums in order, scales, rounds once
// Results are deterministic.  All waits are bounded (HS_ERR_TIMEOUT).
//
// Measured (Dk 576 / Dv 512, 4096 tokens, window 512 + 4 first, in a graph, full
// clock): the whole backward 1.08 ms, 648 TFLOP/s, 0.39 of a cuBLAS matmul's rate
// (1.27 ms in a long run under the power cap, 0.39 of that rate too; pass A
// with delta 0.61 ms, pass B 0.41 ms, reduction 33 us); the passes of
// tc_bwd_dq.cu and tc_bwd_dkdv.cu, which recompute P and dS for dk and dv and
// take one token per CTA, need 3.81 ms for the same and less workspace (333
// tokens, window 64 + 5: 321 us for 67).
// Pass A is bound by its S and dP MMAs (N = 128: ~91 cycles each from one issuing
// warp) and its loads, pass B by q, dout and the band out of L2 and DRAM.

#include <math.h>

#include "hs_device.cuh"
#include "hs_internal.h"
#include "tc_first.cuh"
#include "tc_host.h"
#include "tc_pair.cuh"

namespace hs {
namespace {

using namespace tc;
using namespace first;

constexpr float kLog2e = 1.44269504088896340736f;

// The band's shape: a function of window, first and the longest document.
struct Band {
  int window, first;  // clipped to the longest document
  int wp, bw, fp;     // Wp; columns of the window and of the first tokens
  int64_t stride;     // elements of a (token, head) row
};

// ================================================================ pass A
namespace pa {

constexpr int kThreads = 512;  // 8 dS warps; producers and issuers; 4 epilogue warps
constexpr int kProd1 = 8, kProd2 = 9, kSWarp = 10, kDqWarp = 11;
constexpr int kSlots = 2;               // of each ring
constexpr int kSlot = 16384;            // ring 1: 64-column chunks by keys; ring 2: panels by columns
constexpr int kMaxDC = 8;               // Dv <= 512
constexpr int kDsBytes = 2 * kPPanel;   // 64 rows x 128 keys
constexpr int kStage = 2048;
constexpr int kSCol = 320, kDpCol = 448;  // TMEM: dQ in columns 0..319, two S buffers, dP

struct Params {
  Docs d;
  Band band;
  int nck, ndc, nqb;   // 64-column chunks of Dk and Dv, 128-column blocks of Dk
  int dk, dv;
  float scale, scale_log2;
  const float* lse;
  const float* sink;          // may be null
  const __nv_bfloat16* out;   // null: delta is there already
  const __nv_bfloat16* dout;
  float* delta;
  float* dsink_part;
  __nv_bfloat16* pband;
  __nv_bfloat16* sband;
  __nv_bfloat16* dq;
  int* spoiled;
  int* spoiled_keys;
  int* status;
  long long wait_ns;
};

struct Shared {
  uint64_t afull[kSlots], aempty[kSlots], bfull[kSlots], bempty[kSlots];
  uint64_t qfull[kMaxQC], qempty[kMaxQC], dfull[kMaxDC], dempty[kMaxDC];
  uint64_t sdfull, sempty[2], dpempty, dsfull, dqdone, passdone, oempty, drain[2], delfull[2];
  float delta[2][kH];  // by pass parity
  uint32_t tmem_base;
};
constexpr size_t kSmem = (size_t)2 * kSlots * kSlot + (size_t)(kMaxQC + kMaxDC) * kQChunk + kDsBytes +
                         4 * kStage + sizeof(Shared);
static_assert(kSmem <= 232448, "shared memory of one CTA");

// The tiles of a pass: 128 columns of the band each, the window's before the
// first tokens'.
struct Tiles {
  int key0, bw, cols, bos;  // key of column 0; the window's and all columns
  int lo, hi;               // keys some token of the pass sees in its window
  int nf;                   // first tokens some token of the pass sees
  __device__ __forceinline__ Tiles(const Pass& ps, const Band& b) {
    const int last = ps.t0 + (ps.mode == 2 ? 1 : 0);
    key0 = (ps.t0 & ~7) - b.wp;
    bw = b.bw;
    cols = b.bw + b.fp;
    bos = ps.bos;
    lo = ps.wlo;
    hi = last;
    nf = min(b.first, max(bos, last - b.window + 1) - bos);
  }
  __device__ __forceinline__ int count() const { return (cols + 127) / 128; }
  __device__ __forceinline__ int n(int i) const { return (min(128, cols - 128 * i) + 31) & ~31; }
  __device__ __forceinline__ bool live(int i) const {
    const int c0 = 128 * i, c1 = c0 + n(i);
    return (c0 < bw && key0 + c0 <= hi && key0 + min(c1, bw) > lo) ||
           (c1 > bw && max(c0, bw) - bw < nf);
  }
  // Row of the 16 columns from c (a multiple of 16).
  __device__ __forceinline__ int row(int c) const { return c < bw ? key0 + c : bos + (c - bw); }
};

// The keys of `rows` columns (a multiple of 16) from column c, `cnt` 64-column
// chunks of K or V `pitch` bytes apart.
__device__ __forceinline__ void load_block(const Tiles& tl, const CUtensorMap* big,
                                           const CUtensorMap* small, uint8_t* dst, uint32_t bar,
                                           int c, int rows, int col, int cnt, int pitch, int lane) {
  if (rows == 64 && c + 64 <= tl.bw) {
    if (lane < cnt) tma_pair_2d(dst + lane * pitch, big, bar, col + 64 * lane, tl.row(c));
  } else {
    const int boxes = rows / 16;
    for (int e = lane; e < boxes * cnt; e += 32) {
      const int q = e / boxes, bx = e - q * boxes;
      tma_pair_2d(dst + q * pitch + bx * 2048, small, bar, col + 64 * q, tl.row(c + 16 * bx));
    }
  }
  __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
query_pass(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap kmap16,
           const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap vmap16,
           const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap dmap,
           const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {
    record_status(p.status, HS_ERR_CUDA);
    return;  // every thread of both CTAs alike
  }
  uint8_t* const ring1 = smem_raw;
  uint8_t* const ring2 = ring1 + kSlots * kSlot;
  uint8_t* const qbuf = ring2 + kSlots * kSlot;
  uint8_t* const dbuf = qbuf + kMaxQC * kQChunk;
  uint8_t* const dsbuf = dbuf + kMaxDC * kQChunk;
  uint8_t* const stage = dsbuf + kDsBytes;
  Shared* sh = reinterpret_cast<Shared*>(stage + 4 * kStage);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const long long lim = p.wait_ns;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh->afull[i], 1);
      mbar_init(&sh->aempty[i], 1);
      mbar_init(&sh->bfull[i], 1);
      mbar_init(&sh->bempty[i], 1);
    }
    for (int i = 0; i < kMaxQC; ++i) {
      mbar_init(&sh->qfull[i], 1);
      mbar_init(&sh->qempty[i], 1);
    }
    for (int i = 0; i < kMaxDC; ++i) {
      mbar_init(&sh->dfull[i], 1);
      mbar_init(&sh->dempty[i], 1);
    }
    mbar_init(&sh->sdfull, 1);
    mbar_init(&sh->sempty[0], 16);  // 8 warps of each CTA
    mbar_init(&sh->sempty[1], 16);
    mbar_init(&sh->dpempty, 16);
    mbar_init(&sh->dsfull, 16);
    mbar_init(&sh->dqdone, 1);
    mbar_init(&sh->passdone, 1);
    mbar_init(&sh->oempty, 8);  // 4 epilogue warps of each CTA
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    mbar_init(&sh->delfull[0], 4);  // the epilogue warps
    mbar_init(&sh->delfull[1], 4);
    fence_barrier_init();
  }
  if (warp == kSWarp) tmem_alloc_pair(&sh->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  after_previous();
  const uint32_t tmem = sh->tmem_base;
  Walk walk(p.d, blockIdx.x >> 1, gridDim.x >> 1);
  Pass ps;
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------ P and dS
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int g4 = warp & 3, ch = warp >> 2, hi = g4 >> 1;
    const int row = 32 * (g4 & 1) + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
    uint32_t nt = 0, npass = 0;  // live tiles
    auto tell_leader = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(bar);
    };
    auto no_document = [&](int t) {
      if (rank != 0) return;
      const int units = (p.band.bw + p.band.fp) / 8;
      for (int e = tid; e < kH * units; e += 256) {
        const int64_t at = ((int64_t)t * kH + e / units) * p.band.stride + e % units * 8;
        *reinterpret_cast<uint4*>(p.pband + at) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(p.sband + at) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (tid < kH) p.dsink_part[(int64_t)t * kH + tid] = 0.f;
      if (tid == 0) p.spoiled[t] = p.spoiled_keys[t] = 0;
    };
    while (ok && walk.next(ps, nullptr, no_document)) {
      const Tiles tl(ps, p.band);
      const bool act = ps.active(rank);
      const int t = ps.token(rank);
      const int own = max(ps.bos, t - p.band.window + 1);  // this token's window
      const int nf = min(p.band.first, own - ps.bos);      // and first tokens
      const int64_t th = (int64_t)t * kH + row;
      const float lse2 = act ? __ldg(p.lse + th) * kLog2e : 0.f;
      if (!warp_wait(&sh->delfull[npass & 1], (npass >> 1) & 1, lim)) { ok = false; break; }
      const float del = sh->delta[npass & 1][row];
      ++npass;
      for (int i = 0; i < tl.count() && ok; ++i) {
        const int n2 = tl.n(i) / 2, c0 = 32 * ch, k0 = hi * n2 + c0;  // key of column 0 in the tile
        const bool live = tl.live(i), mine = act && c0 < n2;
        uint32_t pp[16], pd[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) pp[k] = pd[k] = 0u;
        if (live) {
          const uint32_t buf = nt & 1;
          if (!warp_wait(&sh->sdfull, nt & 1, lim)) { ok = false; break; }
          tc_fence_after();
          uint32_t u[32], w[32];
          if (mine) {
            tmem_ld32(lane_base + kSCol + buf * 64 + c0, u);
            tmem_ld32(lane_base + kDpCol + c0, w);
            tmem_ld_wait();
            reg_fence(u);
            reg_fence(w);
          }
          tell_leader(&sh->sempty[buf]);
          tell_leader(&sh->dpempty);
          if (mine) {
            const int s0 = 128 * i + k0;  // band column
            const uint32_t bits = (range_bits(own - tl.key0 - s0, t - tl.key0 - s0) |
                                   range_bits(tl.bw - s0, tl.bw + nf - 1 - s0)) &
                                  low_bits(n2 - c0);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              // zero outside the key set whatever is there
              float p0 = fast_exp2(fmaf(__uint_as_float(u[2 * k]), p.scale_log2, -lse2));
              float p1 = fast_exp2(fmaf(__uint_as_float(u[2 * k + 1]), p.scale_log2, -lse2));
              float d0 = p0 * (__uint_as_float(w[2 * k]) - del);
              float d1 = p1 * (__uint_as_float(w[2 * k + 1]) - del);
              if (!(bits & (1u << (2 * k)))) p0 = d0 = 0.f;
              if (!(bits & (2u << (2 * k)))) p1 = d1 = 0.f;
              __nv_bfloat162 a = __floats2bfloat162_rn(p0, p1), b = __floats2bfloat162_rn(d0, d1);
              pp[k] = *reinterpret_cast<uint32_t*>(&a);
              pd[k] = *reinterpret_cast<uint32_t*>(&b);
            }
          }
          // dQ of the tile before has read dS
          if (nt > 0 && !warp_wait(&sh->dqdone, (nt - 1) & 1, lim)) { ok = false; break; }
          if (mine) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (c0 + 8 * q >= n2) break;
              const int key = k0 + 8 * q;
              *reinterpret_cast<uint4*>(dsbuf + (key >> 6) * kPPanel + row * 128 +
                                        ((((key >> 3) & 7) ^ (row & 7)) << 4)) =
                  make_uint4(pd[4 * q], pd[4 * q + 1], pd[4 * q + 2], pd[4 * q + 3]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          ++nt;
          tell_leader(&sh->dsfull);
        }
        if (mine) {
          const int64_t at = th * p.band.stride + 128 * i + k0;
          const int left = tl.cols - 128 * i - k0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (8 * q >= left || c0 + 8 * q >= n2) break;
            *reinterpret_cast<uint4*>(p.pband + at + 8 * q) =
                make_uint4(pp[4 * q], pp[4 * q + 1], pp[4 * q + 2], pp[4 * q + 3]);
            *reinterpret_cast<uint4*>(p.sband + at + 8 * q) =
                make_uint4(pd[4 * q], pd[4 * q + 1], pd[4 * q + 2], pd[4 * q + 3]);
          }
        }
      }
    }
    if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kProd1 || warp == kProd2) {
      // ---------------------------------------------------------- producers
      const bool two = warp == kProd2;
      uint64_t* const fullb = two ? sh->bfull : sh->afull;
      uint64_t* const emptyb = two ? sh->bempty : sh->aempty;
      uint8_t* const ring = two ? ring2 : ring1;
      int slot = 0;
      uint32_t ph = 0, qph = 0;
      bool first_pass = true;
      auto claim = [&](int bytes) -> bool {
        if (!warp_wait(&emptyb[slot], ph ^ 1, lim)) return false;
        if (leader && lane == 0) mbar_expect_tx(&fullb[slot], 2 * bytes);
        __syncwarp();
        return true;
      };
      auto next = [&]() {
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1;
        }
      };
      while (ok && walk.next(ps, leader && !two ? p.status : nullptr)) {
        const Tiles tl(ps, p.band);
        // Q (with K and V) and dO (with K's columns, which the tile needs last)
        // chunk by chunk, each once the pass before has read it
        uint64_t* const mfull = two ? sh->dfull : sh->qfull;
        uint64_t* const mempty = two ? sh->dempty : sh->qempty;
        for (int c = 0; c < (two ? p.ndc : p.nck) && ok; ++c) {
          if (!first_pass && !warp_wait(&mempty[c], qph ^ 1, lim)) { ok = false; break; }
          if (lane == 0) {
            if (leader) mbar_expect_tx(&mfull[c], 2 * kQChunk);
            tma_pair_3d((two ? dbuf : qbuf) + c * kQChunk, two ? &dmap : &qmap,
                        leader_addr(&mfull[c]), c * 64, 0, ps.token(rank));
          }
          __syncwarp();
        }
        first_pass = false;
        qph ^= 1;
        for (int i = 0; i < tl.count() && ok; ++i) {
          if (!tl.live(i)) continue;
          const int n = tl.n(i);
          if (!two) {  // K, then V: this CTA's half of the keys
            const int rows = n / 2, per = 128 / rows;
            for (int v = 0; v < 2 && ok; ++v) {
              const int nch = v ? p.ndc : p.nck;
              for (int c = 0; c < nch && ok; c += per, next()) {
                const int cnt = min(per, nch - c);
                if (!claim(cnt * rows * 128)) { ok = false; break; }
                load_block(tl, v ? &vmap : &kmap, v ? &vmap16 : &kmap16, ring + slot * kSlot,
                           leader_addr(&fullb[slot]), 128 * i + rank * rows, rows, c * 64, cnt,
                           rows * 128, lane);
              }
            }
          } else {  // K: this CTA's half of each 256 (or last 128) columns
            for (int b = 0; b < p.nqb && ok; b += 2) {
              const int panels = b + 1 < p.nqb ? 2 : 1, col = b * 128 + rank * panels * 64;
              for (int k0 = 0; k0 < n && ok; k0 += 64, next()) {
                const int rows = min(64, n - k0);
                if (!claim(rows * 128 * panels)) { ok = false; break; }
                load_block(tl, &kmap, &kmap16, ring + slot * kSlot, leader_addr(&fullb[slot]),
                           128 * i + k0, rows, col, panels, 8192, lane);
              }
            }
          }
        }
      }
      if (!ok) {  // see tc_first_fwd.cu: copies under way land before the CTA may exit
        if (lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
        for (const uint64_t from = global_ns(); global_ns() - from < 1000000;) {
        }
      }
    } else if (warp == kSWarp || warp == kDqWarp) {
      // ---------------------------------------------------------- MMA issuers
      if (leader) {
        const bool is_dq = warp == kDqWarp;
        const uint64_t a_desc = umma_desc_sw128(smem_u32(ring1), 16, 1024);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(qbuf), 16, 1024);
        const uint64_t do_desc = umma_desc_sw128(smem_u32(dbuf), 16, 1024);
        const uint64_t b_desc = umma_desc_sw128(smem_u32(ring2), 8192, 1024);
        const uint64_t ds_desc = umma_desc_sw128(smem_u32(dsbuf), 16, 1024);
        int slot = 0;
        uint32_t ph = 0, nt = 0, npass = 0;
        auto next = [&]() {
          if (++slot == kSlots) {
            slot = 0;
            ph ^= 1;
          }
        };
        while (ok && walk.next(ps, nullptr)) {
          const Tiles tl(ps, p.band);
          bool first = true;
          int last = 0;  // the pass's last live tile
          for (int i = 0; i < tl.count(); ++i)
            if (tl.live(i)) last = i;
          for (int i = 0; i < tl.count() && ok; ++i) {
            if (!tl.live(i)) continue;
            const int n = tl.n(i);
            if (!is_dq) {
              const uint32_t id = idesc_bf16_f32(128, n, false, false);
              const int rows = n / 2, per = 128 / rows;
              for (int v = 0; v < 2 && ok; ++v) {
                const uint32_t d = tmem + (v ? kDpCol : kSCol + (nt & 1) * 64);
                if (!(v ? warp_wait(&sh->dpempty, (nt & 1) ^ 1, lim)
                        : warp_wait(&sh->sempty[nt & 1], ((nt >> 1) & 1) ^ 1, lim))) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                const int nch = v ? p.ndc : p.nck;
                uint64_t* const full = v ? sh->dfull : sh->qfull;
                uint64_t* const empty = v ? sh->dempty : sh->qempty;
                const uint64_t m_desc = v ? do_desc : q_desc;
                for (int c0 = 0; c0 < nch && ok; c0 += per) {
                  if (!warp_wait(&sh->afull[slot], ph, lim)) { ok = false; break; }
                  tc_fence_after();
                  for (int c = c0; c < min(nch, c0 + per); ++c) {
                    if (first && !warp_wait(&full[c], npass & 1, lim)) { ok = false; break; }
                    const uint64_t a = m_desc + (uint64_t)((c * kQChunk) >> 4);
                    const uint64_t b = a_desc + (uint64_t)((slot * kSlot + (c - c0) * rows * 128) >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                      umma_pair(d, a + 2 * k, b + 2 * k, id, (c > 0 || k > 0) ? 1u : 0u);
                    if (i == last) commit_pair(&empty[c]);
                  }
                  commit_pair(&sh->aempty[slot]);
                  next();
                }
              }
              if (!ok) break;
              commit_pair(&sh->sdfull);
            } else {
              if (!warp_wait(&sh->dsfull, nt & 1, lim) ||
                  (first && npass > 0 && !warp_wait(&sh->oempty, (npass - 1) & 1, lim))) {
                ok = false;
                break;
              }
              tc_fence_after();
              for (int b = 0; b < p.nqb && ok; b += 2) {
                const uint32_t id = idesc_bf16_f32(128, b + 1 < p.nqb ? 256 : 128, false, true);
                for (int k0 = 0; k0 < n; k0 += 64) {
                  if (!warp_wait(&sh->bfull[slot], ph, lim)) { ok = false; break; }
                  tc_fence_after();
                  const uint64_t a = ds_desc + (uint64_t)(((k0 >> 6) * kPPanel) >> 4);
                  const uint64_t bb = b_desc + (uint64_t)((slot * kSlot) >> 4);
                  const int steps = min(64, n - k0) / 16;
                  for (int k = 0; k < steps; ++k)
                    umma_pair(tmem + b * 64, a + 2 * k, bb + (uint64_t)(k * 128), id,
                              (!first || k0 > 0 || k > 0) ? 1u : 0u);
                  commit_pair(&sh->bempty[slot]);
                  next();
                }
              }
              if (!ok) break;
              commit_pair(&sh->dqdone);
              if (i == last) commit_pair(&sh->passdone);
            }
            first = false;
            ++nt;
          }
          ++npass;
        }
        if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
        commit_pair(&sh->drain[is_dq]);  // every MMA done before TMEM is released
        (void)warp_wait(&sh->drain[is_dq], 0, kDefaultWaitNs);
      }
    } else {
      // ---------------------------------------------------------- delta, and dQ out (see tc_first_fwd.cu)
      const int g4 = warp & 3, hi = g4 >> 1, row0 = 32 * (g4 & 1);
      const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
      uint8_t* const st = stage + g4 * kStage;
      uint32_t npass = 0;
      // delta of a pass's token while the pass before it runs: 16 rows a warp, two
      // at a time, dout once more (out of L2, the producer loads it too)
      Walk ahead(walk);
      uint32_t nahead = 0;
      auto delta_of_next = [&]() {
        Pass pn;
        if (!ahead.next(pn, nullptr)) return;
        if (pn.active(rank)) {
          const int t = pn.token(rank), units = p.dv / 8;
          if (p.out && g4 == 0 && lane == 0) p.spoiled[t] = p.spoiled_keys[t] = 0;
#pragma unroll 1
          for (int r = 16 * g4; r < 16 * g4 + 16; r += 2) {
            const int64_t th = (int64_t)t * kH + r;
            float acc[2] = {0.f, 0.f};
            if (p.out) {
              uint4 x[2][2], y[2][2];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = lane + 32 * (k & 1);
                x[k >> 1][k & 1] = y[k >> 1][k & 1] = make_uint4(0u, 0u, 0u, 0u);
                if (e >= units) continue;
                const int64_t at = (th + (k >> 1)) * p.dv + 8 * e;
                x[k >> 1][k & 1] = __ldcs(reinterpret_cast<const uint4*>(p.out + at));
                y[k >> 1][k & 1] = __ldg(reinterpret_cast<const uint4*>(p.dout + at));
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162* const xp =
                    reinterpret_cast<const __nv_bfloat162*>(&x[k >> 1][k & 1]);
                const __nv_bfloat162* const yp =
                    reinterpret_cast<const __nv_bfloat162*>(&y[k >> 1][k & 1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 u = __bfloat1622float2(xp[i]), v = __bfloat1622float2(yp[i]);
                  acc[k >> 1] = fmaf(u.x, v.x, fmaf(u.y, v.y, acc[k >> 1]));
                }
              }
              acc[0] = warp_sum(acc[0]);
              acc[1] = warp_sum(acc[1]);
            }
            if (lane < 2) {
              float d = lane ? acc[1] : acc[0];
              if (p.out) {
                p.delta[th + lane] = d;
                p.dsink_part[th + lane] =
                    p.sink ? -expf(__ldg(p.sink + r + lane) - __ldg(p.lse + th + lane)) * d : 0.f;
              } else {
                d = p.delta[th + lane];
              }
              sh->delta[nahead & 1][r + lane] = d;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->delfull[nahead & 1]);
        ++nahead;
      };
      delta_of_next();
      while (ok && walk.next(ps, nullptr)) {
        delta_of_next();
        if (!warp_wait(&sh->passdone, npass & 1, lim)) { ok = false; break; }
        tc_fence_after();
        if (ps.active(rank)) {
          const int t = ps.token(rank);
          __nv_bfloat16* const o = p.dq + ((int64_t)t * kH + row0) * p.dk;
          float finite = 0.f;
#pragma unroll 1
          for (int c = 0; c < p.nqb * 64; c += 32) {
            const int b = c >> 7, wide = 2 * b + 1 < p.nqb ? 128 : 64;
            const int d = 256 * b + hi * wide + (c - 128 * b);
            uint32_t w[32];
            tmem_ld32(lane_base + c, w);
            tmem_ld_wait();
            reg_fence(w);
            if (d >= p.dk) continue;
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(w[8 * q + 2 * k]) * p.scale;
                const float c1 = __uint_as_float(w[8 * q + 2 * k + 1]) * p.scale;
                finite = fmaf(a, 0.f, fmaf(c1, 0.f, finite));  // NaN from NaN and infinities
                __nv_bfloat162 pr = __floats2bfloat162_rn(a, c1);
                v[k] = *reinterpret_cast<uint32_t*>(&pr);
              }
              *reinterpret_cast<uint4*>(st + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int rr = 8 * j + (lane >> 2), q = lane & 3;
              *reinterpret_cast<uint4*>(o + (int64_t)rr * p.dk + d + 8 * q) =
                  *reinterpret_cast<const uint4*>(st + rr * 64 + ((q ^ ((rr >> 1) & 3)) << 4));
            }
          }
          if (finite != 0.f) p.spoiled[t] = 1;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh->oempty);
        ++npass;
      }
      if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kSWarp) tmem_dealloc_pair(tmem, 512);
}

}  // namespace pa

// ================================================================ pass B
namespace pb {

constexpr int kThreads = 256;   // warp 0 producer, warp 1 issuer, warps 4..7 epilogue
constexpr int kKeys = 256;      // most keys of an item
// Tokens of an item: many make few partial sums and a small workspace, few keep
// every SM busy.  Whole backward at the MLA shape, us with 32 / 64 / 128 / 256 tokens:
//   window 512 + 4: T 150: 64 / 83 / 93 / 124       T 420: 148 / 130 / 146 / 235
//     T 1023: 308 / 294 / 311 / 340                 T 4096: 1220 / 1140 / 1146 / 1157
//     T 8192: 2469 / 2352 / 2335 / 2400
//   window 64 + 5, T 333: 77 / 89 / 123 / 126       window 128 + 4, T 4096: 699 / 679 / 683 / 697
__host__ __device__ constexpr int tok_of(int T) { return T >= 8192 ? 128 : T >= 400 ? 64 : 32; }
constexpr int kStages = 4;
constexpr int kPanel = 8192;    // 64 heads x 64 columns
constexpr int kStageBytes = 6 * kPanel;  // 4 panels of q or dout, 2 of the band

struct Params {
  Docs d;
  Band band;
  int dk, dv;
  int gk, groups;     // 512-column groups of Dk; of Dk and Dv together
  int segs, n;        // items of a chunk's keys, each n of them
  int tok, chunks;    // tokens of an item; as many chunks of them in the batch
  float* wpart;       // [chunks][segs * n][dk + dv]
  float* fpart;       // [chunks + num_docs][fp][dk + dv]
  int* status;
  long long wait_ns;
};

struct Shared {
  uint64_t full[kStages], empty[kStages], done, freed, drain;
  uint32_t tmem_base;
};
constexpr size_t kSmem = (size_t)kStages * kStageBytes + sizeof(Shared);

// One accumulation: tokens [t0, t1) against n keys, columns [col0, col0 + cols)
// of q (dk) or dout (dv), into a partial sum.
struct Job {
  bool is_k, window;
  int t0, t1, n;
  int key0;        // window: first key; else 0
  int col0, cols;  // cols <= 512
  float* dst;      // [keys][dk + dv] at this matrix's column col0
  int keys;        // rows of dst that are written
};

struct Jobs {
  const Params& p;
  int item, step, doc_t;  // doc_t: where the rest of a chunk of documents begins
  __device__ __forceinline__ Jobs(const Params& pp, int first, int pairs)
      : p(pp), item(first), step(pairs), doc_t(-1) {}
  __device__ __forceinline__ bool next(Job& j) {
    // chunk by chunk of tokens, c0 ..: its keys from c0 - Wp, the column groups of
    // each
    const int nwin = p.chunks * p.segs * p.groups;
    const int total = nwin + (p.band.fp > 0 ? p.chunks * p.groups : 0);
    const int W = p.dk + p.dv;
    for (; item < total; item += step) {
      const int e = item < nwin ? item : item - nwin;
      const int g = e % p.groups;
      int r = e / p.groups;
      j.is_k = g < p.gk;
      const int gi = j.is_k ? g : g - p.gk;
      j.col0 = 512 * gi;
      j.cols = min(512, (j.is_k ? p.dk : p.dv) - j.col0);
      const int at = (j.is_k ? 0 : p.dk) + j.col0;
      if (item < nwin) {
        const int c0 = r / p.segs * p.tok;
        j.window = true;
        j.key0 = c0 - p.band.wp + r % p.segs * p.n;
        j.n = p.n;
        // tokens whose windows reach these keys
        j.t0 = max(c0, j.key0);
        j.t1 = min(min(c0 + p.tok, p.d.T), j.key0 + p.n - 1 + p.band.window);
        if (j.t0 >= j.t1) continue;
        j.dst = p.wpart + (int64_t)r * p.n * W + at;
        j.keys = min(p.n, p.d.T - j.key0);
        item += step;
        return true;
      }
      // a chunk of tokens: its documents one after the other
      const int c0 = r * p.tok, c1 = min(p.d.T, c0 + p.tok);
      for (int t = doc_t < 0 ? c0 : doc_t; t < c1;) {
        int lo = 0, hi = p.d.num_docs;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.d.cu + mid) <= t) lo = mid; else hi = mid;
        }
        const int bos = __ldg(p.d.cu + lo), eos = __ldg(p.d.cu + lo + 1);
        if (bos < 0 || bos > t || eos <= t) {  // in no document: pass A reports it
          ++t;
          continue;
        }
        const int from = max(t, bos + p.band.window), to = min(c1, eos);
        t = to;
        if (from >= to) continue;  // every token's window reaches the document's start
        j.window = false;
        j.key0 = 0;
        j.n = (p.band.fp + 31) & ~31;
        j.t0 = from;
        j.t1 = to;
        j.dst = p.fpart + (int64_t)(r + lo) * p.band.fp * W + at;
        j.keys = p.band.fp;
        if (to < c1) {
          doc_t = to;
        } else {
          doc_t = -1;
          item += step;
        }
        return true;
      }
      doc_t = -1;
    }
    return false;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
key_pass(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap dmap,
         const __grid_constant__ CUtensorMap pwmap, const __grid_constant__ CUtensorMap pfmap,
         const __grid_constant__ CUtensorMap swmap, const __grid_constant__ CUtensorMap sfmap,
         const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {
    record_status(p.status, HS_ERR_CUDA);
    return;  // every thread of both CTAs alike
  }
  uint8_t* const ring = smem_raw;
  Shared* sh = reinterpret_cast<Shared*>(ring + kStages * kStageBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const long long lim = p.wait_ns;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->done, 1);
    mbar_init(&sh->freed, 8);  // 4 epilogue warps of each CTA
    mbar_init(&sh->drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(&sh->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  after_previous();
  const uint32_t tmem = sh->tmem_base;
  Jobs jobs(p, blockIdx.x >> 1, gridDim.x >> 1);
  Job j;
  bool ok = true;
  if (warp == 0) {
    int slot = 0;
    uint32_t ph = 0;
    while (ok && jobs.next(j)) {
      const int units = (j.cols + 127) / 128;  // 128-column blocks
      const int bp = (j.n / 2 + 63) / 64;      // band panels of this CTA
      const CUtensorMap* const band = j.window ? (j.is_k ? &swmap : &pwmap) : (j.is_k ? &sfmap : &pfmap);
      for (int t = j.t0; t < j.t1; ++t) {
        if (!warp_wait(&sh->empty[slot], ph ^ 1, lim)) { ok = false; break; }
        const uint32_t bar = leader_addr(&sh->full[slot]);
        // panels: per 256 columns 128 (two panels) of each CTA, of a last 128 one
        if (leader && lane == 0) mbar_expect_tx(&sh->full[slot], 2 * (units + bp) * kPanel);
        __syncwarp();
        uint8_t* const dst = ring + slot * kStageBytes;
        if (lane < units) {
          const int b = lane >> 1, wide = 2 * b + 1 < units ? 2 : 1;
          const int col = j.col0 + 256 * b + (rank * wide + (lane & 1)) * 64;
          tma_pair_3d(dst + lane * kPanel, j.is_k ? &qmap : &dmap, bar, col, 0, t);
        } else if (lane < units + bp) {
          const int pn = lane - units;
          const int x = j.window ? j.key0 - ((t & ~7) - p.band.wp) : 0;
          tma_pair_3d(dst + (4 + pn) * kPanel, band, bar, x + rank * (j.n / 2) + 64 * pn, 0, t);
        }
        __syncwarp();
        if (++slot == kStages) {
          slot = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {  // see tc_first_fwd.cu
      if (lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
      for (const uint64_t from = global_ns(); global_ns() - from < 1000000;) {
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint64_t a_desc = umma_desc_sw128(smem_u32(ring), kPanel, 1024);
      const uint64_t b_desc = umma_desc_sw128(smem_u32(ring) + 4 * kPanel, kPanel, 1024);
      int slot = 0;
      uint32_t ph = 0, njob = 0;
      while (ok && jobs.next(j)) {
        const int units = (j.cols + 127) / 128;
        const uint32_t id2 = idesc_bf16_f32(256, j.n, true, true);
        const uint32_t id1 = idesc_bf16_f32(128, j.n, true, true);
        if (njob > 0 && !warp_wait(&sh->freed, (njob - 1) & 1, lim)) { ok = false; break; }
        tc_fence_after();
        for (int t = j.t0; t < j.t1; ++t) {
          if (!warp_wait(&sh->full[slot], ph, lim)) { ok = false; break; }
          tc_fence_after();
          const uint64_t a = a_desc + (uint64_t)((slot * kStageBytes) >> 4);
          const uint64_t b = b_desc + (uint64_t)((slot * kStageBytes) >> 4);
          for (int u = 0; u < units; u += 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_pair(tmem + (u >> 1) * kKeys, a + (uint64_t)((u * kPanel) >> 4) + k * 128,
                        b + k * 128, u + 1 < units ? id2 : id1, (t > j.t0 || k > 0) ? 1u : 0u);
          }
          commit_pair(&sh->empty[slot]);
          if (++slot == kStages) {
            slot = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        commit_pair(&sh->done);
        ++njob;
      }
      if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
      commit_pair(&sh->drain);
      (void)warp_wait(&sh->drain, 0, kDefaultWaitNs);
    }
  } else if (warp >= 4) {
    // D^T: lanes are columns of dk or dv, TMEM columns are keys.  A 256-column
    // block: lane = column 128 rank + lane, every key.  A 128-column one: lanes
    // 0..63 and 64..127 both are columns 64 rank + .., halves of the keys.
    const int g4 = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
    const int W = p.dk + p.dv;
    uint32_t njob = 0;
    while (ok && jobs.next(j)) {
      if (!warp_wait(&sh->done, njob & 1, lim)) { ok = false; break; }
      tc_fence_after();
      const int units = (j.cols + 127) / 128;
      for (int u = 0; u < units; u += 2) {
        const bool wide = u + 1 < units;
        const int l = 32 * g4 + lane;
        const int col = 128 * u + (wide ? 128 * rank + l : 64 * rank + (l & 63));
        const int kb = wide ? 0 : (l >> 6) * (j.n / 2), nk = wide ? j.n : j.n / 2;
#pragma unroll 1
        for (int c = 0; c < nk; c += 16) {
          uint32_t w[16];
          tmem_ld16(lane_base + (u >> 1) * kKeys + c, w);
          tmem_ld_wait();
          reg_fence(w);
          if (col >= j.cols) continue;
          float* const dst = j.dst + (int64_t)(kb + c) * W + col;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (kb + c + k < j.keys) dst[(int64_t)k * W] = __uint_as_float(w[k]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(&sh->freed);
      ++njob;
    }
    if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// dk and dv of one key: its partial sums in order, only ones that a job wrote.
// A thread has 4 columns of each of its block's keys.  The first kH blocks sum the
// sink's terms where dsink is wanted.
constexpr int kReduce = 288;  // threads, at least (Dk + Dv) / 4
__global__ void __launch_bounds__(kReduce) reduce(const __grid_constant__ Params p, float scale,
                                              __nv_bfloat16* dkey, __nv_bfloat16* dval,
                                              int* spoiled, const float* dsink_part,
                                              float* dsink) {
  const int W = p.dk + p.dv, extra = dsink ? kH : 0;
  after_previous();
  if ((int)blockIdx.x < extra) {
    __shared__ float red[256];
    float acc = 0.f;
    if (threadIdx.x < 256) {
#pragma unroll 4
      for (int t = threadIdx.x; t < p.d.T; t += 256)
        acc += dsink_part[(int64_t)t * kH + blockIdx.x];
      red[threadIdx.x] = acc;
    }
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
      if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
      __syncthreads();
    }
    if (threadIdx.x == 0) dsink[blockIdx.x] = red[0];
    return;
  }
  for (int j = blockIdx.x - extra; j < p.d.T; j += gridDim.x - extra) {
    // chunks with a token whose window reaches j
    const int w0 = j / p.tok, w1 = min(p.d.T - 1, j + p.band.window - 1) / p.tok;
    int bos, eos, doc = 0, c0 = 1, c1 = 0, f = 0;  // chunks with first-token sums
    if (p.band.fp > 0 &&
        find_doc(p.d.cu, p.d.num_docs, p.d.T, p.d.max_seqlen, j, bos, eos, nullptr)) {
      f = j - bos;
      if (f < p.band.first && bos + p.band.window < eos) {
        int lo = 0, hi = p.d.num_docs;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.d.cu + mid) <= j) lo = mid; else hi = mid;
        }
        doc = lo;
        c0 = (bos + p.band.window) / p.tok;
        c1 = (eos - 1) / p.tok;
      }
    }
    const int col = threadIdx.x * 4;
    if (col < W) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](const float* at) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(at));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      };
#pragma unroll 4
      for (int c = w0; c <= w1; ++c)
        add(p.wpart + ((int64_t)c * p.segs * p.n + (j - (c * p.tok - p.band.wp))) * W + col);
#pragma unroll 4
      for (int c = c0; c <= c1; ++c)
        add(p.fpart + ((int64_t)(c + doc) * p.band.fp + f) * W + col);
      const bool is_k = col < p.dk;
      const float m = is_k ? scale : 1.f;
      if (!(isfinite(s.x) && isfinite(s.y) && isfinite(s.z) && isfinite(s.w))) spoiled[j] = 1;
      __nv_bfloat162* const o = reinterpret_cast<__nv_bfloat162*>(
          is_k ? dkey + (int64_t)j * p.dk + col : dval + (int64_t)j * p.dv + (col - p.dk));
      o[0] = __floats2bfloat162_rn(m * s.x, m * s.y);
      o[1] = __floats2bfloat162_rn(m * s.z, m * s.w);
    }
  }
}

}  // namespace pb

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Row stride of the band, at least bw + fp, for a window and first tokens of
// together `span` keys.
int64_t band_stride(int64_t span) { return (span + 51) & ~(int64_t)7; }

struct Sizes {
  size_t band, wpart, fpart;
  int chunks, segs, n;
};
Sizes sizes_of(int T, int num_docs, int span, int window, int fp, int dk, int dv) {
  Sizes z{};
  const size_t W = (size_t)(dk + dv) * sizeof(float);
  z.band = align256((size_t)T * kH * band_stride(span) * 2);
  const int tok = pb::tok_of(T);
  const int keys = ((window - 1 + 7) & ~7) + tok;  // of a chunk
  z.chunks = (T + tok - 1) / tok;
  z.segs = (keys + pb::kKeys - 1) / pb::kKeys;
  z.n = ((keys + z.segs - 1) / z.segs + 31) & ~31;
  z.wpart = align256((size_t)z.chunks * z.segs * z.n * W);
  z.fpart = align256((size_t)(z.chunks + num_docs) * fp * W);
  return z;
}

constexpr size_t kMostBytes = (size_t)4 << 30;  // of workspace; beyond it the other passes run

}  // namespace

size_t tc_first_bwd_workspace(int total_tokens, int num_docs, int max_seqlen, int span, int dk,
                              int dv) {
  max_seqlen = std::min(max_seqlen, total_tokens);  // a loose bound costs nothing
  if (span < 1) span = 1;
  if (span / 2 >= max_seqlen) span = 2 * max_seqlen;
  // the most any split of the span into window and first tokens needs
  const int fp = std::min((span + 15) & ~15, pb::kKeys);
  const Sizes z = sizes_of(total_tokens, num_docs, span, std::min(span, max_seqlen), fp, dk, dv);
  const size_t n = 2 * z.band + z.wpart + z.fpart;
  return n <= kMostBytes ? n : 0;
}

namespace {
Band band_of(const BwdArgs& b) {
  const int longest = std::min(b.p.max_seqlen, b.p.total_tokens);
  Band band;
  band.window = std::min(b.window, longest);
  // a window that holds every document leaves no first token outside
  band.first = band.window >= longest ? 0 : std::min(b.first, longest);
  band.wp = (band.window - 1 + 7) & ~7;
  band.bw = (band.wp + 8 + 15) & ~15;
  band.fp = (band.first + 15) & ~15;
  band.stride = band_stride(band.window + band.first);
  return band;
}
Sizes sizes_of(const BwdArgs& b, const Band& band) {
  return sizes_of(b.p.total_tokens, b.p.num_docs, band.window + band.first, band.window, band.fp,
                  b.p.dk, b.p.dv);
}
}  // namespace

bool tc_first_bwd_takes(const BwdArgs& b) {
  const Band band = band_of(b);
  if (band.fp > pb::kKeys || !b.dkdv_ws) return false;
  const Sizes z = sizes_of(b, band);
  return 2 * z.band + z.wpart + z.fpart <= b.dkdv_bytes;
}

cudaError_t launch_tc_first_bwd(const BwdArgs& b, bool with_delta, float* delta, float* dsink_part,
                                int* spoiled, int* spoiled_keys, long long wait_limit,
                                cudaStream_t s) {
  const Problem& p = b.p;
  const Band band = band_of(b);
  const Sizes z = sizes_of(b, band);
  uint8_t* w = static_cast<uint8_t*>(b.dkdv_ws);
  __nv_bfloat16* const pband = reinterpret_cast<__nv_bfloat16*>(w);
  __nv_bfloat16* const sband = reinterpret_cast<__nv_bfloat16*>(w + z.band);
  CUtensorMap kmap, kmap16, vmap, vmap16, qmap, dmap, pw, pf, sw, sf;
  const int T = p.total_tokens;
  auto band_map = [&](CUtensorMap* m, const __nv_bfloat16* base, int cols) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)kH, (uint64_t)T};
    const uint64_t strides[2] = {(uint64_t)band.stride * 2, (uint64_t)band.stride * kH * 2};
    const uint32_t box[3] = {64, (uint32_t)kH, 1};
    return encode_bf16_map(m, base, 3, dims, strides, box);
  };
  if (!row_map(&kmap, p.k, p.dk, T, p.k_row_stride, 64) ||
      !row_map(&kmap16, p.k, p.dk, T, p.k_row_stride, 16) ||
      !row_map(&vmap, p.v, p.dv, T, p.v_row_stride, 64) ||
      !row_map(&vmap16, p.v, p.dv, T, p.v_row_stride, 16) ||
      !head_map(&qmap, p.q, p.dk, T, p.q_row_stride, p.q_head_stride) ||
      !head_map(&dmap, b.dout, p.dv, T, (int64_t)kH * p.dv, p.dv) ||
      !band_map(&pw, pband, band.bw) || !band_map(&sw, sband, band.bw) ||
      !band_map(&pf, pband + band.bw, band.fp > 0 ? band.fp : 8) ||
      !band_map(&sf, sband + band.bw, band.fp > 0 ? band.fp : 8))
    return cudaErrorInvalidValue;
  pa::Params a{};
  a.d = docs_of(p, band.window, band.first);
  a.band = band;
  a.nck = p.dk / 64;
  a.ndc = p.dv / 64;
  a.nqb = (p.dk + 127) / 128;
  a.dk = p.dk;
  a.scale = p.scale;
  a.scale_log2 = p.scale * kLog2e;
  a.dv = p.dv;
  a.lse = b.lse;
  a.sink = b.sink;
  a.out = with_delta ? static_cast<const __nv_bfloat16*>(b.out) : nullptr;
  a.dout = static_cast<const __nv_bfloat16*>(b.dout);
  a.delta = delta;
  a.dsink_part = dsink_part;
  a.pband = pband;
  a.sband = sband;
  a.dq = static_cast<__nv_bfloat16*>(b.dq);
  a.spoiled = spoiled;
  a.spoiled_keys = spoiled_keys;
  a.status = p.status;
  a.wait_ns = wait_limit > 0 ? wait_limit : kDefaultWaitNs;
  cudaError_t e = cudaFuncSetAttribute(pa::query_pass, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)pa::kSmem);
  if (e != cudaSuccess) return e;
  if (with_delta) {  // the call's first kernel
    pa::query_pass<<<pair_grid(T), pa::kThreads, pa::kSmem, s>>>(kmap, kmap16, vmap, vmap16, qmap,
                                                                dmap, a);
    e = cudaGetLastError();
  } else {
    e = launch_after(pa::query_pass, pair_grid(T), pa::kThreads, pa::kSmem, s, kmap, kmap16, vmap,
                     vmap16, qmap, dmap, a);
  }
  if (e != cudaSuccess) return e;
  pb::Params k{};
  k.d = a.d;
  k.band = band;
  k.dk = p.dk;
  k.dv = p.dv;
  k.gk = (p.dk + 511) / 512;
  k.groups = k.gk + (p.dv + 511) / 512;
  k.segs = z.segs;
  k.n = z.n;
  k.tok = pb::tok_of(T);
  k.chunks = z.chunks;
  k.wpart = reinterpret_cast<float*>(w + 2 * z.band);
  k.fpart = reinterpret_cast<float*>(w + 2 * z.band + z.wpart);
  k.status = p.status;
  k.wait_ns = a.wait_ns;
  e = cudaFuncSetAttribute(pb::key_pass, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)pb::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_after(pb::key_pass, 2 * std::max(1, sm_count() / 2), pb::kThreads, pb::kSmem, s, qmap,
                   dmap, pw, pf, sw, sf, k);
  if (e != cudaSuccess) return e;
  float* const dsink = b.sink ? b.dsink : nullptr;
  return launch_after(pb::reduce, std::min(T, 148 * 7) + (dsink ? kH : 0), pb::kReduce, 0, s, k, p.scale,
                      static_cast<__nv_bfloat16*>(b.dkey), static_cast<__nv_bfloat16*>(b.dval),
                      spoiled_keys, dsink_part, dsink);
}

}  // namespace hs
