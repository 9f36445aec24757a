// hs_swa_first_mqa_fwd on tcgen05 tensor cores (bf16 in, fp32 accumulate), 64
// query heads over one KV head.
//
//   S_t = { j <= t : j >= max(bos, t - window + 1) or j < bos + first },
//   lse[t,h] = log(exp(sink_h) + sum_{j in S_t} exp(s_j)),
//   out[t,h] = sum_{j in S_t} exp(s_j - lse[t,h]) v_j.
//
// What bounds it: 2 * 64 * |S_t| (Dk + Dv) operations per token, so the tensor
// cores if their operands arrive.  A token's 64 heads are the only rows with
// one key set, and its O (64 x 512 fp32) is half of an SM's TMEM: one token per
// SM is all that fits beside two S buffers, and each SM would read every key
// and value of the window for itself.  Neighbouring tokens' windows differ by
// one key, so two tokens run on a pair of CTAs (tc_pair.cuh) over the union of
// their keys: M = 128 rows are token t0's heads in one CTA and t0 + 1's in the
// other, each CTA loads half of every K tile (by keys) and of every V tile (by
// columns), and the halves are read by both.
//   S [128 x N keys]  = Q . K_tile^T          (A, B K-major)
//   O [128 x 256 dv] += P . V_tile            (A K-major, B MN-major)
// With rows as M a row's logits lie in one lane: its maximum and sum need no
// shuffles, only the four threads that share a row exchange a value per tile.
//
// Keys: the window's union first, padded to 16 rows, then the first tokens
// before it, in tiles of 256; the last tile has as many (a multiple of 32) as
// are left.  Padding and keys that only the other token sees are masked.
// A masked value row still meets P = 0 in the product, and 0 * NaN is NaN: a
// row whose result is not finite is marked by a NaN lse and computed again by
// launch_simt_redo, which reads nothing but the key set.
//
// Roles per CTA: K and V producers, 8 softmax warps, 4 epilogue warps; in the
// leader the QK and the PV issuer.  S is double-buffered, so QK of tile i + 1
// runs beside the softmax of tile i, and the output of a pass leaves while the
// next one begins.  The running maximum is raised only past 2^8.
// All waits are bounded (HS_ERR_TIMEOUT).
//
// Measured (Dk 576 / Dv 512, window 512 + 4 first, in a graph, full clock): 4096 tokens
// 280 us, 986 TFLOP/s, 0.60 of a cuBLAS matmul's rate (327 us and 0.60 of that rate in
// a long run under the power cap); the window kernel with one token per CTA
// (tc_attention.cu) takes 376 us for its 512 keys.  What bounds it is the operands'
// way from L2 (11 TB/s into the SMs, 112 KB of ring under way per SM) and the ~85
// cycles between two MMAs of one issuing warp.  Dk 192 / Dv 128, window 1024 + 64:
// 8192 tokens 491 us, 666 TFLOP/s, bound by the softmax (3.7K cycles a tile, a third
// of it exponentials).  The CUDA-core kernel takes 18.5 ms for 512 tokens that take
// 37 us here, and 21 us for 8 that take 10.

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

constexpr int kThreads = 512;  // 8 softmax warps; K and V producers, QK and PV issuers; 4 epilogue warps
constexpr int kStage = 2048;            // per epilogue warp: 32 rows x 32 columns bf16
constexpr int kKProd = 8, kVProd = 9, kQkWarp = 10, kPvWarp = 11;
constexpr int kKSlots = 3, kVSlots = 2;
constexpr int kKSlot = 16384;           // 128 keys x 64 columns
constexpr int kVSlot = 32768;           // two panels of 128 keys x 64 columns
constexpr int kPBytes = 4 * kPPanel;    // 64 rows x 256 keys
constexpr int kSCol = 256;              // two S buffers of 128 columns
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kRescaleLog2 = 8.f;

struct Params {
  Docs d;
  int nck;            // 64-column chunks of K
  int nvb;            // 128-column blocks of V (the last may be half past Dv)
  int dv;
  float scale_log2;
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  int* status;
  long long wait_ns;
};

struct Shared {
  uint64_t kfull[kKSlots], kempty[kKSlots], vfull[kVSlots], vempty[kVSlots];
  uint64_t qfull[kMaxQC], qempty[kMaxQC];
  uint64_t sfull[2], sempty[2], pfull, pvdone, oempty, drain[2], rv;
  // A pass's sums are there, by pass parity: the softmax warps may be through the next
  // pass before an epilogue warp looks, and one barrier, two phases on, would look as if
  // the first had not come.  Two passes on is impossible: PV of pass n + 1 waits for
  // oempty of pass n, and pass n + 2 for that PV.
  uint64_t stat[2];
  // What a row's four threads exchange, maxima and a pass's sums in turn.  An
  // exchange writes one half, meets and reads it; the next one, of whichever pass,
  // takes the other half, so a half is written again only after a meeting that
  // every reader of it reached.
  float red[2][4][kH];
  float inv[2][kH];  // by pass parity
  uint32_t tmem_base;
};
constexpr size_t kSmem = (size_t)kKSlots * kKSlot + (size_t)kVSlots * kVSlot +
                         (size_t)kMaxQC * kQChunk + kPBytes + 4 * kStage + sizeof(Shared);
static_assert(kSmem <= 232448, "shared memory of one CTA");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
tc_first_fwd_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap kmap16,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap vmap16,
                    const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // no room to align it by hand
  if (smem_u32(smem_raw) & 1023) {
    record_status(p.status, HS_ERR_CUDA);
    return;  // every thread of both CTAs alike
  }
  uint8_t* const kring = smem_raw;
  uint8_t* const vring = kring + kKSlots * kKSlot;
  uint8_t* const qbuf = vring + kVSlots * kVSlot;
  uint8_t* const pbuf = qbuf + kMaxQC * kQChunk;
  uint8_t* const stage = pbuf + kPBytes;
  Shared* sh = reinterpret_cast<Shared*>(stage + 4 * kStage);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;
  const long long lim = p.wait_ns;

  if (tid == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&sh->kfull[i], 1);
      mbar_init(&sh->kempty[i], 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&sh->vfull[i], 1);
      mbar_init(&sh->vempty[i], 1);
    }
    for (int i = 0; i < kMaxQC; ++i) {
      mbar_init(&sh->qfull[i], 1);
      mbar_init(&sh->qempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->sfull[i], 1);
      mbar_init(&sh->sempty[i], 16);  // 8 warps of each CTA
      mbar_init(&sh->drain[i], 1);
    }
    mbar_init(&sh->pfull, 16);
    mbar_init(&sh->pvdone, 1);
    mbar_init(&sh->oempty, 8);  // 4 epilogue warps of each CTA
    mbar_init(&sh->rv, 8);
    mbar_init(&sh->stat[0], 8);
    mbar_init(&sh->stat[1], 8);
    fence_barrier_init();
  }
  if (warp == kQkWarp) tmem_alloc_pair(&sh->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs exist
  tc_fence_after();
  cudaTriggerProgrammaticLaunchCompletion();  // the check of the rows waits for the end
  const uint32_t tmem = sh->tmem_base;
  // registers: 512 threads launch with 128 each; 8 softmax warps take 168 and
  // the other two warpgroups give 48 each (8 * 168 + 8 * 80 <= 16 * 128)
  Walk walk(p.d, blockIdx.x >> 1, gridDim.x >> 1);
  Pass ps;
  bool ok = true;

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    // ------------------------------------------------------------ softmax
    // Thread: TMEM lane 32 g4 + lane = (half of the tile's keys, row = head),
    // columns 64 ch .. of that half; part = which of the row's four threads.
    const int g4 = warp & 3, ch = warp >> 2, hi = g4 >> 1, part = 2 * hi + ch;
    const int row = 32 * (g4 & 1) + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
    const float sl2 = p.scale_log2;
    uint32_t sidx = 0, npv = 0, rvph = 0, npass = 0;  // rvph: parity of the exchange, for red too
    auto meet = [&]() -> bool {  // the 8 warps of this CTA
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->rv);
      const bool good = warp_wait(&sh->rv, rvph, lim);
      rvph ^= 1;
      return good;
    };
    auto tell_leader = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_leader(bar);
    };
    // PV of the tile before has read P and added to O
    auto pv_before = [&]() -> bool {
      return npv == 0 || warp_wait(&sh->pvdone, (npv - 1) & 1, lim);
    };
    while (ok && walk.next(ps, nullptr)) {
      const bool act = ps.active(rank);
      const Mask mk = ps.mask(rank, p.d.window, p.d.first);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < ps.ntile && ok; ++i) {
        const int n2 = ps.keys(i) / 2;  // columns of a lane half
        const int col0 = 64 * ch;
        const uint32_t buf = sidx & 1;
        if (!warp_wait(&sh->sfull[buf], (sidx >> 1) & 1, lim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // x: raw scores (scale joins in the exponential's fma)
        float x[2][32];
        float mx = -INFINITY;
        const int slot0 = 256 * i + hi * n2 + col0;  // of x[0][0]
        if (act) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (col0 + 32 * e >= n2) break;
            uint32_t u[32];
            tmem_ld32(lane_base + kSCol + buf * 128 + col0 + 32 * e, u);
            tmem_ld_wait();
            reg_fence(u);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[e][k] = __uint_as_float(u[k]);
          }
        }
        ++sidx;
        tell_leader(&sh->sempty[buf]);
        if (act) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (col0 + 32 * e >= n2) break;
            const uint32_t bits =
                mk.bits(slot0 + 32 * e) & low_bits(n2 - col0 - 32 * e);
            if (bits != 0xffffffffu) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(bits & (1u << k))) x[e][k] = -INFINITY;
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 32; k += 4)
#pragma unroll
              for (int j = 0; j < 4; ++j) m4[j] = fmaxf(m4[j], x[e][k + j]);
            mx = fmaxf(fmaxf(mx, fmaxf(m4[0], m4[1])), fmaxf(m4[2], m4[3]));
          }
          mx *= sl2;
          float(*const red)[kH] = sh->red[rvph];
          red[part][row] = mx;
          if (!meet()) { ok = false; break; }
          const float mt = fmaxf(fmaxf(red[0][row], red[1][row]), fmaxf(red[2][row], red[3][row]));
          const float mn = mt > m + kRescaleLog2 ? mt : m;  // m = -inf: any logit raises it
          const float alpha = mn == m ? 1.f : fast_exp2(m - mn);
          m = mn;
          l *= alpha;
          const float ms = m == -INFINITY ? 0.f : m;  // no key yet: exp2(-inf) = 0
          uint32_t pk[2][16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (col0 + 32 * e >= n2) break;
            float la = 0.f, lb = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float e0 = fast_exp2(fmaf(x[e][2 * k], sl2, -ms));
              const float e1 = fast_exp2(fmaf(x[e][2 * k + 1], sl2, -ms));
              la += e0;
              lb += e1;
              __nv_bfloat162 pr = __floats2bfloat162_rn(e0, e1);
              pk[e][k] = *reinterpret_cast<uint32_t*>(&pr);
            }
            l += la + lb;
          }
          if (!pv_before()) { ok = false; break; }
          tc_fence_after();
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // this row's O: 64 columns of each 128 in TMEM
#pragma unroll 1
            for (int c = 0; c < p.nvb * 64; c += 32) {
              if (((c >> 5) & 1) != ch) continue;
              uint32_t w[32];
              tmem_ld32(lane_base + c, w);
              tmem_ld_wait();
              reg_fence(w);
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * alpha);
              tmem_st32(lane_base + c, w);
            }
            tmem_st_wait();
          }
          const int key0 = hi * n2 + col0;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (col0 + 8 * q >= n2) break;
            const int key = key0 + 8 * q;
            const uint32_t* w = pk[q >> 2] + 4 * (q & 3);
            *reinterpret_cast<uint4*>(pbuf + (key >> 6) * kPPanel + row * 128 +
                                      ((((key >> 3) & 7) ^ (row & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        } else if (!pv_before()) {  // no arrival for a tile before the last one's is used
          ok = false;
          break;
        }
        ++npv;
        tell_leader(&sh->pfull);
      }
      if (!ok) break;
      // ---- the row's sum over its four threads and the sink, for the epilogue
      if (act) {
        float(*const red)[kH] = sh->red[rvph];
        red[part][row] = l;
        if (!meet()) { ok = false; break; }
        if (part == 0) {
          const float lt = (red[0][row] + red[1][row]) + (red[2][row] + red[3][row]);
          const float sk = p.sink ? __ldg(p.sink + row) * kLog2e : -INFINITY;
          const float M = fmaxf(m, sk), Ms = M == -INFINITY ? 0.f : M;
          const float em = m == -INFINITY ? 0.f : fast_exp2(m - Ms);
          const float den = lt * em + fast_exp2(sk - Ms);
          sh->inv[npass & 1][row] = den == 0.f ? 0.f : em / den;
          p.lse[(int64_t)ps.token(rank) * kH + row] =
              den == 0.f ? -INFINITY : (Ms + fast_log2(den)) * kLn2;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->stat[npass & 1]);
      ++npass;
    }
    if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kKProd || warp == kVProd) {
      // ------------------------------------------------------------ producers
      const bool is_v = warp == kVProd;
      uint64_t* const fullb = is_v ? sh->vfull : sh->kfull;
      uint64_t* const emptyb = is_v ? sh->vempty : sh->kempty;
      uint8_t* const ring = is_v ? vring : kring;
      const int slots = is_v ? kVSlots : kKSlots, slot_bytes = is_v ? kVSlot : kKSlot;
      const CUtensorMap* const big = is_v ? &vmap : &kmap;
      const CUtensorMap* const small = is_v ? &vmap16 : &kmap16;
      int slot = 0;
      uint32_t ph = 0, qph = 0;
      bool first_pass = true;
      // a free slot, armed by the leader for both CTAs' bytes
      auto claim = [&](int bytes) -> bool {
        if (!warp_wait(&emptyb[slot], ph ^ 1, lim)) return false;
        if (leader && lane == 0) mbar_expect_tx(&fullb[slot], 2 * bytes);
        __syncwarp();
        return true;
      };
      auto next = [&]() {
        if (++slot == slots) {
          slot = 0;
          ph ^= 1;
        }
      };
      while (ok && walk.next(ps, leader && !is_v ? p.status : nullptr)) {
        if (!is_v) {  // Q chunks, each once the pass before has read it
          for (int c = 0; c < p.nck && ok; ++c) {
            if (!first_pass && !warp_wait(&sh->qempty[c], qph ^ 1, lim)) { ok = false; break; }
            if (lane == 0) {
              if (leader) mbar_expect_tx(&sh->qfull[c], 2 * kQChunk);
              tma_pair_3d(qbuf + c * kQChunk, &qmap, leader_addr(&sh->qfull[c]), c * 64, 0,
                          ps.token(rank));
            }
            __syncwarp();
          }
          first_pass = false;
          qph ^= 1;
        }
        for (int i = 0; i < ps.ntile && ok; ++i) {
          const int n = ps.keys(i);
          if (!is_v) {
            const int s0 = 256 * i + rank * (n / 2), rows = n / 2;
            const int per = 128 / rows;  // chunks of a slot: more where a tile has fewer keys
            for (int c = 0; c < p.nck && ok; c += per, next()) {
              const int cnt = min(per, p.nck - c);
              if (!claim(cnt * rows * 128)) { ok = false; break; }
              load_rows(ps, big, small, ring + slot * slot_bytes, leader_addr(&fullb[slot]), s0, rows,
                        c * 64, lane, cnt, rows * 128);
            }
          } else {
            for (int b = 0; b < p.nvb && ok; b += 2) {
              // 256 columns: 128 (two panels) of each CTA; a last odd block: 64 of each
              const int panels = b + 1 < p.nvb ? 2 : 1;
              const int col = b * 128 + rank * panels * 64;
              for (int k0 = 0; k0 < n && ok; k0 += 128, next()) {
                const int rows = min(128, n - k0);
                if (!claim(rows * 128 * panels)) { ok = false; break; }
                load_rows(ps, big, small, ring + slot * slot_bytes, leader_addr(&fullb[slot]),
                          256 * i + k0, rows, col, lane, panels, 16384);
              }
            }
          }
        }
      }
      if (!ok) {
        // The leader's barriers count both CTAs' copies and its issuers wait for
        // all of them; after a timeout they do not, so copies still under way get
        // a millisecond to land before the CTA may exit.
        if (lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
        for (const uint64_t from = global_ns(); global_ns() - from < 1000000;) {
        }
      }
    } else if (warp == kQkWarp || warp == kPvWarp) {
      // ------------------------------------------------------------ MMA issuers
      if (leader) {
        const bool is_pv = warp == kPvWarp;
        const uint64_t k_desc = umma_desc_sw128(smem_u32(kring), 16, 1024);
        const uint64_t q_desc = umma_desc_sw128(smem_u32(qbuf), 16, 1024);
        const uint64_t v_desc = umma_desc_sw128(smem_u32(vring), 16384, 1024);
        const uint64_t p_desc = umma_desc_sw128(smem_u32(pbuf), 16, 1024);
        int slot = 0;
        uint32_t ph = 0, sidx = 0, npv = 0, npass = 0;
        while (ok && walk.next(ps, nullptr)) {
          for (int i = 0; i < ps.ntile && ok; ++i) {
            const int n = ps.keys(i);
            if (!is_pv) {
              const uint32_t id = idesc_bf16_f32(128, n, false, false);
              const uint32_t buf = sidx & 1, d = tmem + kSCol + buf * 128;
              if (!warp_wait(&sh->sempty[buf], ((sidx >> 1) & 1) ^ 1, lim)) { ok = false; break; }
              tc_fence_after();
              const int rows = n / 2, per = 128 / rows;
              for (int c0 = 0; c0 < p.nck; c0 += per) {
                if (!warp_wait(&sh->kfull[slot], ph, lim)) { ok = false; break; }
                tc_fence_after();
                for (int c = c0; c < min(p.nck, c0 + per); ++c) {
                  if (i == 0 && !warp_wait(&sh->qfull[c], npass & 1, lim)) { ok = false; break; }
                  const uint64_t a = q_desc + (uint64_t)((c * kQChunk) >> 4);
                  const uint64_t b = k_desc + (uint64_t)((slot * kKSlot + (c - c0) * rows * 128) >> 4);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    umma_pair(d, a + 2 * k, b + 2 * k, id, (c > 0 || k > 0) ? 1u : 0u);
                  if (i + 1 == ps.ntile) commit_pair(&sh->qempty[c]);
                }
                commit_pair(&sh->kempty[slot]);
                if (++slot == kKSlots) {
                  slot = 0;
                  ph ^= 1;
                }
              }
              if (!ok) break;
              commit_pair(&sh->sfull[buf]);
              ++sidx;
            } else {
              if (!warp_wait(&sh->pfull, npv & 1, lim) ||
                  (i == 0 && npass > 0 && !warp_wait(&sh->oempty, (npass - 1) & 1, lim))) {
                ok = false;
                break;
              }
              tc_fence_after();
              for (int b = 0; b < p.nvb && ok; b += 2) {
                const uint32_t id = idesc_bf16_f32(128, b + 1 < p.nvb ? 256 : 128, false, true);
                for (int k0 = 0; k0 < n; k0 += 128) {
                  if (!warp_wait(&sh->vfull[slot], ph, lim)) { ok = false; break; }
                  tc_fence_after();
                  const uint64_t v = v_desc + (uint64_t)((slot * kVSlot) >> 4);
                  const uint64_t a = p_desc + (uint64_t)(((k0 >> 6) * kPPanel) >> 4);
                  const int steps = min(128, n - k0) / 16;
                  if (steps == 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                      umma_pair(tmem + b * 64, a + (uint64_t)(((k >> 2) * kPPanel) >> 4) + 2 * (k & 3),
                                v + (uint64_t)(k * 128), id, (i > 0 || k0 > 0 || k > 0) ? 1u : 0u);
                  } else {
                    for (int k = 0; k < steps; ++k)
                      umma_pair(tmem + b * 64, a + (uint64_t)(((k >> 2) * kPPanel) >> 4) + 2 * (k & 3),
                                v + (uint64_t)(k * 128), id, (i > 0 || k0 > 0 || k > 0) ? 1u : 0u);
                  }
                  commit_pair(&sh->vempty[slot]);
                  if (++slot == kVSlots) {
                    slot = 0;
                    ph ^= 1;
                  }
                }
              }
              if (!ok) break;
              commit_pair(&sh->pvdone);
              ++npv;
            }
          }
          ++npass;
        }
        if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
        commit_pair(&sh->drain[is_pv]);  // every MMA done before TMEM is released
        (void)warp_wait(&sh->drain[is_pv], 0, kDefaultWaitNs);
      }
    } else {
      // ------------------------------------------------------------ epilogue
      // Thread: TMEM lane 32 g4 + lane, all its columns.  O is normalised,
      // turned in this warp's 2 KB of shared memory and stored 64 bytes of a
      // row at a time, while the softmax warps are in the next pass.
      const int g4 = warp & 3, hi = g4 >> 1, row0 = 32 * (g4 & 1);
      const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
      uint8_t* const st = stage + g4 * kStage;
      uint32_t npass = 0, npv = 0;
      while (ok && walk.next(ps, nullptr)) {
        npv += ps.ntile;
        if (!warp_wait(&sh->stat[npass & 1], (npass >> 1) & 1, lim) ||
            !warp_wait(&sh->pvdone, (npv - 1) & 1, lim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (ps.active(rank)) {
          const int64_t th = (int64_t)ps.token(rank) * kH + row0;
          const float inv = sh->inv[npass & 1][row0 + lane];
          float finite = 0.f;
#pragma unroll 1
          for (int c = 0; c < p.nvb * 64; c += 32) {
            // TMEM column -> Dv column: blocks of 256 split over the lane halves
            const int b = c >> 7, wide = 2 * b + 1 < p.nvb ? 128 : 64;
            const int d = 256 * b + hi * wide + (c - 128 * b);
            uint32_t w[32];
            tmem_ld32(lane_base + c, w);
            tmem_ld_wait();
            reg_fence(w);
            if (d >= p.dv) continue;
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __uint_as_float(w[8 * q + 2 * k]) * inv;
                const float c1 = __uint_as_float(w[8 * q + 2 * k + 1]) * inv;
                finite = fmaf(a, 0.f, fmaf(c1, 0.f, finite));  // NaN from NaN and infinities
                __nv_bfloat162 pr = __floats2bfloat162_rn(a, c1);
                v[k] = *reinterpret_cast<uint32_t*>(&pr);
              }
              // unit q of row `lane`: 8 rows' units fall into 8 different bank groups
              *reinterpret_cast<uint4*>(st + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int rr = 8 * j + (lane >> 2), q = lane & 3;
              *reinterpret_cast<uint4*>(p.out + (th + rr) * p.dv + d + 8 * q) =
                  *reinterpret_cast<const uint4*>(st + rr * 64 + ((q ^ ((rr >> 1) & 3)) << 4));
            }
          }
          // a row that is not finite: launch_simt_redo computes it again
          if (finite != 0.f) p.lse[th + lane] = __int_as_float(0x7fffffff);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh->oempty);
        ++npass;
      }
      if (!ok && lane == 0) record_status(p.status, HS_ERR_TIMEOUT);
    }
  }
  // neither CTA leaves, or frees TMEM, while the other's MMAs and copies may
  // still touch it
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc_pair(tmem, 512);
}

}  // namespace

bool tc_first_shape_ok(hs_dtype dtype, int num_heads, int dk, int dv) {
  return dtype == HS_BF16 && num_heads == kH && dk % 64 == 0 && dk >= 64 && dk <= 64 * kMaxQC &&
         dv % 64 == 0 && dv >= 64 && dv <= 512;
}

bool tc_first_eligible(const Problem& p) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return tc_first_shape_ok(p.dtype, p.num_heads, p.dk, p.dv) && al16(p.q) && al16(p.k) &&
         al16(p.v) && p.q_row_stride % 8 == 0 && p.q_head_stride % 8 == 0 &&
         p.k_row_stride % 8 == 0 && p.v_row_stride % 8 == 0;
}

cudaError_t launch_tc_first_fwd(const AttnArgs& a, long long wait_limit, cudaStream_t s) {
  const Problem& p = a.p;
  CUtensorMap kmap, kmap16, vmap, vmap16, qmap;
  if (!row_map(&kmap, p.k, p.dk, p.total_tokens, p.k_row_stride, 128) ||
      !row_map(&kmap16, p.k, p.dk, p.total_tokens, p.k_row_stride, 16) ||
      !row_map(&vmap, p.v, p.dv, p.total_tokens, p.v_row_stride, 128) ||
      !row_map(&vmap16, p.v, p.dv, p.total_tokens, p.v_row_stride, 16) ||
      !head_map(&qmap, p.q, p.dk, p.total_tokens, p.q_row_stride, p.q_head_stride))
    return cudaErrorInvalidValue;
  Params ap;
  ap.d = docs_of(p, a.window, a.first);
  ap.nck = p.dk / 64;
  ap.nvb = (p.dv + 127) / 128;
  ap.dv = p.dv;
  ap.scale_log2 = p.scale * kLog2e;
  ap.sink = a.sink;
  ap.out = static_cast<__nv_bfloat16*>(a.out);
  ap.lse = a.lse;
  ap.status = p.status;
  ap.wait_ns = wait_limit > 0 ? wait_limit : kDefaultWaitNs;
  cudaError_t e = cudaFuncSetAttribute(
      tc_first_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  tc_first_fwd_kernel<<<pair_grid(p.total_tokens), kThreads, kSmem, s>>>(kmap, kmap16, vmap, vmap16,
                                                                        qmap, ap);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_simt_redo(a, s);
}

}  // namespace hs
