// hs_kv4_mqa_decode on tcgen05 tensor cores (bf16 queries, up to 64 heads per
// pass, fp32 accumulate) over the 4-bit paged cache (format: kv4.cuh).
//
// With s_j = scale <q[b,h], k_j> over the attended cached positions j,
//   lse[b,h] = log(exp(sink_h) + sum_j exp(s_j)),  out[b,h] = sum_j exp(s_j - lse) v_j.
//
// What bounds it: a key costs 308 bytes (Dk 576, values in the same row) and
// 2 * 64 * (576 + 512) operations, 452 per byte, so with 64 heads the tensor
// cores are the limit, not memory.  Every value code * scale has at most 7
// significant bits and is exact in bf16, so keys are turned into bf16 MMA
// operands in shared memory and nothing is lost before the products.
//
// As in the window kernel the products are transposed, so that keys and
// value columns fill M = 128 and the heads are N = 64:
//   S^T [128 keys x heads]  = K_tile (A, K-major) . Q^T
//   O^T [Dv x 64 heads]    += V_tile^T (A, MN-major) . P^T (B, MN-major)
// A 128-byte-swizzled panel of 128 keys x 64 columns is the K-major A of the
// first product and the MN-major A of the second: where the values are the
// first Dv columns of the keys, a tile is expanded once and used by both.
// One tile's panels (9 x 16 KB), Q (72 KB) and P^T (16 KB) do not fit one
// SM's 227 KB together; P^T therefore takes the place of the ninth panel,
// which only S^T reads.  The expansion of tile i + 1 follows PV of tile i
// panel by panel (panels 2c, 2c + 1 once PV chunk c has read them), and QK of
// tile i + 1 follows the expansion, so the three overlap;
// codes of tile i + 1 wait in registers since before the softmax of tile i.
// A value plane of its own is expanded into the panels after QK.
//
// 16 warps expand and compute the softmax (thread = key row of S^T, 16 heads);
// two further warps issue the QK and the PV MMAs.  The running maximum of a
// head is raised only when a logit passes it by more than 2^8, so a tile
// usually needs one vote and no reduction.
//
// Work: the tiles of all sequences in order are cut into equal ranges, one
// per CTA, whatever the lengths; a sequence inside one CTA is finished there,
// one that several CTAs share goes through fp32 partials in the workspace
// and a second kernel that joins them in order (deterministic).  A CTA has at
// most two partial sequences, its first and its last.
// All waits are bounded (HS_ERR_TIMEOUT).
//
// Measured (64 heads, Dk 576 / Dv 512 in one plane, in a graph): 64 sequences of
// ~4900 keys 84 us, 520 TFLOP/s and 1.25 TB/s; 4 sequences of 65536 keys at most 97 us.  A
// tile of 128 keys costs ~6.3K cycles (PV 1.7K, then expansion, QK and softmax
// behind one another in part); ~20 us are prologue, epilogue and the join.
// The CUDA-core kernel takes 353 us for 8 sequences of 2048 keys at most that
// take 23 us here, and 39 us for one of 777 that takes 18.

#include <math.h>

#include "kv4.cuh"
#include "tc_common.cuh"
#include "tc_host.h"

namespace hs {
namespace {

using namespace tc;

constexpr int kWarps = 16;              // expansion and softmax (8: 88 us for 80)
constexpr int kParts = kWarps / 4;    // each part of the warps has 64 / kParts heads
constexpr int kHP = 64 / kParts;
constexpr int kPE = 8 / kParts;       // panels of a thread
constexpr int kWorkers = kWarps * 32;
constexpr int kThreads = kWorkers + 64;  // + QK issuer, PV issuer
constexpr int kTile = 128;             // keys per tile
constexpr int kHG = 64;                // heads per pass
constexpr int kPanel = 16384;          // 128 keys x 64 columns bf16
constexpr int kQChunk = kHG * 128;     // 64 heads x 64 columns bf16
constexpr int kPBytes = kTile * 128;   // P^T: 128 keys x 64 heads bf16
constexpr int kSCol = 256;             // TMEM: O^T in columns 0..255, S^T behind
constexpr int kMaxCtas = 148;          // workspace slots (a constant of the sizes alone)
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleLog2 = 8.f;

struct Params {
  Kv4Decode a;
  int nck, nvp, nvc;   // K panels, V panels, 128-row V chunks
  int groups, ctas;    // head groups, CTAs of one head group
  int panels;          // panels in shared memory
  int qrows;           // heads of a Q box
  int own_p;           // P^T has its own place (else the ninth panel's)
  float scale_log2;
  int* prefix;         // [num_seqs + 1] first tile of each sequence
  float2* part_ml;     // [groups][ctas][2][64] (max in log2 units, sum)
  float* part_o;       // [groups][ctas][2][64][dv]
  long long wait_ns;
};

struct Shared {
  uint64_t kfull[9], vfull[4], pvchunk[4], qfull;
  uint64_t sfull, pfull, drain[2];
  uint64_t rv[kParts], seg;   // the 4 warps of a part meet; all after a segment
  alignas(16) float mrun[kHG];  // read as float4
  float alpha[kHG], inv[kHG];
  float red[kParts][4][kHP];  // [part][warp][head]
  int flag[kParts][2];
  int scan[kWarps];
  int total, seq0, tile0;     // tiles of the batch; this CTA's first sequence and tile in it
  uint32_t tmem_base;
};

__host__ __device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) {
  return total * c / ctas;
}


// Attended keys of sequence b; a length out of range counts as 0.
__device__ __forceinline__ kv4::KeyList seq_keys(const Kv4Decode& a, int b) {
  const int len = __ldg(a.seq_lens + b);
  return kv4::key_list(len < 0 || len > a.max_seqlen ? 0 : len, a.window, a.first);
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// 32 codes and their scale -> 32 bf16 as four 16-byte units of row `row` of a
// panel (128 bytes per row, 128-byte swizzle), units 4 * half ...  A code
// n becomes the bf16 number 128 + n by setting its bits under the exponent of
// 128; (128 + n) s - 136 s is one fma, exact because 136 s = 17 s * 8 still
// fits bf16 (17 * 15 < 2^8).
__device__ __forceinline__ void expand(uint8_t* panel, int row, int half, uint4 codes,
                                       uint32_t byte) {
  const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
  const float sf = kv4::scale_value(byte);
  const __nv_bfloat162 s2 = __float2bfloat162_rn(sf), z2 = __float2bfloat162_rn(-136.f * sf);
  uint8_t* r = panel + row * 128;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t t = ((word[w] >> (4 * k)) & 0x000f000fu) | 0x43004300u;
      const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&t), s2, z2);
      o[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(r + (((4 * half + w) ^ (row & 7)) << 4)) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// This thread's share of a tile of one plane: its key's 64 columns (groups
// 2 pn, 2 pn + 1) of the panels pn = hh + kParts e, and for keys half of the
// ninth panel (group 16 + hh, hh < 2).
struct Codes {
  uint4 c[kPE][2], c8;
  uint32_t s[kPE], s8;  // scale words
};
template <bool kKeys>
__device__ __forceinline__ void load_codes(Codes& d, const uint8_t* cache, int width, int ps_log2,
                                           int page, int slot, int hh) {
  const int G = kv4::groups(width), ps = 1 << ps_log2;
  const uint8_t* pg = cache + (int64_t)page * kv4::page_bytes(width, ps) + slot * 16;
  const uint8_t* sc = pg + G * ps * 16 - slot * 12;
#pragma unroll
  for (int e = 0; e < kPE; ++e) {
    const int pn = hh + kParts * e;
    d.c[e][0] = d.c[e][1] = make_uint4(0u, 0u, 0u, 0u);
    d.s[e] = 0u;
    if (page >= 0 && 2 * pn < G) {
      d.c[e][0] = __ldg(reinterpret_cast<const uint4*>(pg + 2 * pn * ps * 16));
      d.c[e][1] = __ldg(reinterpret_cast<const uint4*>(pg + (2 * pn + 1) * ps * 16));
      d.s[e] = __ldg(reinterpret_cast<const uint32_t*>(sc + (pn >> 1) * ps * 4));
    }
  }
  if (kKeys) {
    d.c8 = make_uint4(0u, 0u, 0u, 0u);
    d.s8 = 0u;
    if (page >= 0 && G == 18 && hh < 2) {
      d.c8 = __ldg(reinterpret_cast<const uint4*>(pg + (16 + hh) * ps * 16));
      d.s8 = __ldg(reinterpret_cast<const uint32_t*>(sc + 4 * ps * 4));
    }
  }
}
// Panel hh + kParts e; its groups' scales are half hh & 1 of their word.
__device__ __forceinline__ void expand_panel(const Codes& d, uint8_t* panels, int r, int e, int hh) {
  uint8_t* pn = panels + (hh + kParts * e) * kPanel;
  const uint32_t two = d.s[e] >> (16 * (hh & 1));
  expand(pn, r, 0, d.c[e][0], two & 0xffu);
  expand(pn, r, 1, d.c[e][1], (two >> 8) & 0xffu);
}

// Lanes 4h .. 4h + 3 receive op over the 32 lanes of v[h].
template <bool kMax>
__device__ __forceinline__ float reduce8(float (&v)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off >= 4; off >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < off / 4; ++j) {
      const float send = upper ? v[j] : v[j + off / 4];
      const float keep = upper ? v[j + off / 4] : v[j];
      const float got = __shfl_xor_sync(0xffffffffu, send, off);
      v[j] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int off = 2; off >= 1; off >>= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], off);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// Bounded wait of a whole warp: all its lanes go on, or all give up.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long lim) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, lim));
}
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity, long long lim) {
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, lim));
}

// Warps meet: one arrival per warp (the 4 of a head half, or all).
__device__ __forceinline__ bool meet(uint64_t* bar, uint32_t& ph, int lane, long long lim) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  const bool ok = warp_wait(bar, ph, lim);
  ph ^= 1;
  return ok;
}

// One arrival per warp, this warp's shared-memory writes made visible to the
// tensor cores, and its TMEM accesses done, first.
__device__ __forceinline__ void publish(uint64_t* bar, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void tmem_ld_heads(uint32_t at, uint32_t (&u)[kHP]) {
  static_assert(kHP == 16, "the heads of a part");
  tmem_ld16(at, u);
}

template <bool kAlias>
__global__ void __launch_bounds__(kThreads, 1)
tc_kv4_decode_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ Params p) {
  // Not aligned by hand: through an integer the compiler loses that the pointer
  // is into shared memory, and every access below became a generic one with a
  // 64-bit address (106 us against 88, and 240 registers wanted).
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {
    record_status(p.a.status, HS_ERR_CUDA);
    return;
  }
  uint8_t* const panels = smem_raw;
  uint8_t* const qbuf = panels + p.panels * kPanel;
  uint8_t* const pown = qbuf + p.nck * kQChunk;
  uint8_t* const pbuf = p.own_p ? pown : panels + 8 * kPanel;
  Shared* sh = reinterpret_cast<Shared*>(pown + (p.own_p ? kPBytes : 0));
  const Kv4Decode& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int group = blockIdx.x % p.groups, cta = blockIdx.x / p.groups;
  const int h0 = group * kHG, hn = min(kHG, a.num_heads - h0);
  const long long lim = p.wait_ns;

  if (tid == 0) {
    for (int i = 0; i < 9; ++i) mbar_init(&sh->kfull[i], i < 8 ? 4 : 8);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh->vfull[i], 8);
      mbar_init(&sh->pvchunk[i], 1);
    }
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sh->rv[i], 4);
      sh->flag[i][0] = sh->flag[i][1] = 0;
    }
    mbar_init(&sh->qfull, 1);
    mbar_init(&sh->sfull, 1);
    mbar_init(&sh->pfull, kWarps);
    mbar_init(&sh->seg, kWarps);
    fence_barrier_init();
  }
  // The sequences' tiles: a worker owns a run of sequences.
  const int per = (a.num_seqs + kWorkers - 1) / kWorkers;
  const int b0 = min(a.num_seqs, tid * per), b1 = tid < kWorkers ? min(a.num_seqs, b0 + per) : b0;
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(seq_keys(a, b).n);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31 && warp < kWarps) sh->scan[warp] = incl;
  if (warp == kWarps) tmem_alloc(&sh->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  int total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp && warp < kWarps) incl += sh->scan[w];
    total += sh->scan[w];
  }
  const int g0 = (int)range_start(total, cta, p.ctas), g1 = (int)range_start(total, cta + 1, p.ctas);
  if (tid < kWorkers) {
    int at = incl - mine;
    const bool out = blockIdx.x == 0;  // the first CTA keeps the offsets for the join
    for (int b = b0; b < b1; ++b) {
      const int n = tiles_of(seq_keys(a, b).n);
      if (out) {
        p.prefix[b] = at;
        const int len = __ldg(a.seq_lens + b);
        if (len < 0 || len > a.max_seqlen) record_status(a.status, HS_ERR_INVALID_ARG);
      }
      if (g0 < g1 && g0 >= at && g0 < at + n) {
        sh->seq0 = b;
        sh->tile0 = g0 - at;
      }
      at += n;
    }
    if (out && tid == 0) p.prefix[a.num_seqs] = total;
  }
  __syncthreads();

  // Segments of [g0, g1): every role walks them alike.
  int left = g1 - g0, b = left > 0 ? sh->seq0 : 0, ta = left > 0 ? sh->tile0 : 0;
  if (warp >= kWarps) {
    // ------------------------------------------------------------ MMA issuers
    if (left > 0) {
      const bool is_pv = warp == kWarps + 1;
      const int nqk = (hn + 15) & ~15;  // heads of S^T
      const uint32_t id_qk = idesc_bf16_f32(kTile, nqk, false, false);
      constexpr uint32_t id_pv = idesc_bf16_f32(128, kHG, true, true);
      const uint64_t k_desc = umma_desc_sw128(smem_u32(panels), 16, 1024);
      const uint64_t q_desc = umma_desc_sw128(smem_u32(qbuf), 16, 1024);
      const uint64_t v_desc = umma_desc_sw128(smem_u32(panels), kPanel, 1024);
      const uint64_t p_desc = umma_desc_sw128(smem_u32(pbuf), kPanel, 1024);
      uint32_t ph = 0, qph = 0;
      bool ok = true;
      for (; left > 0 && ok; ++b, ta = 0) {
        const int tb = min(tiles_of(seq_keys(a, b).n), ta + left);
        for (int i = ta; i < tb && ok; ++i, ph ^= 1) {
          if (!is_pv) {
            if (i == ta && !warp_spin(&sh->qfull, qph, lim)) { ok = false; break; }
            for (int c = 0; c < p.nck; ++c) {
              if (!warp_spin(&sh->kfull[c], ph, lim)) { ok = false; break; }
              tc_fence_after();
              const uint64_t ka = k_desc + (uint64_t)((c * kPanel) >> 4);
              const uint64_t qa = q_desc + (uint64_t)((c * kQChunk) >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_ss_warp(tmem + kSCol, ka + 2 * k, qa + 2 * k, id_qk,
                             (c > 0 || k > 0) ? 1u : 0u);
            }
            if (ok) umma_commit_warp(&sh->sfull);
          } else {
            if (!warp_spin(&sh->pfull, ph, lim)) { ok = false; break; }
            tc_fence_after();
            for (int c = 0; c < p.nvc; ++c) {
              if (!kAlias) {
                if (!warp_spin(&sh->vfull[c], ph, lim)) { ok = false; break; }
                tc_fence_after();
              }
              const uint64_t va = v_desc + (uint64_t)((2 * c * kPanel) >> 4);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_ss_warp(tmem + c * kHG, va + (uint64_t)(k * 128), p_desc + (uint64_t)(k * 128),
                             id_pv, (i > ta || k > 0) ? 1u : 0u);
              umma_commit_warp(&sh->pvchunk[c]);
            }
          }
        }
        if (tb > ta) qph ^= 1;
        left -= tb - ta;
      }
      if (!ok && lane == 0) record_status(a.status, HS_ERR_TIMEOUT);
      umma_commit_warp(&sh->drain[is_pv]);  // every MMA done before TMEM is released
      (void)warp_spin(&sh->drain[is_pv], 0, kDefaultWaitNs);
    }
  } else {
    // ------------------------------------------------------------ expansion, softmax, epilogue
    const int g4 = warp & 3, hh = warp >> 2;  // TMEM lane quarter, part
    const int r = 32 * g4 + lane;             // key row of a tile; row of an O^T chunk
    const int hb = kHP * hh;
    const bool act = hb < hn;                 // this part has heads
    const uint32_t lane_base = tmem + ((uint32_t)(32 * g4) << 16);
    const float sl2 = p.scale_log2;
    uint32_t ph = 0, rvph = 0, segph = 0;     // tile parity; parities of the meetings
    bool ok = true, any_pv = false, first_seg = true;
    Codes kc;
    // The table entry of this thread's key of a tile, loaded a tile ahead and
    // checked where it is used.
    auto entry_at = [&](const kv4::KeyList& kl, int bb, int tile) -> int {
      const int x = tile * kTile + r;
      if (x >= kl.n) return -1;
      const int e = kl.pos(x) >> a.ps_log2;
      return e < a.table_width ? __ldg(a.table + (int64_t)bb * a.table_stride + e) : -1;
    };
    auto checked = [&](const kv4::KeyList& kl, int tile, int page) -> int {
      if ((unsigned)page < (unsigned)a.num_pages) return page;
      if (tile * kTile + r < kl.n) record_status(a.status, HS_ERR_INVALID_INDEX);
      return -1;
    };
    auto slot_of = [&](const kv4::KeyList& kl, int tile) {
      return kl.pos(tile * kTile + r) & ((1 << a.ps_log2) - 1);
    };
    for (; left > 0 && ok; ++b, ta = 0) {
      const kv4::KeyList kl = seq_keys(a, b);
      const int nt = tiles_of(kl.n), tb = min(nt, ta + left);
      if (tb == ta) continue;  // an empty sequence
      if (tid == 0) {  // Q (every QK of the sequence before is complete)
        mbar_expect_tx(&sh->qfull, p.nck * p.qrows * 128);
        for (int c = 0; c < p.nck; ++c)
          tma_load_3d(qbuf + c * kQChunk, &qmap, &sh->qfull, c * 64, h0, b);
      }
      int page = entry_at(kl, b, ta), next = ta + 1 < tb ? entry_at(kl, b, ta + 1) : -1;
      page = checked(kl, ta, page);
      load_codes<true>(kc, a.k_cache, a.dk, a.ps_log2, page, slot_of(kl, ta), hh);
      float lpart[kHP];
#pragma unroll
      for (int k = 0; k < kHP; ++k) lpart[k] = 0.f;
      for (int i = ta; i < tb && ok; ++i) {
        // ---- this part's K panels, each once PV of the tile before has read it
#pragma unroll
        for (int e = 0; e < kPE; ++e) {
          const int pn = hh + kParts * e;
          if (pn >= p.nck) break;
          const int c = min(pn >> 1, p.nvc - 1);
          if (any_pv && !warp_wait(&sh->pvchunk[c], ph ^ 1, lim)) { ok = false; break; }
          expand_panel(kc, panels, r, e, hh);
          publish(&sh->kfull[pn], lane);
        }
        if (!ok) break;
        if (p.nck == 9 && hh < 2) {  // half of the ninth panel, where P^T was
          if (any_pv && !warp_wait(&sh->pvchunk[p.nvc - 1], ph ^ 1, lim)) { ok = false; break; }
          expand(panels + 8 * kPanel, r, hh, kc.c8, (kc.s8 >> (8 * hh)) & 0xffu);
          publish(&sh->kfull[8], lane);
        }
        // ---- codes ahead: the next tile's keys, or this tile's values
        if (!kAlias) {
          load_codes<false>(kc, a.v_cache, a.dv, a.ps_log2, page, slot_of(kl, i), hh);
        } else if (i + 1 < tb) {
          page = checked(kl, i + 1, next);
          load_codes<true>(kc, a.k_cache, a.dk, a.ps_log2, page, slot_of(kl, i + 1), hh);
          if (i + 2 < tb) next = entry_at(kl, b, i + 2);
        }
        // ---- softmax: row r of S^T, heads hb .. hb + kHP - 1
        if (!warp_wait(&sh->sfull, ph, lim)) { ok = false; break; }
        // PV of the tile before has read P^T (and V) and added to O^T
        if (any_pv && !warp_wait(&sh->pvchunk[p.nvc - 1], ph ^ 1, lim)) { ok = false; break; }
        tc_fence_after();
        const bool first = i == ta;
        if (act) {
          uint32_t u[kHP];
          tmem_ld_heads(lane_base + kSCol + hb, u);
          tmem_ld_wait();
          reg_fence(u);
          const bool valid = i * kTile + r < kl.n;
          const float4* const mr = reinterpret_cast<const float4*>(sh->mrun + hb);
          float x[kHP];
          float most = -INFINITY;  // above the running maximum
#pragma unroll
          for (int k = 0; k < kHP; ++k) x[k] = valid ? __uint_as_float(u[k]) * sl2 : -INFINITY;
#pragma unroll
          for (int k = 0; k < kHP / 4; ++k) {
            const float4 m = mr[k];
            most = fmaxf(most, fmaxf(fmaxf(x[4 * k] - m.x, x[4 * k + 1] - m.y),
                                     fmaxf(x[4 * k + 2] - m.z, x[4 * k + 3] - m.w)));
          }
          bool over = first || most > kRescaleLog2;
          const int par = i & 1;
          if (!first) {
            if (__any_sync(0xffffffffu, over) && lane == 0) sh->flag[hh][par] = 1;
            if (g4 == 0 && lane == 0) sh->flag[hh][par ^ 1] = 0;
            if (!meet(&sh->rv[hh], rvph, lane, lim)) { ok = false; break; }
            over = *reinterpret_cast<volatile int*>(&sh->flag[hh][par]) != 0;
          } else if (g4 == 0 && lane == 0) {
            sh->flag[hh][0] = sh->flag[hh][1] = 0;  // read next after two meetings
          }
          if (over) {
            // the tile's maximum per head joins the running one (from TMEM
            // again, 8 heads at a time: rare, and small in code and registers)
#pragma unroll 1
            for (int k = 0; k < kHP; k += 8) {
              uint32_t w[8];
              tmem_ld8(lane_base + kSCol + hb + k, w);
              tmem_ld_wait();
              reg_fence(w);
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = valid ? __uint_as_float(w[e]) * sl2 : -INFINITY;
              const float wm = reduce8<true>(y);
              if (!(lane & 3)) sh->red[hh][g4][k + (lane >> 2)] = wm;
            }
            if (!meet(&sh->rv[hh], rvph, lane, lim)) { ok = false; break; }
            if (g4 == 0 && lane < kHP) {
              const float tm = fmaxf(fmaxf(sh->red[hh][0][lane], sh->red[hh][1][lane]),
                                     fmaxf(sh->red[hh][2][lane], sh->red[hh][3][lane]));
              const float mo = first ? -INFINITY : sh->mrun[hb + lane];
              const float mn = first || tm > mo + kRescaleLog2 ? tm : mo;
              sh->alpha[hb + lane] = first || mn == mo ? 1.f : fast_exp2(mo - mn);
              sh->mrun[hb + lane] = mn;
            }
            if (!meet(&sh->rv[hh], rvph, lane, lim)) { ok = false; break; }
            if (!first) {
#pragma unroll
              for (int k = 0; k < kHP; ++k) lpart[k] *= sh->alpha[hb + k];
#pragma unroll 1
              for (int c = 0; c < p.nvc * (kHP / 8); ++c) {
                const int k = 8 * (c % (kHP / 8));
                const uint32_t at = lane_base + (c / (kHP / 8)) * kHG + hb + k;
                uint32_t w[8];
                tmem_ld8(at, w);
                tmem_ld_wait();
                reg_fence(w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  w[e] = __float_as_uint(__uint_as_float(w[e]) * sh->alpha[hb + k + e]);
                tmem_st8(at, w);
              }
              tmem_st_wait();
            }
          }
          uint8_t* prow = pbuf + r * 128;
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < kHP / 4; ++k) {
            // every logit so far -inf: exp2(-inf - 0) = 0
            float4 m = mr[k];
            m.x = m.x == -INFINITY ? 0.f : m.x;
            m.y = m.y == -INFINITY ? 0.f : m.y;
            m.z = m.z == -INFINITY ? 0.f : m.z;
            m.w = m.w == -INFINITY ? 0.f : m.w;
            const float e0 = fast_exp2(x[4 * k] - m.x), e1 = fast_exp2(x[4 * k + 1] - m.y);
            const float e2 = fast_exp2(x[4 * k + 2] - m.z), e3 = fast_exp2(x[4 * k + 3] - m.w);
            lpart[4 * k] += e0;
            lpart[4 * k + 1] += e1;
            lpart[4 * k + 2] += e2;
            lpart[4 * k + 3] += e3;
            __nv_bfloat162 p0 = __floats2bfloat162_rn(e0, e1), p1 = __floats2bfloat162_rn(e2, e3);
            pk[2 * (k & 1)] = *reinterpret_cast<uint32_t*>(&p0);
            pk[2 * (k & 1) + 1] = *reinterpret_cast<uint32_t*>(&p1);
            if (k & 1)
              *reinterpret_cast<uint4*>(prow + (((kHP / 8 * hh + (k >> 1)) ^ (r & 7)) << 4)) =
                  make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        publish(&sh->pfull, lane);
        if (!kAlias) {
          // ---- the value plane's panels (QK has read the keys there)
#pragma unroll
          for (int e = 0; e < kPE; ++e) {
            const int pn = hh + kParts * e;
            if (pn >= 2 * p.nvc) break;
            if (pn < p.nvp) expand_panel(kc, panels, r, e, hh);
            publish(&sh->vfull[pn >> 1], lane);
          }
          if (i + 1 < tb) {
            page = checked(kl, i + 1, next);
            load_codes<true>(kc, a.k_cache, a.dk, a.ps_log2, page, slot_of(kl, i + 1), hh);
            if (i + 2 < tb) next = entry_at(kl, b, i + 2);
          }
        }
        any_pv = true;
        ph ^= 1;
      }
      if (!ok) break;
      // ---- the segment's sums and output
      const bool whole = ta == 0 && tb == nt;
      const int64_t slot2 = ((int64_t)group * p.ctas + cta) * 2 + (first_seg ? 0 : 1);
      if (act) {
#pragma unroll
        for (int k = 0; k < kHP; k += 8) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = lpart[k + e];
          const float ws = reduce8<false>(y);
          if (!(lane & 3)) sh->red[hh][g4][k + (lane >> 2)] = ws;
        }
        if (!meet(&sh->rv[hh], rvph, lane, lim)) { ok = false; break; }
        const int h = h0 + hb + lane;
        if (g4 == 0 && lane < kHP && hb + lane < hn) {
          const float l = (sh->red[hh][0][lane] + sh->red[hh][1][lane]) +
                          (sh->red[hh][2][lane] + sh->red[hh][3][lane]);
          const float m = sh->mrun[hb + lane];
          if (whole) {
            const float sk = a.sink ? __ldg(a.sink + h) * kLog2e : -INFINITY;
            const float M = fmaxf(m, sk), Ms = M == -INFINITY ? 0.f : M;
            const float em = m == -INFINITY ? 0.f : fast_exp2(m - Ms);
            const float den = l * em + fast_exp2(sk - Ms);
            sh->inv[hb + lane] = den == 0.f ? 0.f : em / den;
            a.lse[(int64_t)b * a.num_heads + h] = den == 0.f ? -INFINITY : (Ms + fast_log2(den)) * kLn2;
          } else {
            sh->inv[hb + lane] = 1.f;
            p.part_ml[slot2 * kHG + hb + lane] = make_float2(m, l);
          }
        }
        if (!meet(&sh->rv[hh], rvph, lane, lim)) { ok = false; break; }
        if (!warp_wait(&sh->pvchunk[p.nvc - 1], ph ^ 1, lim)) { ok = false; break; }
        tc_fence_after();
        // rows of a chunk = consecutive d: a warp stores 32 of one head at a time
        const int hc = min(kHP, hn - hb);
        __nv_bfloat16* const ob = static_cast<__nv_bfloat16*>(a.out) +
                                  ((int64_t)b * a.num_heads + h0 + hb) * a.dv + r;
        float* const op = p.part_o + (slot2 * kHG + hb) * a.dv + r;
#pragma unroll 1
        for (int c = 0; c < p.nvc; ++c) {
          uint32_t w[kHP];
          tmem_ld_heads(lane_base + c * kHG + hb, w);
          tmem_ld_wait();
          reg_fence(w);
          if (c * 128 + r >= a.dv) continue;
          if (whole) {
            __nv_bfloat16* o = ob + c * 128;
#pragma unroll
            for (int k = 0; k < kHP; ++k, o += a.dv)
              if (k < hc) *o = __float2bfloat16_rn(__uint_as_float(w[k]) * sh->inv[hb + k]);
          } else {
            float* o = op + c * 128;
#pragma unroll
            for (int k = 0; k < kHP; ++k, o += a.dv)
              if (k < hc) *o = __uint_as_float(w[k]);
          }
        }
        tc_fence_before();  // the next segment's first PV follows this thread's P^T
      }
      left -= tb - ta;
      first_seg = false;
      // Q and the sums are rewritten only after every warp is here
      if (!meet(&sh->seg, segph, lane, lim)) ok = false;
    }
    if (!ok) record_status(a.status, HS_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarps) tmem_dealloc(tmem, 512);
}

// Joins the partials of a sequence that several CTAs share, and serves empty
// sequences.  One block per (sequence, 8 heads).
__global__ void __launch_bounds__(256) tc_kv4_join_kernel(const __grid_constant__ Params p) {
  const Kv4Decode& a = p.a;
  cudaGridDependencySynchronize();  // launched while the decode kernel still runs
  const int b = blockIdx.x, h = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int gs = p.prefix[b], ge = p.prefix[b + 1], total = p.prefix[a.num_seqs];
  if (h >= a.num_heads) return;
  const int64_t bh = (int64_t)b * a.num_heads + h;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + bh * a.dv;
  const float sink = a.sink ? __ldg(a.sink + h) : -INFINITY;
  if (gs == ge) {
    for (int d = lane; d < a.dv; d += 32) out[d] = __float2bfloat16_rn(0.f);
    if (lane == 0) a.lse[bh] = sink;
    return;
  }
  // the CTAs of tiles gs and ge - 1: the last one that starts at or before
  auto owner = [&](int g) {
    int c = (int)((int64_t)g * p.ctas / total);
    while (c + 1 < p.ctas && range_start(total, c + 1, p.ctas) <= g) ++c;
    while (c > 0 && range_start(total, c, p.ctas) > g) --c;
    return c;
  };
  const int c0 = owner(gs), c1 = owner(ge - 1);
  if (c0 == c1) return;  // finished by its CTA
  const int group = h / kHG, hh = h % kHG;
  auto slot = [&](int c) -> int64_t {  // -1: a CTA without tiles
    const int64_t s0 = range_start(total, c, p.ctas);
    if (s0 == range_start(total, c + 1, p.ctas)) return -1;
    return (((int64_t)group * p.ctas + c) * 2 + (s0 >= gs ? 0 : 1)) * kHG + hh;
  };
  // lane j holds the weight of CTA base + j
  const float sk = sink * kLog2e;
  float M = sk;
  for (int c = c0 + lane; c <= c1; c += 32) {
    const int64_t s = slot(c);
    if (s >= 0) M = fmaxf(M, p.part_ml[s].x);
  }
  M = warp_max(M);
  const float Ms = M == -INFINITY ? 0.f : M;
  float den = 0.f;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = c0; base <= c1; base += 32) {
    const int64_t s = base + lane <= c1 ? slot(base + lane) : -1;
    float w = 0.f;
    if (s >= 0) {
      const float2 ml = p.part_ml[s];
      w = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - Ms);
      den = fmaf(ml.y, w, den);
    }
    const int n = min(32, c1 - base + 1);
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int64_t sj = __shfl_sync(0xffffffffu, s, j);
      if (sj < 0) continue;
      const float* src = p.part_o + sj * a.dv + lane * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (lane * 4 + q * 128 >= a.dv) continue;
        const float4 v = *reinterpret_cast<const float4*>(src + q * 128);
        o[q].x = fmaf(wj, v.x, o[q].x);
        o[q].y = fmaf(wj, v.y, o[q].y);
        o[q].z = fmaf(wj, v.z, o[q].z);
        o[q].w = fmaf(wj, v.w, o[q].w);
      }
    }
  }
  den = warp_sum(den) + fast_exp2(sk - Ms);
  const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int d = lane * 4 + q * 128;
    if (d >= a.dv) continue;
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out + d);
    dst[0] = __floats2bfloat162_rn(o[q].x * inv, o[q].y * inv);
    dst[1] = __floats2bfloat162_rn(o[q].z * inv, o[q].w * inv);
  }
  if (lane == 0) a.lse[bh] = den == 0.f ? -INFINITY : (Ms + fast_log2(den)) * kLn2;
}

size_t align16(size_t n) { return (n + 15) & ~(size_t)15; }
int head_groups(int num_heads) { return (num_heads + kHG - 1) / kHG; }

}  // namespace

bool tc_kv4_decode_shape_ok(int num_heads, int dk, int dv, hs_dtype dtype) {
  return dtype == HS_BF16 && num_heads >= 1 && num_heads <= 128 && dk % 64 == 0 && dk >= 64 &&
         dk <= 576 && dv % 64 == 0 && dv >= 64 && dv <= 512;
}

bool tc_kv4_decode_eligible(const Kv4Decode& a) {
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  return tc_kv4_decode_shape_ok(a.num_heads, a.dk, a.dv, a.dtype) && al16(a.q) && al16(a.out) &&
         a.q_row_stride % 8 == 0 && a.q_head_stride % 8 == 0;
}

size_t tc_kv4_decode_workspace(int num_seqs, int num_heads, int dv) {
  const size_t slots = (size_t)head_groups(num_heads) * (kMaxCtas / head_groups(num_heads)) * 2 * kHG;
  return align16(sizeof(int) * ((size_t)num_seqs + 1)) + slots * (sizeof(float2) + sizeof(float) * dv);
}

cudaError_t launch_tc_kv4_decode(const Kv4Decode& a, long long wait_limit, cudaStream_t s) {
  Params p{};
  p.a = a;
  p.nck = a.dk / 64;
  p.nvp = a.dv / 64;
  p.nvc = (p.nvp + 1) / 2;
  p.panels = p.nck > 2 * p.nvc ? p.nck : 2 * p.nvc;
  p.own_p = p.nck < 9;
  p.groups = head_groups(a.num_heads);
  // no more CTAs than tiles the longest sequences could have
  const int64_t keys = a.window > 0 && (int64_t)a.window + a.first < a.max_seqlen
                           ? (int64_t)a.window + a.first
                           : a.max_seqlen;
  const int64_t most = (int64_t)a.num_seqs * ((keys + kTile - 1) / kTile);
  int64_t ctas = (sm_count() < kMaxCtas ? sm_count() : kMaxCtas) / p.groups;
  if (ctas > most) ctas = most;
  p.ctas = (int)ctas;
  p.scale_log2 = a.scale * kLog2e;
  uint8_t* w = static_cast<uint8_t*>(a.workspace);
  p.prefix = reinterpret_cast<int*>(w);
  w += align16(sizeof(int) * ((size_t)a.num_seqs + 1));
  const size_t slots = (size_t)p.groups * p.ctas * 2 * kHG;
  p.part_ml = reinterpret_cast<float2*>(w);
  p.part_o = reinterpret_cast<float*>(w + slots * sizeof(float2));
  p.wait_ns = wait_limit > 0 ? wait_limit : kDefaultWaitNs;
  CUtensorMap qmap;
  {
    p.qrows = a.num_heads < kHG ? a.num_heads : kHG;
    const uint64_t dims[3] = {(uint64_t)a.dk, (uint64_t)a.num_heads, (uint64_t)a.num_seqs};
    const uint64_t strides[2] = {(uint64_t)a.q_head_stride * 2, (uint64_t)a.q_row_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)p.qrows, 1};
    if (!encode_bf16_map(&qmap, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const size_t bytes = (size_t)p.panels * kPanel + (size_t)p.nck * kQChunk +
                       (p.own_p ? kPBytes : 0) + sizeof(Shared);
  auto kern = a.v_cache ? tc_kv4_decode_kernel<false> : tc_kv4_decode_kernel<true>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  kern<<<p.ctas * p.groups, kThreads, bytes, s>>>(qmap, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.num_seqs, (a.num_heads + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tc_kv4_join_kernel, p);
}

}  // namespace hs
