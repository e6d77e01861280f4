// Split kernel of tq_paged_decode_attn (instantiated per key width in tq_paged_split_k*.cu).
//
// Work.  The tokens a sequence shows (all, or a window's) are cut into groups of 16, which never cross
// a page.  The groups of all units -- a unit is one (sequence, kv-head) and up to eight of its query
// heads -- are laid end to end and cut into one even, contiguous range per CTA, so ragged batches
// load every SM alike.  The cut follows from the lengths on the device: every CTA sums them itself.
// A range is processed as segments, each inside one unit; a segment ends with one (max, sum, o')
// partial per head, which the merge kernel joins.
//
// CTA.  One producer warp and NW consumer warps.  The producer walks the segments: it looks up the
// pages of a stage (one group per consumer warp) one stage ahead, and moves each run of groups inside
// a page with one bulk copy per cache array into a ring of shared-memory slots, and each segment's
// query operands (built by the prep kernel) into a double buffer, all completing on mbarriers.  It
// needs no query, so the ring fills while the prep kernel still runs (programmatic dependent
// launch).  A consumer warp turns 16 tokens of every stage into tensor-core operands:
//   scores   D[16 tokens x 8] += A[tokens x dims] B[dims x (4 heads, fp16 hi and lo)]: A are centroid
//            pairs from a lane-replicated shared-memory table; a second product with the sign bits
//            placed in fp16 mantissas gives the QJL term
//   values   O'^T[16 dims x 8] += A[dims x tokens] B[tokens x (4 heads, hi and lo)]: A are centroid
//            pairs of two tokens, B the weights p ||v|| / sqrt(128)
// with online softmax in log2 units in between.  q' and the weights enter as fp16 hi + lo (about 22
// bits), sums are fp32.  Rows outside the tokens shown are masked by selection, never by a product,
// so whatever they hold (NaN too) stays out.
#pragma once

#include <algorithm>

#include "tq_decode_core.h"
#include "tq_paged.h"

namespace tq {
namespace {

template <int NB>
struct PShape {
  // Registers split between the SM's four schedulers: 12 warps leave 168 a thread, enough for one
  // n-block of four heads; two n-blocks need up to 255 and run with 8 warps.
  static constexpr int NW = NB == 1 ? 11 : 7;
  static constexpr int THREADS = 32 * (NW + 1);
};
constexpr int P_NS_MAX = 8;
constexpr long long P_WAIT_LIMIT = 4000000000LL;  // ~2 s of SM clock per wait

// What the producer tells the consumers of a segment.
struct Seg {
  int32_t n;         // groups; 0: the range is done
  int32_t tok0;      // first token of the first group
  int32_t first, len;  // tokens shown: [first, len)
  int64_t slot;      // partial record
};

struct PCtrl {
  uint64_t full[P_NS_MAX], empty[P_NS_MAX];
  uint64_t sfull[2], sempty[2];
  Seg seg[2];
  uint32_t stage_off[P_NS_MAX];
  uint32_t tbl_addr, seg_off, merge_off;
  int ns;
  unsigned int err;
};
constexpr int P_CTRL_BYTES = 384;
static_assert(sizeof(PCtrl) <= P_CTRL_BYTES, "control block");

template <int KB, int VB, bool QJL, int NB>
struct PLayout {
  static constexpr int NW = PShape<NB>::NW, ST = 16 * NW, HGN = 4 * NB;
  static constexpr int K_ROW = 16 * KB, V_ROW = 16 * VB;
  static constexpr int OFF_KC = 0;
  static constexpr int OFF_SG = OFF_KC + ST * K_ROW;
  static constexpr int OFF_VC = OFF_SG + (QJL ? ST * 16 : 0);
  static constexpr int OFF_NK = OFF_VC + ST * V_ROW;
  static constexpr int OFF_RN = OFF_NK + ST * 4;
  static constexpr int OFF_NV = OFF_RN + (QJL ? ST * 4 : 0);
  static constexpr int STAGE_BYTES = (OFF_NV + ST * 4 + 127) / 128 * 128;
  static constexpr int TX_PER_TOKEN = K_ROW + V_ROW + 8 + (QJL ? 20 : 0);
  static constexpr bool kPacked = KB == 4 && VB == 4;
  static constexpr int K_TBL = kPacked ? 0 : (1 << (2 * KB)) * 128;
  static constexpr int V_TBL = kPacked ? 0 : (1 << (2 * VB)) * 128;
  static constexpr int TBL_BYTES = kPacked ? 65536 : K_TBL + V_TBL;
  static constexpr int SEG_BYTES = seg_bytes(NB);            // a segment's operands, twice
  // warps' partials of a segment, one n-block at a time: (max, sum) and o' of four heads per warp
  static constexpr int MERGE_BYTES = 4 * (NW * 4 * 2 + NW * 4 * D);
  static_assert(STAGE_BYTES % 16 == 0 && OFF_NK % 16 == 0 && OFF_RN % 16 == 0 && OFF_NV % 16 == 0, "bulk copies");
};

// Shared memory: pair tables (at a 64 KB boundary of the window when packed), then first-fit around
// them the segment operands, the merge area and as many ring slots as fit.
template <int KB, int VB, bool QJL, int NB>
__device__ void place_smem(uint32_t base, int dyn, PCtrl& c) {
  using Lay = PLayout<KB, VB, QJL, NB>;
  const uint32_t end = base + (uint32_t)dyn - P_CTRL_BYTES;
  const uint32_t tbl = Lay::kPacked ? ((base + 0xFFFFu) & ~0xFFFFu) : base;
  uint32_t r0 = base, r1 = tbl + Lay::TBL_BYTES;
  auto take = [&](uint32_t bytes, uint32_t& off) {
    bytes = (bytes + 127u) & ~127u;
    if (tbl - r0 >= bytes) {
      off = r0 - base;
      r0 += bytes;
      return true;
    }
    if (r1 <= end && end - r1 >= bytes) {
      off = r1 - base;
      r1 += bytes;
      return true;
    }
    return false;
  };
  c.tbl_addr = tbl;
  c.ns = 0;
  if (r1 > end || !take(Lay::MERGE_BYTES, c.merge_off) || !take(2 * Lay::SEG_BYTES, c.seg_off)) return;
  int ns = 0;
  while (ns < P_NS_MAX && take(Lay::STAGE_BYTES, c.stage_off[ns])) ++ns;
  c.ns = ns >= 2 ? ns : 0;
}

__device__ __forceinline__ bool pwait(PCtrl& c, uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  const long long t0 = clock64();
  while (true) {
    if (__any_sync(FULL, mbar_try(addr, parity))) return true;
    const bool stop = (*reinterpret_cast<volatile unsigned int*>(&c.err) & 3u) != 0 || clock64() - t0 > P_WAIT_LIMIT;
    if (__any_sync(FULL, stop)) {
      if ((threadIdx.x & 31) == 0) atomicOr(&c.err, 1u);
      return false;
    }
  }
}
template <int NW>
__device__ __forceinline__ void pconsumers_sync() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(NW * 32) : "memory");
}

template <int KB, int VB, bool QJL, int NB>
__global__ void __launch_bounds__(PShape<NB>::THREADS, 1) paged_split(const __grid_constant__ PagedArgs a) {
  using Lay = PLayout<KB, VB, QJL, NB>;
  using Lut = PairLut<KB, VB>;
  constexpr int NW = Lay::NW, HGN = Lay::HGN;
  extern __shared__ __align__(1024) unsigned char smem[];
  PCtrl& ctl = *reinterpret_cast<PCtrl*>(smem + a.dyn_smem - P_CTRL_BYTES);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    place_smem<KB, VB, QJL, NB>(smem_u32(smem), a.dyn_smem, ctl);
    ctl.err = ctl.ns ? 0u : 2u;
    for (int i = 0; i < ctl.ns; ++i) {
      mbar_init_(&ctl.full[i], 1);
      mbar_init_(&ctl.empty[i], NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init_(&ctl.sfull[i], 1);
      mbar_init_(&ctl.sempty[i], NW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __syncthreads();
  const int ns = ctl.ns;
  if (ns == 0) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (tid == 0) atomicOr(a.err, 2u);
    return;
  }

  if (warp == NW) {
    // ================================================================ producer
    const int U = a.Hkv * a.hgroups;  // units of a sequence
    // groups of sequence b, and the tokens shown
    auto shown = [&](int b, int& first, int& len) -> int {
      return seq_groups(a.lens[b], a.max_tokens, a.window, first, len);
    };
    int64_t mine = 0;
    bool bad = false;
#pragma unroll 8
    for (int b = lane; b < a.B; b += 32) {
      int first, len;
      mine += shown(b, first, len);
      bad = bad || a.lens[b] < 0 || a.lens[b] > a.max_tokens;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(FULL, mine, o);
    if (__any_sync(FULL, bad) && lane == 0) atomicOr(&ctl.err, 16u);
    const int64_t N = mine * U;
    const int C = active_ctas(N, gridDim.x);
    int64_t f = range_start(N, C, blockIdx.x);
    const int64_t f_end = (int)blockIdx.x < C ? range_start(N, C, blockIdx.x + 1) : f;
    // the sequence that holds group f: lane i keeps the groups of sequence b0 + i
    int b0 = 0, b = 0, G = 0, first = 0, len = 0, uu = 0, gi = 0;
    int lg = 0, lfirst = 0, llen = 0;  // this lane's sequence of the current 32
    auto load32 = [&](int base) {
      b0 = base;
      lg = 0;
      if (base + lane < a.B) lg = shown(base + lane, lfirst, llen);
    };
    auto pick = [&](int bb) {
      b = bb;
      G = __shfl_sync(FULL, lg, bb - b0);
      first = __shfl_sync(FULL, lfirst, bb - b0);
      len = __shfl_sync(FULL, llen, bb - b0);
    };
    if (f < f_end) {
      const int64_t t = f / U;
      int64_t before = 0;
      for (int base = 0; base < a.B; base += 32) {
        load32(base);
        int64_t incl = lg;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(FULL, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned m = __ballot_sync(FULL, before + incl > t);
        if (m) {
          const int l = __ffs(m) - 1;
          pick(base + l);
          before += __shfl_sync(FULL, incl, l) - G;
          break;
        }
        before += __shfl_sync(FULL, incl, 31);
      }
      const int64_t rem = f - before * U;
      uu = (int)(rem / G);
      gi = (int)(rem - (int64_t)uu * G);
    }
    int it = 0, issued = 0, slot = 0, round = 0, si = 0;
    bool prep_done = false;
    while (true) {
      const bool done = f >= f_end;
      const int n = done ? 0 : (int)min((int64_t)(G - gi), f_end - f);
      const int64_t unit = (int64_t)b * U + uu;
      // ---- the segment's stages.  Its operands come from the prep kernel, so with the first segment
      // the ring fills before the wait for that kernel.
      const int64_t rowh = (int64_t)(uu / a.hgroups) * a.ps;  // kv-head's rows of a page
      const int tok0 = 16 * (first / 16 + gi);
      auto page_of = [&](int s0) -> int {  // page of this lane's group of stage s0 (-1: none)
        if (lane >= NW || s0 + lane >= n) return -1;
        return a.table[(int64_t)b * a.table_stride + (tok0 + 16 * (s0 + lane)) / a.ps];
      };
      auto open_segment = [&]() {
        if (!prep_done) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        prep_done = true;
        const int k = si & 1;
        if (si >= 2 && !pwait(ctl, &ctl.sempty[k], ((si >> 1) - 1) & 1)) return;
        if (lane == 0) {
          ctl.seg[k].n = n;
          ctl.seg[k].tok0 = tok0;
          ctl.seg[k].first = first;
          ctl.seg[k].len = len;
          ctl.seg[k].slot = gi == 0 ? unit : (int64_t)a.B * U + blockIdx.x;
          if (done) mbar_arrive_(&ctl.sfull[k]);
          else {
            mbar_expect_tx_(&ctl.sfull[k], Lay::SEG_BYTES);
            bulk_g2s(smem + ctl.seg_off + k * Lay::SEG_BYTES, a.ops + unit * (Lay::SEG_BYTES / 4), Lay::SEG_BYTES, &ctl.sfull[k]);
          }
        }
        __syncwarp();
      };
      if (done) {
        open_segment();
        break;
      }
      bool opened = false;
      if (prep_done) {
        open_segment();
        opened = true;
      }
      int page = page_of(0);
      int stages = 0;
      for (int s0 = 0; s0 < n; s0 += NW, ++it, ++stages) {
        const int cur = slot, cur_round = round;
        if (++slot == ns) {
          slot = 0;
          ++round;
        }
        if (!opened && stages == ns) {  // the ring is full: now the operands are needed
          open_segment();
          opened = true;
        }
        if (cur_round > 0 && !pwait(ctl, &ctl.empty[cur], (cur_round - 1) & 1)) continue;
        if (*reinterpret_cast<volatile unsigned int*>(&ctl.err) & 3u) continue;
        const int here = page;
        page = page_of(s0 + NW);
        const int cnt = min(NW, n - s0);
        const int t = tok0 + 16 * (s0 + lane);
        const int at = t % a.ps;
        const unsigned lead = __ballot_sync(FULL, lane < cnt && (lane == 0 || at == 0));
        if (lane == 0) mbar_expect_tx_(&ctl.full[cur], (uint32_t)(16 * cnt * Lay::TX_PER_TOKEN));
        __syncwarp();
        if ((lead >> lane) & 1u) {
          const unsigned rest = lane < 31 ? lead >> (lane + 1) : 0u;
          const int run = rest ? __ffs(rest) : cnt - lane;  // groups up to the next page
          int p = here;
          if ((unsigned)p >= (unsigned)a.pages) {  // a bad table entry: recorded, page 0 read instead
            atomicOr(&ctl.err, 16u);
            p = 0;
          }
          const int64_t row = (int64_t)p * a.Hkv * a.ps + rowh + at;
          unsigned char* st = smem + ctl.stage_off[cur];
          const uint32_t i = 16u * lane, rows = 16u * run;
          bulk_g2s(st + Lay::OFF_KC + i * Lay::K_ROW, a.k_codes + row * Lay::K_ROW, rows * Lay::K_ROW, &ctl.full[cur]);
          if constexpr (QJL) {
            bulk_g2s(st + Lay::OFF_SG + i * 16, a.k_signs + row * 16, rows * 16, &ctl.full[cur]);
            bulk_g2s(st + Lay::OFF_RN + i * 4, a.k_rnorm + row, rows * 4, &ctl.full[cur]);
          }
          bulk_g2s(st + Lay::OFF_VC + i * Lay::V_ROW, a.v_codes + row * Lay::V_ROW, rows * Lay::V_ROW, &ctl.full[cur]);
          bulk_g2s(st + Lay::OFF_NK + i * 4, a.k_norm + row, rows * 4, &ctl.full[cur]);
          bulk_g2s(st + Lay::OFF_NV + i * 4, a.v_norm + row, rows * 4, &ctl.full[cur]);
        }
        __syncwarp();
        issued = it + 1;
      }
      if (!opened) open_segment();
      ++si;
      f += n;
      // ---- the next unit
      gi = 0;
      if (++uu == U && f < f_end) {
        uu = 0;
        int nb = b + 1;
        while (true) {  // (f < f_end: some later sequence has groups)
          if (nb >= b0 + 32) load32(b0 + 32);
          const unsigned m = __ballot_sync(FULL, lg > 0) & (nb - b0 == 0 ? FULL : ~((1u << (nb - b0)) - 1u));
          if (m) {
            pick(b0 + __ffs(m) - 1);
            break;
          }
          nb = b0 + 32;
          if (nb >= a.B) break;
        }
      }
    }
    // every copy issued has landed before the CTA may exit (bounded)
    for (int j = max(0, issued - ns); j < issued; ++j) {
      const uint32_t addr = smem_u32(&ctl.full[j % ns]);
      const long long t0 = clock64();
      while (!__all_sync(FULL, mbar_try(addr, (j / ns) & 1)) && clock64() - t0 < P_WAIT_LIMIT) {
      }
    }
    if (si > 0) {  // the last segment's operands (its buffer is not the one the closing message used)
      const uint32_t addr = smem_u32(&ctl.sfull[(si - 1) & 1]);
      const long long t0 = clock64();
      while (!__all_sync(FULL, mbar_try(addr, ((si - 1) >> 1) & 1)) && clock64() - t0 < P_WAIT_LIMIT) {
      }
    }
    return;
  }

  // ================================================================ consumers
  // pair tables: entry e = lo | hi << b -> half2(c[lo], c[hi]), four lane replicas per 16-byte store
  Lut lut;
  {
    float* cbs = reinterpret_cast<float*>(smem + ctl.merge_off);
    if (tid < 16) cbs[tid] = tid < (1 << KB) ? a.kc[tid] : 0.0f;
    else if (tid < 32) cbs[tid] = tid - 16 < (1 << VB) ? a.vc[tid - 16] : 0.0f;
    pconsumers_sync<NW>();
    const uint32_t tbl = ctl.tbl_addr;
    unsigned char* tp = smem + (tbl - smem_u32(smem));
    if constexpr (Lut::kPacked) {
      for (int i = tid; i < 256 * 2 * 8; i += NW * 32) {  // (entry, half, group of four lanes)
        const int e = i >> 4, half = (i >> 3) & 1, q4 = i & 7;
        const float* cb = cbs + 16 * half;
        const uint32_t v = pack_half2(cb[e & 15], cb[e >> 4]);
        *reinterpret_cast<uint4*>(tp + e * 256 + half * 128 + 16 * q4) = make_uint4(v, v, v, v);
      }
      lut.rk = tbl | (4u * lane);
      lut.rv = tbl | 128u | (4u * lane);
    } else {
      for (int i = tid; i < (Lay::K_TBL + Lay::V_TBL) / 16; i += NW * 32) {
        const bool isv = i >= Lay::K_TBL / 16;
        const int e = (isv ? i - Lay::K_TBL / 16 : i) >> 3;
        const int bits = isv ? VB : KB;
        const float* cb = cbs + (isv ? 16 : 0);
        const uint32_t v = pack_half2(cb[e & ((1 << bits) - 1)], cb[e >> bits]);
        *reinterpret_cast<uint4*>(tp + 16 * i) = make_uint4(v, v, v, v);
      }
      lut.rk = tbl + 4u * lane;
      lut.rv = tbl + Lay::K_TBL + 4u * lane;
    }
    pconsumers_sync<NW>();
  }

  const int gq = lane >> 2, t = lane & 3;
  int slot = 0;
  uint32_t phase = 0;
  for (int si = 0;; ++si) {
    const int k = si & 1;
    if (!pwait(ctl, &ctl.sfull[k], (si >> 1) & 1)) break;
    const int n = ctl.seg[k].n;
    if (n == 0) break;
    const int tok0 = ctl.seg[k].tok0, first = ctl.seg[k].first, len = ctl.seg[k].len;
    const int64_t pslot = ctl.seg[k].slot;
    uint32_t bq[NB][8][2], bsq[NB][8][2];
    float fK[NB], fQ[NB], Kh[NB];
    {
      const unsigned char* seg = smem + ctl.seg_off + k * Lay::SEG_BYTES;
      const uint4* fp = reinterpret_cast<const uint4*>(seg) + lane;
      const float4* hc = reinterpret_cast<const float4*>(seg + NB * 4096);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int w4 = 0; w4 < 8; ++w4) {
          const uint4 v = fp[(nb * 8 + w4) * 32];
          const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int word = 4 * w4 + j;
            if (word < 16) bq[nb][word >> 1][word & 1] = wv[j];
            else bsq[nb][(word >> 1) & 7][word & 1] = wv[j];
          }
        }
        const float4 h = hc[4 * nb + t];
        fK[nb] = h.x;
        fQ[nb] = h.y;
        Kh[nb] = h.z;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_(&ctl.sempty[k]);

    // Output accumulators: n-block nb, dim block db: (dim 16db + gq, head 4nb + t) hi/lo in [0]/[1],
    // (dim 16db + 8 + gq) in [2]/[3].
    float oacc[NB][8][4];
    float m_run[NB], l_run[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 8; ++i) oacc[nb][i][0] = oacc[nb][i][1] = oacc[nb][i][2] = oacc[nb][i][3] = 0.0f;
      m_run[nb] = -1e30f;  // finite: ex2(s - m) and ex2(m_old - m_new) never see inf - inf
      l_run[nb] = 0.0f;
    }

    for (int s0 = 0; s0 < n; s0 += NW) {
      const bool ok = pwait(ctl, &ctl.full[slot], phase);
      if (ok && s0 + warp < n) {
        const unsigned char* stage = smem + ctl.stage_off[slot];
        const int r0 = 16 * warp + gq, r1 = r0 + 8;  // this lane's token rows in the stage
        const int tk = tok0 + 16 * (s0 + warp) + gq;
        const bool v0ok = tk >= first && tk < len, v1ok = tk + 8 >= first && tk + 8 < len;

        VPairs<VB> p01, p89;
        // Value codes of rows 2t, 2t+1, 2t+8, 2t+9 of the warp's 16, paired for the value MMAs (with
        // 4-bit values and one n-block before the score MMAs, whose latency they then fill).
        constexpr bool EARLY_V = VB == 4 && NB == 1;
        auto load_vpairs = [&]() {
          const unsigned char* vbase = stage + Lay::OFF_VC + (16 * warp) * Lay::V_ROW;
          uint64_t cv0, cv1, cv2, cv3;
          if constexpr (VB == 4) {
            // lanes with odd t read their odd row first: two bank groups instead of one
            const int sw = t & 1;
            const uint2 a0 = lds64(vbase + (2 * t + sw) * Lay::V_ROW + 8 * gq);
            const uint2 a1 = lds64(vbase + (2 * t + 1 - sw) * Lay::V_ROW + 8 * gq);
            const uint2 a2 = lds64(vbase + (2 * t + 8 + sw) * Lay::V_ROW + 8 * gq);
            const uint2 a3 = lds64(vbase + (2 * t + 9 - sw) * Lay::V_ROW + 8 * gq);
            const uint64_t x0 = (uint64_t)a0.x | ((uint64_t)a0.y << 32), x1 = (uint64_t)a1.x | ((uint64_t)a1.y << 32);
            const uint64_t x2 = (uint64_t)a2.x | ((uint64_t)a2.y << 32), x3 = (uint64_t)a3.x | ((uint64_t)a3.y << 32);
            cv0 = sw ? x1 : x0;
            cv1 = sw ? x0 : x1;
            cv2 = sw ? x3 : x2;
            cv3 = sw ? x2 : x3;
          } else {
            cv0 = load_v_chunk<VB>(vbase + (2 * t) * Lay::V_ROW, gq);
            cv1 = load_v_chunk<VB>(vbase + (2 * t + 1) * Lay::V_ROW, gq);
            cv2 = load_v_chunk<VB>(vbase + (2 * t + 8) * Lay::V_ROW, gq);
            cv3 = load_v_chunk<VB>(vbase + (2 * t + 9) * Lay::V_ROW, gq);
          }
          p01.build(cv0, cv1);
          p89.build(cv2, cv3);
        };
        if constexpr (EARLY_V) load_vpairs();

        // ---- scores of tokens r0, r1 and heads 4nb + t; two accumulators per product
        float kacc[NB][4], qacc[NB][4], kacc2[NB][4], qacc2[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) kacc[nb][e] = qacc[nb][e] = kacc2[nb][e] = qacc2[nb][e] = 0.0f;
        {
          uint32_t c0[KB], c1[KB];
          const unsigned char* k0 = stage + Lay::OFF_KC + r0 * Lay::K_ROW + 4 * KB * t;
          const unsigned char* k1 = stage + Lay::OFF_KC + r1 * Lay::K_ROW + 4 * KB * t;
          if constexpr (KB == 4) {
            const uint4 x0 = lds128(k0), x1 = lds128(k1);
            c0[0] = x0.x; c0[1] = x0.y; c0[2] = x0.z; c0[3] = x0.w;
            c1[0] = x1.x; c1[1] = x1.y; c1[2] = x1.z; c1[3] = x1.w;
          } else if constexpr (KB == 2) {
            const uint2 x0 = lds64(k0), x1 = lds64(k1);
            c0[0] = x0.x; c0[1] = x0.y;
            c1[0] = x1.x; c1[1] = x1.y;
          } else {
#pragma unroll
            for (int i = 0; i < KB; ++i) {
              c0[i] = reinterpret_cast<const uint32_t*>(k0)[i];
              c1[i] = reinterpret_cast<const uint32_t*>(k1)[i];
            }
          }
#define TQ_KSTEP(KK)                                                                         \
          {                                                                                  \
            const uint32_t A[4] = {k_pair<KB, VB, 2 * (KK)>(lut, c0), k_pair<KB, VB, 2 * (KK)>(lut, c1), \
                                   k_pair<KB, VB, 2 * (KK) + 1>(lut, c0),                    \
                                   k_pair<KB, VB, 2 * (KK) + 1>(lut, c1)};                   \
            _Pragma("unroll") for (int nb = 0; nb < NB; ++nb)                                \
                mma16816((KK) & 1 ? kacc2[nb] : kacc[nb], A, bq[nb][KK][0], bq[nb][KK][1]);    \
          }
          TQ_KSTEP(0) TQ_KSTEP(1) TQ_KSTEP(2) TQ_KSTEP(3) TQ_KSTEP(4) TQ_KSTEP(5) TQ_KSTEP(6) TQ_KSTEP(7)
#undef TQ_KSTEP
        }
        if constexpr (QJL) {
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(stage + Lay::OFF_SG + r0 * 16 + 4 * t);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(stage + Lay::OFF_SG + r1 * 16 + 4 * t);
#define TQ_SSTEP(KK)                                                                         \
          {                                                                                  \
            const uint32_t A[4] = {sgn<2 * (KK)>(w0), sgn<2 * (KK)>(w1), sgn<2 * (KK) + 1>(w0), \
                                   sgn<2 * (KK) + 1>(w1)};                                   \
            _Pragma("unroll") for (int nb = 0; nb < NB; ++nb)                                \
                mma16816((KK) & 1 ? qacc2[nb] : qacc[nb], A, bsq[nb][KK][0], bsq[nb][KK][1]);  \
          }
          TQ_SSTEP(0) TQ_SSTEP(1) TQ_SSTEP(2) TQ_SSTEP(3) TQ_SSTEP(4) TQ_SSTEP(5) TQ_SSTEP(6) TQ_SSTEP(7)
#undef TQ_SSTEP
        }

        // ---- online softmax (log2 units) per head 4nb + t over the warp's 16 tokens
        const float nk0 = *reinterpret_cast<const float*>(stage + Lay::OFF_NK + 4 * r0);
        const float nk1 = *reinterpret_cast<const float*>(stage + Lay::OFF_NK + 4 * r1);
        float rn0 = 0.0f, rn1 = 0.0f;
        if constexpr (QJL) {
          rn0 = *reinterpret_cast<const float*>(stage + Lay::OFF_RN + 4 * r0);
          rn1 = *reinterpret_cast<const float*>(stage + Lay::OFF_RN + 4 * r1);
        }
        constexpr float VSC = 0.08838834764831845f;  // 1 / sqrt(128)
        const float nv0 = v0ok ? *reinterpret_cast<const float*>(stage + Lay::OFF_NV + 4 * r0) * VSC : 0.0f;
        const float nv1 = v1ok ? *reinterpret_cast<const float*>(stage + Lay::OFF_NV + 4 * r1) * VSC : 0.0f;
        uint32_t bp[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float s0v = ((kacc[nb][0] + kacc2[nb][0]) + (kacc[nb][1] + kacc2[nb][1])) * (nk0 * fK[nb]);
          float s1v = ((kacc[nb][2] + kacc2[nb][2]) + (kacc[nb][3] + kacc2[nb][3])) * (nk1 * fK[nb]);
          if constexpr (QJL) {
            s0v = fmaf(((qacc[nb][0] + qacc2[nb][0]) + (qacc[nb][1] + qacc2[nb][1])) + Kh[nb], rn0 * fQ[nb], s0v);
            s1v = fmaf(((qacc[nb][2] + qacc2[nb][2]) + (qacc[nb][3] + qacc2[nb][3])) + Kh[nb], rn1 * fQ[nb], s1v);
          }
          s0v = v0ok ? s0v : -INFINITY;
          s1v = v1ok ? s1v : -INFINITY;
          float mx = fmaxf(s0v, s1v);
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
          if (mx > m_run[nb]) {  // uniform over the 8 lanes of head 4nb + t
            const float alpha = ex2(m_run[nb] - mx);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              oacc[nb][i][0] *= alpha;
              oacc[nb][i][1] *= alpha;
              oacc[nb][i][2] *= alpha;
              oacc[nb][i][3] *= alpha;
            }
            l_run[nb] *= alpha;
            m_run[nb] = mx;
          }
          const float e0 = ex2(s0v - m_run[nb]);  // ex2(-inf) = 0 for rows that are not shown
          const float e1 = ex2(s1v - m_run[nb]);
          l_run[nb] += e0 + e1;
          // weights as fp16 hi + lo: row token, columns (head t, hi) and (head t, lo)
          bp[nb][0] = movmatrix_trans(hilo_half2(e0 * nv0));  // tokens 2t, 2t+1 of column gq
          bp[nb][1] = movmatrix_trans(hilo_half2(e1 * nv1));  // tokens 2t+8, 2t+9
        }

        // ---- O'^T += Vhat^T P~
        if constexpr (!EARLY_V) load_vpairs();
#define TQ_VSTEP(DB)                                                                          \
        {                                                                                     \
          const uint32_t A[4] = {v_pair<KB, VB, 2 * (DB)>(lut, p01), v_pair<KB, VB, 2 * (DB) + 1>(lut, p01), \
                                 v_pair<KB, VB, 2 * (DB)>(lut, p89), v_pair<KB, VB, 2 * (DB) + 1>(lut, p89)}; \
          _Pragma("unroll") for (int nb = 0; nb < NB; ++nb)                                   \
              mma16816(oacc[nb][DB], A, bp[nb][0], bp[nb][1]);                                 \
        }
        TQ_VSTEP(0) TQ_VSTEP(1) TQ_VSTEP(2) TQ_VSTEP(3) TQ_VSTEP(4) TQ_VSTEP(5) TQ_VSTEP(6) TQ_VSTEP(7)
#undef TQ_VSTEP
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_(&ctl.empty[slot]);
      if (++slot == ns) {
        slot = 0;
        phase ^= 1u;
      }
    }

    // ---- the segment's partial: the warps' (max, sum, o') joined through shared memory
    float* mw = reinterpret_cast<float*>(smem + ctl.merge_off);  // [NW][4]
    float* lw = mw + NW * 4;
    float* ow = lw + NW * 4;  // [NW][4][D]
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float lq = l_run[nb];
      lq += __shfl_xor_sync(FULL, lq, 4);
      lq += __shfl_xor_sync(FULL, lq, 8);
      lq += __shfl_xor_sync(FULL, lq, 16);
      pconsumers_sync<NW>();  // the area's last use has been read
      if (gq == 0) {
        mw[warp * 4 + t] = m_run[nb];
        lw[warp * 4 + t] = lq;
      }
      float* o = ow + (warp * 4 + t) * D;
#pragma unroll
      for (int db = 0; db < 8; ++db) {
        o[16 * db + gq] = oacc[nb][db][0] + oacc[nb][db][1];
        o[16 * db + 8 + gq] = oacc[nb][db][2] + oacc[nb][db][3];
      }
      pconsumers_sync<NW>();
      for (int idx = tid; idx < 4 * D; idx += NW * 32) {
        const int r = idx / D, dd = idx % D;
        float M = -1e30f;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, mw[w * 4 + r]);
        float Ls = 0.0f, O = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float fw = ex2(mw[w * 4 + r] - M);
          Ls = fmaf(fw, lw[w * 4 + r], Ls);
          O = fmaf(fw, ow[(w * 4 + r) * D + dd], O);
        }
        float* dst = a.part + (pslot * HGN + 4 * nb + r) * PART;
        dst[4 + dd] = O;
        if (dd == 0) {
          dst[0] = M;
          dst[1] = Ls;
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (tid == 0) {
    const unsigned int e = *reinterpret_cast<volatile unsigned int*>(&ctl.err);
    if (e) atomicOr(a.err, e);
  }
}

template <int KB, int VB, bool QJL, int NB>
tq_status launch_paged(const PagedArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(paged_split<KB, VB, QJL, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, a.dyn_smem);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "smem attribute: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(PShape<NB>::THREADS);
  cfg.dynamicSmemBytes = a.dyn_smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // dependent of the prep kernel
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_split<KB, VB, QJL, NB>, a);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "paged split launch: %s", cudaGetErrorString(e));
  return TQ_OK;
}

template <int KB, int VB>
tq_status launch_paged_v(const PagedArgs& a, bool qjl, cudaStream_t s) {
  if (a.g <= 4) return qjl ? launch_paged<KB, VB, true, 1>(a, s) : launch_paged<KB, VB, false, 1>(a, s);
  return qjl ? launch_paged<KB, VB, true, 2>(a, s) : launch_paged<KB, VB, false, 2>(a, s);
}

template <int KB>
tq_status launch_paged_k(const PagedArgs& a, int v_bits, bool qjl, cudaStream_t s) {
  if (v_bits == 2) return launch_paged_v<KB, 2>(a, qjl, s);
  if (v_bits == 3) return launch_paged_v<KB, 3>(a, qjl, s);
  return launch_paged_v<KB, 4>(a, qjl, s);
}

}  // namespace
}  // namespace tq
