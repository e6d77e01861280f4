// Split kernel of tq_paged_decode_attn (instantiated per key width in tq_paged_split_k*.cu).
//
// Work.  The tokens a sequence shows (all, or a window's) are cut into groups of 16, which never cross
// a page.  The groups of all units -- a unit is one (sequence, kv-head) and up to eight of its query
// heads -- are laid end to end and cut into one even, contiguous range per warp, so ragged batches
// load every warp alike.  The cut follows from the lengths on the device: every CTA sums them itself, up to
// P_LENS sequences; past that it takes the prep kernel's sums.
// A warp's range is processed as segments, each inside one unit; a segment ends with one
// (max, sum, o') partial per head, which the merge kernel joins.  A CTA whose whole range lies in one
// unit (long contexts) joins its warps first, so that a long unit leaves one partial per CTA.
//
// Warps run on their own: each keeps a ring of DEPTH groups in shared memory and fetches its next
// groups itself with 16-byte cp.async (five per lane and group); the page of the next run (the groups of one
// page) is looked up while the run before it is fetched.
// (One producer warp with bulk copies per page, an mbarrier ring and CTA-wide segments measured 134 us
// at 16 sequences x 16K tokens in 4 bits with pages of 64, against 97 us of the same bytes with pages
// of 128: it was bound by issuing the copies, and short sequences by the barriers at their ends.)
// Nothing before the first product needs a query, so the rings fill while the prep kernel still runs
// (programmatic dependent launch; past P_LENS sequences only behind it, as its sums are needed first).
// 16 tokens become tensor-core operands:
//   scores   D[16 tokens x 8] += A[tokens x dims] B[dims x 8]: A are centroid pairs from a
//            lane-replicated shared-memory table; a second product with the sign bits placed in fp16
//            mantissas gives the QJL term
//   values   O'^T[16 dims x 8] += A[dims x tokens] B[tokens x 8]: A are centroid pairs of two tokens, B
//            the weights p ||v|| / sqrt(128)
// with online softmax in log2 units in between.  q' and the weights enter as fp16 hi + lo (about 22
// bits), sums are fp32.  The sums over tokens are formed on the FP32 units, 16 tokens at a time: the
// tensor cores cut off instead of rounding, always towards zero, which over 128K tokens left an error of
// 6.3e-6 where this leaves 1.8e-6 (four sequences of that length: 171 us, 165 with the tensor cores' sums).
// The 8 columns of B are four heads, hi and lo side by side (one product), or, for five to eight heads,
// eight heads, hi and lo in two products onto the same sums: that keeps the sums at 32 registers.  The
// running maximum moves only when a score passes it by more than LAZY (a vote instead of a three-step
// exchange per group), so exp reaches 2^LAZY.  The weights exp * norm of a head carry a scale that brings
// them into fp16 range.  It is set from the weights themselves (set from the norms alone, a large norm at a
// score far below the maximum would push the weights that count into fp16's subnormals, and past 2^36 times
// the other norms to zero), by the same vote: when the maximum moves, and when a norm could carry a weight
// past the range.
// Rows outside the tokens shown are masked by selection, never by a product, so whatever they hold
// (NaN too) stays out.
#pragma once

#include <algorithm>

#include "tq_decode_core.h"
#include "tq_launch.h"
#include "tq_paged.h"

namespace tq {
namespace {

constexpr float LAZY = 4.0f;
// Weights in fp16: the largest of a group is brought into [2^W_EXP, 2^(W_EXP + 1)) when a head's scale is
// set (hi + lo then leaves 2^-31 of it), and the scale is looked at again when a norm times it passes W_LIMIT:
// times 2^LAZY that stays below fp16's 65504.  With W_EXP = 8 ordinary norms passed the limit so often that
// 64 sequences to 16K in 3/2 bits took 131 us, with 6 they take 125 us.
constexpr int W_EXP = 6;
constexpr float W_LIMIT = 2048.0f;
constexpr float W_START = 0x1p120f;         // scale of a segment without sums: any weight sets it anew
constexpr int P_LENS = 512;                 // sequences whose lengths and running sums are kept in shared memory
constexpr int P_SMEM = 232448;              // dynamic shared memory of a CTA (all an SM gives one)
constexpr int P_MISC = 8192;                // lengths, sums, codebooks

// NB: 1 for up to four heads per unit, 2 for up to eight.
template <int KB, int VB, bool QJL, int NB>
struct PLayout {
  static constexpr int NW = paged_warps(NB), THREADS = 32 * NW, HGN = 4 * NB;
  static constexpr int K_ROW = 16 * KB, V_ROW = 16 * VB;
  // a group in the ring
  static constexpr int OFF_KC = 0;
  static constexpr int OFF_VC = OFF_KC + 16 * K_ROW;
  static constexpr int OFF_SG = OFF_VC + 16 * V_ROW;
  static constexpr int OFF_NK = OFF_SG + (QJL ? 256 : 0);
  static constexpr int OFF_NV = OFF_NK + 64;
  static constexpr int OFF_RN = OFF_NV + 64;
  static constexpr int SLOT = OFF_RN + (QJL ? 64 : 0);
  // Pair tables: 4/4 bits: 256 entries of 256 bytes (key replicas at +0, value replicas at +128) at a
  // 64 KB boundary of the shared window, so that one byte permute makes an address of a byte of codes;
  // other widths: 128-byte entries, each table at a multiple of its size (the larger first), so that an
  // address is a shifted field of codes or'ed into the lane's address of entry 0.  2-bit values: entries of
  // two pairs (two codes of each of two tokens: a byte) of 256 bytes at a 64 KB boundary, one 8-byte load
  // for two operands.
  static constexpr bool kPacked = KB == 4 && VB == 4, kQuadV = VB == 2;
  static constexpr int K_TBL = (1 << (2 * KB)) * 128, V_TBL = kQuadV ? 65536 : (1 << (2 * VB)) * 128;
  static constexpr int TBL_BYTES = K_TBL + V_TBL;
  static constexpr int TBL_ALIGN = kPacked || kQuadV ? 65536 : K_TBL > V_TBL ? K_TBL : V_TBL;
  // places of the tables
  static constexpr uint32_t K_AT = kPacked || K_TBL >= V_TBL ? 0 : V_TBL;
  static constexpr uint32_t V_AT = kPacked ? 128 : K_TBL >= V_TBL ? K_TBL : 0;
  // Rings of the warps, before the tables (the first 1 KB of the window is the system's) and behind them.
  static constexpr int FRONT = TBL_ALIGN > 1024 ? TBL_ALIGN - 1024 : 0;
  static constexpr int BACK = P_SMEM - P_MISC - TBL_BYTES - FRONT - 1024;
  static constexpr int rings(int depth) { return FRONT / (depth * SLOT) + BACK / (depth * SLOT); }
  static constexpr int depth() {
    int d = 6;
    while (d > 2 && rings(d) < NW) --d;
    return d;
  }
  static constexpr int DEPTH = depth();
  static_assert(rings(DEPTH) >= NW, "shared memory");
  static_assert(SLOT % 16 == 0, "16-byte copies");
};

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

template <int OFF>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;\n" ::"r"(dst), "l"(src), "n"(OFF) : "memory");
}
// Loads of a group's rows (after its wait: volatile) ...
template <int OFF>
__device__ __forceinline__ uint32_t ld32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1 + %2];\n" : "=r"(v) : "r"(p), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ float ldf(uint32_t p) { return __uint_as_float(ld32<OFF>(p)); }
template <int OFF>
__device__ __forceinline__ uint2 ld64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];\n" : "=r"(v.x), "=r"(v.y) : "r"(p), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint4 ld128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p), "n"(OFF));
  return v;
}
// ... and of the tables, which do not change; their order and the products' is the compiler's.
__device__ __forceinline__ uint32_t lut32(uint32_t p) {
  uint32_t v;
  asm("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lut64(uint32_t p) {
  uint2 v;
  asm("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
// mma16816 without `volatile`, so that the compiler may interleave the products with the lookups.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Table entry of the W-bit field at bit POS of a code stream: r is the lane's address of entry 0.
// PACKED: W = 8 and 256-byte entries (see PLayout).
template <bool PACKED, int POS, int W, int NWORDS>
__device__ __forceinline__ uint32_t pair_of(const uint32_t (&c)[NWORDS], uint32_t r) {
  constexpr int w = POS / 32, s = POS % 32;
  if constexpr (PACKED) {
    return lut32(__byte_perm(c[w], r, 0x7604u | (uint32_t)((s / 8) << 4)));
  } else {
    constexpr uint32_t mask = ((1u << W) - 1u) << 7;
    uint32_t x;
    if constexpr (s + W > 32) x = __funnelshift_r(c[w], c[w + 1], s - 7);
    else if constexpr (s > 7) x = c[w] >> (s - 7);
    else x = c[w] << (7 - s);
    return lut32((x & mask) | r);
  }
}

// Value codes of one token for lane group gq: 16 codes of VB bits (bits past them are never used).
template <int VB, int OFF>
__device__ __forceinline__ void v_codes_at(uint32_t p, uint32_t odd, uint32_t (&c)[(VB + 1) / 2]) {
  if constexpr (VB == 4) {
    const uint2 v = ld64<OFF>(p);
    c[0] = v.x;
    c[1] = v.y;
  } else if constexpr (VB == 3) {  // six bytes from byte 6 gq: p is that rounded down to a word
    const uint32_t v0 = ld32<OFF>(p), v1 = ld32<OFF + 4>(p);
    c[0] = __funnelshift_r(v0, v1, odd);
    c[1] = v1 >> odd;
  } else {
    c[0] = ld32<OFF>(p);
  }
}
// Codes of two tokens a and b field by field: even fields to e, odd fields to o, a's below b's.
template <int VB, int NWORDS>
__device__ __forceinline__ void interleave(const uint32_t (&a)[NWORDS], const uint32_t (&b)[NWORDS], uint32_t (&e)[NWORDS], uint32_t (&o)[NWORDS]) {
  auto sel = [](uint32_t m, uint32_t x, uint32_t y) { return (x & m) | (y & ~m); };
  if constexpr (VB == 3) {  // 3-bit fields cross the word: 6-bit period, bits 32 .. 47 in the second word
    constexpr uint64_t m = 0x71C71C71C71C71C7ull;
    e[0] = sel((uint32_t)m, a[0], b[0] << 3);
    e[1] = sel((uint32_t)(m >> 32), a[1], __funnelshift_l(b[0], b[1], 3));
    o[0] = sel((uint32_t)m, __funnelshift_r(a[0], a[1], 3), b[0]);
    o[1] = sel((uint32_t)(m >> 32), a[1] >> 3, b[1]);
  } else {
    // (2-bit codes: fields of two codes, as the table of their quads wants them)
#pragma unroll
    for (int i = 0; i < NWORDS; ++i) {
      e[i] = sel(0x0F0F0F0Fu, a[i], b[i] << 4);
      o[i] = sel(0x0F0F0F0Fu, a[i] >> 4, b[i]);
    }
  }
}

// Where a warp stands in the work: group gi of unit uu of sequence b, and what follows of its length.
struct Cursor {
  int b, uu, gi, G, first, len;
};

template <int KB, int VB, bool QJL, int NB>
__global__ void __launch_bounds__(PLayout<KB, VB, QJL, NB>::THREADS, 1) paged_split(const __grid_constant__ PagedArgs a) {
  using Lay = PLayout<KB, VB, QJL, NB>;
  constexpr int NW = Lay::NW, HGN = Lay::HGN, DEPTH = Lay::DEPTH, SLOT = Lay::SLOT;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int U = a.Hkv * a.hgroups;  // units of a sequence
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // ---- shared memory: [front rings] tables [back rings] ... misc at the end
  const uint32_t base = smem_u32(smem);
  const uint32_t tbl = (base + Lay::TBL_ALIGN - 1) & ~(uint32_t)(Lay::TBL_ALIGN - 1);
  const int front = (int)(tbl - base) / (DEPTH * SLOT);  // rings before the tables
  const uint32_t ring = warp < front ? base + warp * (DEPTH * SLOT) : tbl + Lay::TBL_BYTES + (warp - front) * (DEPTH * SLOT);
  unsigned char* misc = smem + P_SMEM - P_MISC;
  int64_t* pre = reinterpret_cast<int64_t*>(misc);               // [P_LENS + 1] groups before a sequence
  int32_t* lens = reinterpret_cast<int32_t*>(misc + 8 * P_LENS + 16);  // [P_LENS]
  float* cbs = reinterpret_cast<float*>(misc + 12 * P_LENS + 32);     // [32]
  int64_t* joint_rec = reinterpret_cast<int64_t*>(misc + 12 * P_LENS + 160);
  static_assert(12 * P_LENS + 168 <= P_MISC, "misc");
  const bool few = a.B <= P_LENS;
  if (few)
    for (int b = tid; b < a.B; b += Lay::THREADS) lens[b] = a.lens[b];
  if (tid < 16) cbs[tid] = tid < (1 << KB) ? a.kc[tid] : 0.0f;
  else if (tid < 32) cbs[tid] = tid - 16 < (1 << VB) ? a.vc[tid - 16] : 0.0f;
  if (base + P_SMEM < tbl + Lay::TBL_BYTES + (uint32_t)(NW > front ? NW - front : 0) * (DEPTH * SLOT) + P_MISC) {
    // dynamic shared memory starts where the rings do not fit (never on sm_100)
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (tid == 0) atomicOr(a.err, 2u);
    return;
  }
  __syncthreads();

  bool bad = false;  // a page number out of range (the prep kernel checks the lengths)
  auto len_of = [&](int b) { return few ? lens[b] : a.lens[b]; };
  if (few && warp == 0) {  // running sums
    int64_t sum = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int first, len, n = b0 + lane < a.B ? lens[b0 + lane] : 0;
      const int G = seq_groups(n, a.max_tokens, a.window, first, len);
      int64_t x = G;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < a.B) pre[b0 + lane] = sum + x - G;
      sum += __shfl_sync(FULL, x, 31);
    }
    if (lane == 0) pre[a.B] = sum;
  }
  // ---- pair tables: entry e = lo | hi << b -> half2(c[lo], c[hi]), a replica per lane, four to a store
  constexpr int PITCH = Lay::kPacked ? 256 : 128;
  unsigned char* tp = smem + (tbl - base);
  for (int i = tid; i < Lay::K_TBL / 16; i += Lay::THREADS) {
    const int e = i >> 3;
    const uint32_t v = pack_half2(cbs[e & ((1 << KB) - 1)], cbs[e >> KB]);
    *reinterpret_cast<uint4*>(tp + Lay::K_AT + e * PITCH + 16 * (i & 7)) = make_uint4(v, v, v, v);
  }
  for (int i = tid; i < Lay::V_TBL / 16; i += Lay::THREADS) {
    if constexpr (Lay::kQuadV) {  // entry: two codes of token a (low four bits), two of token b
      const int e = i >> 4, a4 = e & 15, b4 = e >> 4;
      const uint32_t v = pack_half2(cbs[16 + (a4 & 3)], cbs[16 + (b4 & 3)]), w = pack_half2(cbs[16 + (a4 >> 2)], cbs[16 + (b4 >> 2)]);
      *reinterpret_cast<uint4*>(tp + Lay::V_AT + 16 * i) = make_uint4(v, w, v, w);
    } else {
      const int e = i >> 3;
      const uint32_t v = pack_half2(cbs[16 + (e & ((1 << VB) - 1))], cbs[16 + (e >> VB)]);
      *reinterpret_cast<uint4*>(tp + Lay::V_AT + e * PITCH + 16 * (i & 7)) = make_uint4(v, v, v, v);
    }
  }
  const uint32_t rk = (tbl + Lay::K_AT) | (4u * lane), rv = (tbl + Lay::V_AT) | ((Lay::kQuadV ? 8u : 4u) * lane);
  __syncthreads();
  // a batch too large for shared memory: the prep kernel's sums
  if (!few) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  auto before = [&](int b) { return few ? pre[b] : __ldcg(a.before + b); };
  const int64_t N = before(a.B) * U;
  const Cut cut = cut_of(N, a.ctas, NW);
  const bool mine = (int)blockIdx.x < cut.ctas && warp < cut.warps;
  const int W = blockIdx.x * cut.warps + warp;
  const int64_t f0 = mine ? range_start(N, cut, W) : 0;
  int left = mine ? (int)(range_start(N, cut, W + 1) - f0) : 0;  // groups to go

  auto enter = [&](Cursor& c) { c.G = seq_groups(len_of(c.b), a.max_tokens, a.window, c.first, c.len); };
  auto next_unit = [&](Cursor& c) {
    c.gi = 0;
    if (++c.uu < U) return;
    c.uu = 0;
    do {
      if (++c.b >= a.B) {  // behind the last group: nothing is taken from here
        c.b = a.B - 1;
        c.G = 1;
        return;
      }
      enter(c);
    } while (c.G == 0);
  };
  Cursor cur;
  cur.b = cur.uu = cur.gi = 0;
  cur.G = 1;
  cur.first = cur.len = 0;
  if (left > 0) {
    int lo = 0, hi = a.B;  // before(lo) * U <= f0 < before(hi) * U
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before(mid) * U <= f0) lo = mid;
      else hi = mid;
    }
    cur.b = lo;
    enter(cur);
    const int64_t rem = f0 - before(lo) * U;
    cur.uu = (int)div64(rem, cur.G);
    cur.gi = (int)(rem - (int64_t)cur.uu * cur.G);
  }

  // ---- fetching.  A run is the groups of one page (of one unit): its addresses are formed once, and
  // the page of the run after it is looked up then.
  const int gpp = a.ps / kGroup;  // groups of a page
  auto page_index = [&](int grp) -> int { return gpp == 1 ? grp : (int)__umul64hi((uint64_t)(uint32_t)grp, a.gpp_inv); };
  Cursor nxt = cur;  // the next run's first group
  int to_fetch = left, run = 0;
  auto look_up = [&]() -> int { return __ldg(a.table + (int64_t)nxt.b * a.table_stride + page_index(nxt.first / kGroup + nxt.gi)); };
  int page = to_fetch > 0 ? look_up() : 0;
  // per lane: its 16 bytes of the key and value codes, and of the small arrays: lanes 0 .. 15 the signs,
  // 16 .. 27 the norms (four lanes each)
  const uint8_t *kc = nullptr, *vc = nullptr, *sm = nullptr;
  const uint8_t* sm0 = lane < 16 ? (QJL ? a.k_signs : nullptr) : lane < 20 ? reinterpret_cast<const uint8_t*>(a.k_norm)
                       : lane < 24 ? reinterpret_cast<const uint8_t*>(a.v_norm)
                       : lane < 28 && QJL ? reinterpret_cast<const uint8_t*>(a.k_rnorm) : nullptr;
  const int sm_row = lane < 16 ? 16 : 4;
  const uint32_t sm_at = lane < 16 ? Lay::OFF_SG + 16 * lane : lane < 20 ? Lay::OFF_NK + 16 * (lane - 16)
                         : lane < 24 ? Lay::OFF_NV + 16 * (lane - 20) : Lay::OFF_RN + 16 * (lane - 24);
  if (sm0) sm0 += 16 * (lane < 16 ? lane : (lane & 3));
  uint32_t fdst = ring;
  auto fetch = [&]() {  // (commits a group of copies every time, empty when nothing is left)
    if (to_fetch > 0) {
      if (run == 0) {
        int p = page;
        if ((unsigned)p >= (unsigned)a.pages) {  // a bad table entry: recorded, page 0 read instead
          bad = true;
          p = 0;
        }
        const int grp = nxt.first / kGroup + nxt.gi, in_page = grp - gpp * page_index(grp);
        const int kvh = a.hgroups == 1 ? nxt.uu : nxt.uu / a.hgroups;
        const int64_t row = ((int64_t)p * a.Hkv + kvh) * a.ps + kGroup * in_page;
        kc = a.k_codes + row * Lay::K_ROW + 16 * lane;
        vc = a.v_codes + row * Lay::V_ROW + 16 * lane;
        sm = sm0 + row * sm_row;
        run = min(gpp - in_page, nxt.G - nxt.gi);
        if (run < to_fetch) {
          nxt.gi += run;
          if (nxt.gi == nxt.G) next_unit(nxt);
          page = look_up();
        }
      }
      const uint32_t dst = fdst + 16 * lane;
      cp_async16_at<Lay::OFF_KC>(dst, kc);
      if (KB == 4 || (KB == 3 && lane < 16)) cp_async16_at<Lay::OFF_KC + 512>(dst, kc + 512);
      cp_async16_at<Lay::OFF_VC>(dst, vc);
      if (VB == 4 || (VB == 3 && lane < 16)) cp_async16_at<Lay::OFF_VC + 512>(dst, vc + 512);
      if (sm0) cp_async16_at<0>(fdst + sm_at, sm);
      kc += 16 * Lay::K_ROW;
      vc += 16 * Lay::V_ROW;
      sm += 16 * sm_row;
      --run;
      --to_fetch;
      fdst += SLOT;
      if (fdst == ring + DEPTH * SLOT) fdst = ring;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) fetch();
  asm volatile("griddepcontrol.wait;\n" ::: "memory");

  // Column 2t + x of a lane's sums (x = 0, 1): NB = 1: hi and lo of head t; NB = 2: heads 2t and 2t + 1.
  constexpr int H = NB;  // heads of a lane
  const int gq = lane >> 2, t = lane & 3;
  // rows of a pair of tokens are read in swapped order by lanes with odd t (two bank groups instead of
  // one); the weights of those lanes are swapped alike
  const int sw = VB == 4 ? t & 1 : 0;
  const uint32_t swap_sel = sw ? 0x1032u : 0x3210u;
  // this lane's places in a group
  const uint32_t k_at = Lay::OFF_KC + gq * Lay::K_ROW + 4 * KB * t;
  const uint32_t v_at = Lay::OFF_VC + (2 * t + sw) * Lay::V_ROW + ((2 * VB * gq) & ~3);
  const uint32_t v_odd = VB == 3 ? 16 * (gq & 1) : 0;
  const uint32_t s_at = Lay::OFF_SG + 16 * gq + 4 * t, n_at = Lay::OFF_NK + 4 * gq;
  // a CTA whose range lies in one unit joins its warps at the end (the merge kernel counts likewise);
  // warp 0, which stands at the range's first group, decides
  if (tid == 0) {
    const int64_t begin = f0 - cur.gi;  // the unit's first group in the order of all
    const bool j = left > 0 && range_start(N, cut, (blockIdx.x + 1) * cut.warps) <= begin + cur.G;
    *joint_rec = !j ? -1 : cur.gi == 0 ? (int64_t)cur.b * U + cur.uu : (int64_t)a.B * U + W;
  }
  __syncthreads();
  const int64_t rec_joint = *joint_rec;
  const bool joint = rec_joint >= 0;
  uint32_t src = ring;  // the slot in turn
  // Sums of the values: dim block db: dims 16db + gq (columns 2t, 2t + 1 in [0], [1]) and 16db + 8 + gq
  // ([2], [3]).
  float oacc[8][4];
  float m_run[H], l_run[H], vscale[H];  // weights are exp * norm * vscale
  while (left > 0) {
    const int64_t unit = (int64_t)cur.b * U + cur.uu;
    const bool opens = cur.gi == 0;
    int n = min(left, cur.G - cur.gi);
    left -= n;
    // B fragments of q' and S q': NB = 1: one block, hi and lo in neighbouring columns; NB = 2: block 0
    // hi, block 1 lo
    uint32_t bq[NB][8][2], bsq[NB][8][2];
    float fK[H], fQ[H], Kh[H];
    {
      const uint4* fp = reinterpret_cast<const uint4*>(a.ops + unit * (seg_bytes(NB) / 4)) + lane;
      const float4* hc = reinterpret_cast<const float4*>(a.ops + unit * (seg_bytes(NB) / 4) + NB * 1024);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int w4 = 0; w4 < (QJL ? 8 : 4); ++w4) {
          const uint4 v = __ldcg(fp + (nb * 8 + w4) * 32);
          const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int word = 4 * w4 + j;
            (word < 16 ? bq : bsq)[nb][(word >> 1) & 7][word & 1] = wv[j];
          }
        }
      }
#pragma unroll
      for (int x = 0; x < H; ++x) {
        const float4 h = __ldcg(hc + NB * t + x);
        fK[x] = h.x;
        fQ[x] = h.y;
        Kh[x] = h.z;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.0f;
#pragma unroll
    for (int x = 0; x < H; ++x) {
      m_run[x] = kNoScore;
      l_run[x] = 0.0f;
      vscale[x] = W_START;
    }
    int tk = kGroup * (cur.first / kGroup + cur.gi) + gq - cur.first;  // row gq's place among the tokens shown
    const uint32_t shown = (uint32_t)(cur.len - cur.first);
    for (; n > 0; --n, tk += kGroup) {
      cp_async_wait<DEPTH - 2>();  // the oldest group has landed ...
      __syncwarp();                // ... for every lane, and every lane is done with the slot to fill
      fetch();
      const bool v0ok = (uint32_t)tk < shown, v1ok = (uint32_t)(tk + 8) < shown;

      // ---- scores of tokens gq and gq + 8: products with the key codes and the sign bits in turn
      float ka[NB][4], qa[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) ka[nb][e] = qa[nb][e] = 0.0f;
      uint32_t c0[KB], c1[KB], w0 = 0, w1 = 0;
      const uint32_t kp = src + k_at;
      if constexpr (KB == 4) {
        const uint4 x0 = ld128<0>(kp), x1 = ld128<8 * Lay::K_ROW>(kp);
        c0[0] = x0.x; c0[1] = x0.y; c0[2] = x0.z; c0[3] = x0.w;
        c1[0] = x1.x; c1[1] = x1.y; c1[2] = x1.z; c1[3] = x1.w;
      } else if constexpr (KB == 2) {
        const uint2 x0 = ld64<0>(kp), x1 = ld64<8 * Lay::K_ROW>(kp);
        c0[0] = x0.x; c0[1] = x0.y;
        c1[0] = x1.x; c1[1] = x1.y;
      } else {
        c0[0] = ld32<0>(kp); c0[1] = ld32<4>(kp); c0[2] = ld32<8>(kp);
        c1[0] = ld32<8 * Lay::K_ROW>(kp); c1[1] = ld32<8 * Lay::K_ROW + 4>(kp); c1[2] = ld32<8 * Lay::K_ROW + 8>(kp);
      }
      if constexpr (QJL) {
        w0 = ld32<0>(src + s_at);
        w1 = ld32<128>(src + s_at);
      }
#define TQ_STEP(KK)                                                                                   \
      {                                                                                               \
        const uint32_t A[4] = {pair_of<Lay::kPacked, 4 * KB * (KK), 2 * KB>(c0, rk),                   \
                               pair_of<Lay::kPacked, 4 * KB * (KK), 2 * KB>(c1, rk),                   \
                               pair_of<Lay::kPacked, 4 * KB * (KK) + 2 * KB, 2 * KB>(c0, rk),          \
                               pair_of<Lay::kPacked, 4 * KB * (KK) + 2 * KB, 2 * KB>(c1, rk)};         \
        _Pragma("unroll") for (int nb = 0; nb < NB; ++nb) mma(ka[nb], A, bq[nb][KK]);                  \
        if constexpr (QJL) {                                                                          \
          const uint32_t Z[4] = {sgn<2 * (KK)>(w0), sgn<2 * (KK)>(w1), sgn<2 * (KK) + 1>(w0), sgn<2 * (KK) + 1>(w1)}; \
          _Pragma("unroll") for (int nb = 0; nb < NB; ++nb) mma(qa[nb], Z, bsq[nb][KK]);               \
        }                                                                                             \
      }
      TQ_STEP(0) TQ_STEP(1) TQ_STEP(2) TQ_STEP(3) TQ_STEP(4) TQ_STEP(5) TQ_STEP(6) TQ_STEP(7)
#undef TQ_STEP

      // ---- online softmax (log2 units) of the lane's heads over the warp's 16 tokens
      const uint32_t np = src + n_at;
      const float nk0 = ldf<0>(np), nk1 = ldf<32>(np);
      float rn0 = 0.0f, rn1 = 0.0f;
      if constexpr (QJL) {
        rn0 = ldf<Lay::OFF_RN - Lay::OFF_NK>(np);
        rn1 = ldf<Lay::OFF_RN - Lay::OFF_NK + 32>(np);
      }
      const float nv0 = v0ok ? ldf<64>(np) : 0.0f, nv1 = v1ok ? ldf<96>(np) : 0.0f;
      float sc0[H], sc1[H];  // scores of the two tokens
      const float nv = fmaxf(nv0, nv1);
      bool over = false;
#pragma unroll
      for (int x = 0; x < H; ++x) {
        // a head's sum: its columns hi + lo, or its column of the blocks hi + lo
        auto col = [&](const float (&u)[NB][4], int row) {
          return NB == 1 ? u[0][2 * row] + u[0][2 * row + 1] : u[0][2 * row + x] + u[NB - 1][2 * row + x];
        };
        float s0v = col(ka, 0) * (nk0 * fK[x]);
        float s1v = col(ka, 1) * (nk1 * fK[x]);
        if constexpr (QJL) {
          s0v = fmaf(col(qa, 0) + Kh[x], rn0 * fQ[x], s0v);
          s1v = fmaf(col(qa, 1) + Kh[x], rn1 * fQ[x], s1v);
        }
        sc0[x] = v0ok ? s0v : -INFINITY;
        sc1[x] = v1ok ? s1v : -INFINITY;
        over = over || fmaxf(sc0[x], sc1[x]) > m_run[x] + LAZY || nv * vscale[x] > W_LIMIT;
      }
      if (__any_sync(FULL, over)) {  // the running maximum of some head moves, or its weights' scale
#pragma unroll
        for (int x = 0; x < H; ++x) {
          auto top = [](float v) {  // over the 16 tokens
            v = fmaxf(v, __shfl_xor_sync(FULL, v, 4));
            v = fmaxf(v, __shfl_xor_sync(FULL, v, 8));
            return fmaxf(v, __shfl_xor_sync(FULL, v, 16));
          };
          const float mx = fmaxf(top(fmaxf(sc0[x], sc1[x])), m_run[x]);
          const float alpha = ex2(m_run[x] - mx), grow = ex2(mx - m_run[x]);
          l_run[x] *= alpha;
          m_run[x] = mx;
          // The new scale is the one for this group's weights, or the one at which the sums so far stay as
          // they are (their weights fitted), whichever is smaller.
          const float w = top(fmaxf(ex2(sc0[x] - mx) * nv0, ex2(sc1[x] - mx) * nv1));
          const int ex = max(((__float_as_int(w) >> 23) & 255) - 127, -100);
          const float fresh = __int_as_float((127 + W_EXP - ex) << 23);
          const float scale = fminf(fresh, vscale[x] * grow);  // (grow is infinite where alpha is 0)
          const float r = __fdividef(alpha * scale, vscale[x]);
          vscale[x] = scale;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            oacc[i][x] *= r;
            oacc[i][2 + x] *= r;
            if constexpr (NB == 1) {
              oacc[i][1] *= r;
              oacc[i][3] *= r;
            }
          }
        }
      }
      // weights as fp16 hi and lo, turned from (token row, columns 2t, 2t + 1) into (column gq, tokens 2t,
      // 2t + 1 and + 8): B fragments of the value products
      uint32_t bp[NB][2];
      {
        float p0[H], p1[H];
#pragma unroll
        for (int x = 0; x < H; ++x) {
          const float e0 = ex2(sc0[x] - m_run[x]);  // ex2(-inf) = 0 for rows that are not shown
          const float e1 = ex2(sc1[x] - m_run[x]);
          l_run[x] += e0 + e1;
          p0[x] = e0 * nv0 * vscale[x];  // (in this order: norm times scale can pass fp32 where exp is 0)
          p1[x] = e1 * nv1 * vscale[x];
        }
        if constexpr (NB == 1) {
          bp[0][0] = movmatrix_trans(hilo_half2(p0[0]));
          bp[0][1] = movmatrix_trans(hilo_half2(p1[0]));
        } else {
          auto hi_lo = [](float x, float y, uint32_t& hi, uint32_t& lo) {
            const __half2 h = __floats2half2_rn(x, y);
            const float2 f = __half22float2(h);
            hi = *reinterpret_cast<const uint32_t*>(&h);
            lo = pack_half2(x - f.x, y - f.y);
          };
          uint32_t h0, l0, h1, l1;
          hi_lo(p0[0], p0[H - 1], h0, l0);
          hi_lo(p1[0], p1[H - 1], h1, l1);
          bp[0][0] = movmatrix_trans(h0);
          bp[0][1] = movmatrix_trans(h1);
          bp[NB - 1][0] = movmatrix_trans(l0);
          bp[NB - 1][1] = movmatrix_trans(l1);
        }
        if constexpr (VB == 4) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            bp[nb][0] = __byte_perm(bp[nb][0], 0u, swap_sel);
            bp[nb][1] = __byte_perm(bp[nb][1], 0u, swap_sel);
          }
        }
      }

      // ---- O'^T += Vhat^T P: token pairs (2t, 2t + 1) and (2t + 8, 2t + 9)
      constexpr int VW = (VB + 1) / 2;
      uint32_t e01[VW], o01[VW], e89[VW], o89[VW];
      {
        uint32_t x[VW], y[VW];
        const uint32_t vp = src + v_at, vq = sw ? vp - Lay::V_ROW : vp + Lay::V_ROW;
        v_codes_at<VB, 0>(vp, v_odd, x);
        v_codes_at<VB, 0>(vq, v_odd, y);
        interleave<VB>(x, y, e01, o01);
        v_codes_at<VB, 8 * Lay::V_ROW>(vp, v_odd, x);
        v_codes_at<VB, 8 * Lay::V_ROW>(vq, v_odd, y);
        interleave<VB>(x, y, e89, o89);
      }
      // (2-bit values: a byte of e or o holds blocks 2j or 2j + 1 of both tokens)
#define TQ_STEP(DB)                                                                                   \
      {                                                                                               \
        uint32_t A[4];                                                                                \
        if constexpr (Lay::kQuadV) {                                                                  \
          const uint2 x = lut64(__byte_perm(((DB) & 1 ? o01 : e01)[0], rv, 0x7604u | (((DB) / 2) << 4)));  \
          const uint2 y = lut64(__byte_perm(((DB) & 1 ? o89 : e89)[0], rv, 0x7604u | (((DB) / 2) << 4)));  \
          A[0] = x.x; A[1] = x.y; A[2] = y.x; A[3] = y.y;                                             \
        } else {                                                                                      \
          A[0] = pair_of<Lay::kPacked, 2 * VB * (DB), 2 * VB>(e01, rv);                                \
          A[1] = pair_of<Lay::kPacked, 2 * VB * (DB), 2 * VB>(o01, rv);                                \
          A[2] = pair_of<Lay::kPacked, 2 * VB * (DB), 2 * VB>(e89, rv);                                \
          A[3] = pair_of<Lay::kPacked, 2 * VB * (DB), 2 * VB>(o89, rv);                                \
        }                                                                                             \
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};                                                        \
        _Pragma("unroll") for (int nb = 0; nb < NB; ++nb) mma(z, A, bp[nb]);                           \
        _Pragma("unroll") for (int i = 0; i < 4; ++i) oacc[DB][i] += z[i];                             \
      }
      TQ_STEP(0) TQ_STEP(1) TQ_STEP(2) TQ_STEP(3) TQ_STEP(4) TQ_STEP(5) TQ_STEP(6) TQ_STEP(7)
#undef TQ_STEP
      src += SLOT;
      if (src == ring + DEPTH * SLOT) src = ring;
    }
    // on to the next unit (the segment ended there, or the range did)
    const int64_t rec = opens ? unit : (int64_t)a.B * U + W;
    if (left > 0) next_unit(cur);

    // ---- the segment's partial
#pragma unroll
    for (int x = 0; x < H; ++x) {
      l_run[x] += __shfl_xor_sync(FULL, l_run[x], 4);
      l_run[x] += __shfl_xor_sync(FULL, l_run[x], 8);
      l_run[x] += __shfl_xor_sync(FULL, l_run[x], 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float vback = 0.08838834764831845f / vscale[NB == 1 ? 0 : j & (H - 1)];  // with the values' 1 / sqrt(128)
#pragma unroll
      for (int i = 0; i < 8; ++i) oacc[i][j] *= vback;
    }
    if (joint) break;  // (the range's only segment)
#pragma unroll
    for (int x = 0; x < H; ++x) {
      float* dst = a.part + (rec * HGN + NB * t + x) * PART;
      if (gq == 0) *reinterpret_cast<float2*>(dst) = make_float2(m_run[x], l_run[x]);
#pragma unroll
      for (int db = 0; db < 8; ++db) {
        const float o0 = NB == 1 ? oacc[db][0] + oacc[db][1] : oacc[db][x];
        const float o1 = NB == 1 ? oacc[db][2] + oacc[db][3] : oacc[db][2 + x];
        dst[4 + 16 * db + gq] = o0;
        dst[4 + 16 * db + 8 + gq] = o1;
      }
    }
  }
  cp_async_wait<0>();
  if (joint) {  // CTA-uniform
    __syncthreads();  // the rings are free
    // a warp's (max, sum) and o' of each head, in its own ring
    static_assert(DEPTH * SLOT >= HGN * (2 + D) * 4, "join area");
    if (mine) {
      float* my = reinterpret_cast<float*>(smem + (ring - base));
#pragma unroll
      for (int x = 0; x < H; ++x) {
        const int i = NB * t + x;
        if (gq == 0) {
          my[2 * i] = m_run[x];
          my[2 * i + 1] = l_run[x];
        }
        float* o = my + 2 * HGN + i * D;
#pragma unroll
        for (int db = 0; db < 8; ++db) {
          o[16 * db + gq] = NB == 1 ? oacc[db][0] + oacc[db][1] : oacc[db][x];
          o[16 * db + 8 + gq] = NB == 1 ? oacc[db][2] + oacc[db][3] : oacc[db][2 + x];
        }
      }
    }
    __syncthreads();
    for (int idx = tid; idx < HGN * D; idx += Lay::THREADS) {
      const int i = idx / D, dd = idx % D;
      auto of = [&](int w) {
        const uint32_t r = w < front ? base + w * (DEPTH * SLOT) : tbl + Lay::TBL_BYTES + (w - front) * (DEPTH * SLOT);
        return reinterpret_cast<const float*>(smem + (r - base));
      };
      float M = kNoScore, Ls = 0.0f, O = 0.0f;
      for (int w = 0; w < cut.warps; ++w) M = fmaxf(M, of(w)[2 * i]);
      for (int w = 0; w < cut.warps; ++w) {
        const float* v = of(w);
        const float fw = ex2(v[2 * i] - M);
        Ls = fmaf(fw, v[2 * i + 1], Ls);
        O = fmaf(fw, v[2 * HGN + i * D + dd], O);
      }
      float* dst = a.part + (rec_joint * HGN + i) * PART;
      dst[4 + dd] = O;
      if (dd == 0) *reinterpret_cast<float2*>(dst) = make_float2(M, Ls);
    }
  }
  if (bad) atomicOr(a.err, 16u);
}

template <int KB, int VB, bool QJL, int NB>
tq_status launch_paged(const PagedArgs& a, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(paged_split<KB, VB, QJL, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM);
  if (e != cudaSuccess) return fail(TQ_ERR_CUDA, "smem attribute: %s", cudaGetErrorString(e));
  // (a dependent of the prep kernel)
  return launch(paged_split<KB, VB, QJL, NB>, a.ctas, PLayout<KB, VB, QJL, NB>::THREADS, P_SMEM, stream, true, "paged split", a);
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
