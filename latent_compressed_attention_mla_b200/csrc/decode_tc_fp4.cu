// S3 on the 5th-generation tensor cores over the 4-bit cache (e2m1 codes, e4m3 scales of
// 16 columns, a token scale, bf16 k^R): decode_tc.cu's scheme (CTA pairs, cta_group::2
// MMAs, an operand ring each for QK and PV fed by converter warps, online softmax
// from TMEM), with these differences:
//  * The converters turn e2m1 pairs into f16 by one conversion and one multiply with
//    the block's scale times the token's: exact for token scales from 2^-14 (at most
//    six significant bits).  Below, f16's subnormals are off by up to 2^-25 in that
//    scale, times a code of up to 6, and in the product: 7 x 2^-25 in all.  A staging
//    slot holds 128 columns, enough for two units.  k^R and q^R stay bf16: TMA brings
//    the k^R unit straight into the ring, and its MMAs take the bf16 form.
//  * Any head count: the rows (query token, head) of a sequence, r = t * n_heads +
//    h, form groups of 128, each row with its own causal limit (rows behind the
//    last are computed and not stored).
//  * P is handed over in two halves, and the warpgroups share out the registers, so
//    that the softmax holds a tile's probabilities while the previous PV runs.
//  * Roles: warps 0-3 softmax and epilogue, 4 TMEM allocation and (leader) QK issue,
//    5 (leader) PV issue, 6 / 7 TMA for Q and QK / PV data, 8-11 / 12-15 converters
//    of QK / PV units.
// Measured (this kernel's span on the device): 128 heads, 128 sequences of 16,386 keys
// with two query tokens 1,209 us (963 TFLOP/s; CUDA cores 410 ms), 64 ragged sequences
// of up to 32,769 keys 349 us (64 heads: 312 us).  A tile of 256 keys takes 5.5 us, of
// which the QK converters are busy 5.1, but no unit is at its limit (shared memory
// 63%, tensor pipe and ALU 38%): each scheduler has one warp of a ring's four, whose
// waits, loads, conversions and stores follow one another, and that chain's latency is
// the time.  The bf16 cache, which needs no conversion, takes 1,071 us on the large
// batch: with all heads on one GPU the 4-bit cache saves memory, not time.  On the
// way: k^R converted like the codes 1.475 ms, P handed over whole 1.412, a loop
// unrolled over the units 1.69 (instruction cache; the producers' loops alone,
// unrolled, 1.255: hence their unroll 1).
//
// A kernel of its own and not a variant of decode_tc.cu's: in one template, with this
// one's order of roles, the FP8 variant took 1,739 us for 1,630 on the same sequences.
#include "decode_tc.cuh"

namespace mla {

namespace {

// scales of one page: [64 rows][32] e4m3, then [64 rows] fp32 token scales
constexpr uint32_t kPageScl = 64 * 32 + 64 * 4;

// Shared memory layout and warp roles (offsets from a 1024-byte aligned base).
struct L {
  static constexpr int QKSlots = 2, PVSlots = 2, QStSlots = 3, PStSlots = 2;
  // The QK scale blocks hold this CTA's two pages of a tile, and a PV staging slot
  // brings its page's scales along: one block for both rings would tie the QK
  // units of tile g + 2 to the PV units of tile g (measured: 7.8 us a tile, 1.9 ms
  // on 128 sequences of 16,384 with two tokens).
  static constexpr int SclBufs = 2, SclPages = 2;
  static constexpr uint32_t PageScl = kPageScl, SclBytes = SclPages * PageScl;
  // (slots are 512-byte aligned: their codes carry the 64-byte swizzle)
  static constexpr uint32_t PStBytes = kStageBytes + (PageScl + 511) / 512 * 512;
  static constexpr uint32_t OffQ = 0;
  static constexpr uint32_t OffP = OffQ + kQBytes;
  static constexpr uint32_t OffQKRing = OffP + kPBytes;
  static constexpr uint32_t OffPVRing = OffQKRing + QKSlots * kUnitBytes;
  static constexpr uint32_t OffQSt = OffPVRing + PVSlots * kUnitBytes;
  static constexpr uint32_t OffPSt = OffQSt + QStSlots * kStageBytes;
  static constexpr uint32_t OffScl = OffPSt + PStSlots * PStBytes;
  static constexpr uint32_t OffBar = OffScl + SclBufs * SclBytes;
  // barrier indices
  static constexpr int QK_FULL = 0;                     // [QKSlots] leader: unit written in both CTAs
  static constexpr int QK_EMPTY = QK_FULL + QKSlots;    // [QKSlots] each CTA: unit consumed (MMA commit)
  static constexpr int PV_FULL = QK_EMPTY + QKSlots;    // [PVSlots]
  static constexpr int PV_EMPTY = PV_FULL + PVSlots;    // [PVSlots]
  static constexpr int S_FULL = PV_EMPTY + PVSlots;     // [2] each CTA: S tile ready (MMA commit)
  static constexpr int S_FREE = S_FULL + 2;             // [2] leader: S read by both CTAs' softmax warps
  static constexpr int P_FULL = S_FREE + 2;             // leader: P written + O rescaled by both CTAs
  static constexpr int O_DONE = P_FULL + 1;             // each CTA: the tile's PV MMAs finished
  static constexpr int O_FREE = O_DONE + 1;             // leader: O read out by both CTAs' epilogues
  static constexpr int Q_FULL = O_FREE + 1;             // [kChunks] leader: Q chunk bytes of both CTAs
  static constexpr int Q_EMPTY = Q_FULL + kChunks;      // each CTA: last QK of a segment finished
  static constexpr int QST_FULL = Q_EMPTY + 1;          // [QStSlots] local: staged bytes landed
  static constexpr int QST_EMPTY = QST_FULL + QStSlots; // [QStSlots] local: both converter warps done
  static constexpr int PST_FULL = QST_EMPTY + QStSlots; // [PStSlots]
  static constexpr int PST_EMPTY = PST_FULL + PStSlots; // [PStSlots]
  static constexpr int SCL_FULL = PST_EMPTY + PStSlots;  // [SclBufs] local: a tile's scales landed
  static constexpr int SCL_EMPTY = SCL_FULL + SclBufs;   // [SclBufs] local: all converter warps done
  static constexpr int DRAIN = SCL_EMPTY + SclBufs;      // each CTA: both MMA issuers' operations completed
  static constexpr int P_FULL2 = DRAIN + 1;              // leader: P of key positions 2 and 3 written
  static constexpr int P_FREE = P_FULL2 + 1;             // each CTA: the MMAs reading P positions 0 and 1 finished
  static constexpr int NumBars = P_FREE + 1;
  static constexpr uint32_t OffMisc = OffBar + NumBars * 8;
  static constexpr uint32_t OffRedMax = OffMisc + 16;   // float [2][64]
  static constexpr uint32_t OffRedL = OffRedMax + 512;  // float [2][64]
  static constexpr uint32_t SmemBytes = OffRedL + 512 + 1024;  // + alignment slack
  static constexpr int QKWarp = 4, PVWarp = 5;          // TMEM alloc (QKWarp); leader lane 0 issues the MMAs
  static constexpr int QKProdWarp = 6, PVProdWarp = 7, ConvWarps = 4;
  static constexpr int QKConvWarp = 8, PVConvWarp = QKConvWarp + ConvWarps;
  static constexpr int Threads = 32 * (PVConvWarp + ConvWarps);
  // arrivals completing one phase of a unit's FULL barrier: every converter warp of both CTAs
  static constexpr int UnitFullCount = 2 * ConvWarps;
};
static_assert(L::SmemBytes <= 232448, "shared memory");

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}

// Two blocks' e4m3 scales (low byte first) times the token's scale, as an f16 pair;
// nan: what a NaN becomes (block scales are not negative).  The product is formed in
// fp32: a token's scale alone may lie outside f16's range, with a block scale of up to
// 448 that brings it back, or with 0s where k^R alone makes it large.
__device__ __forceinline__ uint32_t block_scales(uint32_t sc, uint32_t nan, float ts) {
  const float2 s = f16x2_to_float2(max_f16x2(e4m3x2_to_f16x2(sc), nan));
  const __half2 h = __floats2half2_rn(s.x * ts, s.y * ts);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 e2m1 codes (two blocks of 16 columns) times their scales s -> 64 bytes of
// f16: the 16-byte units u0 ^ e, e = 0..3, of a 128-byte swizzled row.
__device__ __forceinline__ void store_e2m1x32(uint8_t* row, uint32_t u0, const uint4& w, uint32_t s) {
  const uint32_t words[4] = {w.x, w.y, w.z, w.w}, s0 = dup_lo(s), s1 = dup_hi(s);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r[4];
    e2m1x8_to_f16x2(words[i], r);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = mul_f16x2(r[e], i < 2 ? s0 : s1);
    *reinterpret_cast<uint4*>(row + ((u0 ^ i) << 4)) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) into
// this CTA's shared memory, completing on a local barrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

struct TcParams {
  DecodeParams p;
  int groups;            // groups of 128 query rows
  CUtensorMap map_q;     // q_abs rows, box 64 x 64 (f16, the q^R columns bf16)
  CUtensorMap map_o;     // o_part [rows][512] f16, box 64 x 64, 128-byte swizzle
  CUtensorMap map_codes; // [pages][64 rows][256 bytes], box 64 bytes x 64 rows, 64-byte swizzle
  CUtensorMap map_kr;    // bf16 k^R, box 64 x 64 rows, 128-byte swizzle
  size_t scl_off;        // the scales' offset in a page (block scales, then token scales)
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(L::Threads, 1)
    decode_tc_fp4_kernel(const __grid_constant__ TcParams P) {
  constexpr uint32_t kIdescQK = idesc(128, 256, false, false, true);
  constexpr uint32_t kIdescQKb = idesc(128, 256, false, false, false);  // k^R unit: bf16 operands
  constexpr uint32_t kIdescPV = idesc(128, 256, false, true, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const DecodeParams& p = P.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0 = leader (issues the MMAs)
  const int pair = blockIdx.x >> 1;
  const int grp = pair % P.groups, w = pair / P.groups;
  const int n_heads = p.d.n_heads, n_rows = p.n_q * n_heads;  // of a sequence
  const int row0 = kHeads * grp + kHalfHeads * (int)rank;                     // this CTA's first
  const int t = min(n_rows - 1, kHeads * grp + kHeads - 1) / n_heads;  // (last) query token of the group

  auto bar = [&](int i) -> uint32_t { return sbase + L::OffBar + 8u * i; };
  auto leader_bar = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OffMisc + 4);
  float* red_max = reinterpret_cast<float*>(smem + L::OffRedMax);
  float* red_l = reinterpret_cast<float*>(smem + L::OffRedL);

  pdl_trigger();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::QKSlots; ++i) {
      mbar_init(bar(L::QK_FULL + i), L::UnitFullCount);
      mbar_init(bar(L::QK_EMPTY + i), 1);
    }
    for (int i = 0; i < L::PVSlots; ++i) {
      mbar_init(bar(L::PV_FULL + i), L::UnitFullCount);
      mbar_init(bar(L::PV_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::S_FULL + i), 1);
      mbar_init(bar(L::S_FREE + i), 8);
    }
    mbar_init(bar(L::P_FULL), 8);
    mbar_init(bar(L::O_DONE), 1);
    mbar_init(bar(L::O_FREE), 8);
    for (int c = 0; c < kChunks; ++c) mbar_init(bar(L::Q_FULL + c), 1);
    mbar_init(bar(L::Q_EMPTY), 1);
    for (int i = 0; i < L::QStSlots; ++i) {
      mbar_init(bar(L::QST_FULL + i), 1);
      mbar_init(bar(L::QST_EMPTY + i), L::ConvWarps);
    }
    for (int i = 0; i < L::PStSlots; ++i) {
      mbar_init(bar(L::PST_FULL + i), 1);
      mbar_init(bar(L::PST_EMPTY + i), L::ConvWarps);
    }
    for (int i = 0; i < L::SclBufs; ++i) {
      mbar_init(bar(L::SCL_FULL + i), 1);
      mbar_init(bar(L::SCL_EMPTY + i), L::ConvWarps);
    }
    mbar_init(bar(L::P_FULL2), 4);
    mbar_init(bar(L::P_FREE), 1);
    mbar_init(bar(L::DRAIN), 2);  // the QK and the PV issuer's final commit
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == L::QKWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // everything below reads the absorbed queries, the plan and the cache, or
  // writes the split partials
  // Before the grid-dependency wait, warm L2 with the pages of this CTA's
  // first tile (small batches, where that tile's latency is the step's).
  if (warp == L::PVProdWarp && p.batch <= 32) prefetch_first_tile(p, w, (int)rank, lane);
  pdl_wait();
  tl_begin(p.timeline, MLA_TRACE_ATTEND);

  auto page_of = [&](int b, int pg) -> int {
    int page = p.page_table[(size_t)b * p.max_pages + pg];
    if (page < 0 || page >= p.num_pages) {
      record_status(p.status, MLA_ERR_BOUNDS);
      page = 0;
    }
    return page;
  };

  // Self-test of failure detection: no producer issues a load, so the MMA
  // issuers' and softmax warps' bounded waits expire with no copy in flight.
  const bool stall = (p.d.flags & MLA_FLAG_SELFTEST_STALL) != 0;
  // Roles by warpgroup, called at the end.  The 512 threads are launched with 128
  // registers each and share them out anew, so that the softmax holds a tile's
  // probabilities: 128 x 192 (softmax) + 128 x 64 (issuers, producers) + 256 x 120
  // (converters) = 63,488 of 65,536.
  auto softmax = [&]() {
    // ------------------------------------------------------- softmax, epilogue
    // Thread L (TMEM lane) holds head hl of this CTA; lanes 0-63 see the
    // keys of the leader's pages (0 and 2 of a tile), lanes 64-127 those of the
    // peer's (1 and 3): the QK B operand holds the leader's two pages in N
    // columns [0,128), the peer's in [128,256); 2x2 layout.  S is read twice from TMEM: once for the max,
    // once for the probabilities, so that few registers hold scores at a time.
    // The per-page loops stay rolled: the smaller code runs measurably faster
    // (the first tile of a step executes it from a cold instruction cache).
    const int Lt = warp * 32 + lane;
    const int hl = Lt & 63, half = Lt >> 6;
    const int row = row0 + hl;                          // this thread's query row,
    const int row_t = min(row, n_rows - 1) / n_heads;  // its token
    const bool row_ok = row < n_rows;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    SegmentWalker walk(p, w, t);
    Segment s;
    uint32_t g = 0;
    bool ok = true;
    while (walk.next(s)) {
      // the row's place among the split partials, 16-bit rows on this path (the combine reads them so)
      auto part = [&]() -> size_t {
        return ((size_t)row_t * p.n_slots + (w + s.b)) * n_heads + (row - row_t * n_heads);
      };
      if (s.n_pages == 0 || !ok) {
        __half* od = reinterpret_cast<__half*>(p.o_part) + part() * kDC;
        if (row_ok) {
          for (int j = 0; j < 2; ++j)
            for (int c = 0; c < 128; c += 8)
              *reinterpret_cast<uint4*>(od + 256 * j + 128 * half + c) = make_uint4(0, 0, 0, 0);
          if (half == 0) p.lse_part[part()] = -INFINITY;
        }
        continue;
      }
      const int row_vis = p.seq_lens[s.b] - p.n_q + row_t + 1;  // keys the row sees
      float m_ref = -INFINITY, l_part = 0.f;
      const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
      for (int it = 0; it < n_tiles; ++it, ++g) {
        ok = softmax_all_ok(mbar_wait(bar(L::S_FULL + (g & 1)), (g >> 1) & 1, abort_flag, p.status) && ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_addr = tmem + lane_base + ((g & 1) ? kColS1 : kColS0);
        // visible keys of this thread's two key positions 2*half + q (pages tile_page(2*half + q))
        const int pg0 = s.page_lo + it * kTilePages;
        int nv[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int pg = pg0 + tile_page(2 * half + q);
          nv[q] = pg < s.page_lo + s.n_pages ? max(0, min(kPage, row_vis - pg * kPage)) : 0;
        }
        // pass 1: the tile's max (scale > 0 commutes with max)
        float mx = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t sr[64];
          tmem_ld32(s_addr + 64 * q, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(s_addr + 64 * q + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_wait_ld();
          mask_scores(sr, q ? nv[1] : nv[0]);
          mx = fmaxf(mx, max64(sr));
        }
        mx = mx * p.scale_log2;
        red_max[half * 64 + hl] = mx;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const float tile_max = fmaxf(mx, red_max[(half ^ 1) * 64 + hl]);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        bool rescale = false;
        float alpha = 1.f;
        if (it == 0) {
          m_ref = tile_max;
        } else if (tile_max > m_ref + kRescaleThreshold) {
          rescale = true;
          alpha = fast_exp2(m_ref - tile_max);
          m_ref = tile_max;
        }
        // a row whose causal limit lies before the group's may not see a key yet
        const float m_sub = m_ref == -INFINITY ? 0.f : m_ref;
        // pass 2: probabilities of page sub-tile 2*half + q, packed in pairs
        float psum = 0.f;
        auto probs = [&](int q, uint32_t(&pk)[32]) {
          uint32_t sr[64];
          tmem_ld32(s_addr + 64 * q, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(s_addr + 64 * q + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_wait_ld();
          mask_scores(sr, q ? nv[1] : nv[0]);
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float e0 = fast_exp2(__uint_as_float(sr[2 * j]) * p.scale_log2 - m_sub);
            const float e1 = fast_exp2(__uint_as_float(sr[2 * j + 1]) * p.scale_log2 - m_sub);
            const __half2 h2 = __floats2half2_rn(e0, e1);
            s4[j & 1] += e0;
            s4[2 + (j & 1)] += e1;
            pk[j] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          psum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        };
        // P row hl of sub-tile 2*half + q (64 keys, 128 B per row, 128-byte swizzle)
        auto store_p = [&](int q, const uint32_t(&pk)[32]) {
          uint8_t* prow = smem + L::OffP + (2 * half + q) * 8192 + hl * 128;
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<uint4*>(prow + ((u ^ (hl & 7)) * 16)) =
                make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        };
        // S of this tile is consumed: the QK MMAs two tiles on may overwrite it
        auto release_s = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(leader_bar(L::S_FREE + (g & 1)));
        };
        // the previous tile's PV MMAs read P and write O: wait for them, then
        // rescale O if the reference max moved (tcgen05.ld/st are whole-warp
        // instructions: the warp's lanes rescale together, alpha = 1 on lanes
        // whose head keeps its reference)
        auto wait_pv_rescale = [&]() -> bool {
          if (g >= 1) {
            // warp-uniform outcome: the TMEM accesses below are whole-warp
            if (!__all_sync(0xffffffffu, mbar_wait(bar(L::O_DONE), (g - 1) & 1, abort_flag, p.status)))
              return false;
            tc_fence_after();
          }
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
              const uint32_t col = (c < 128 ? kColO0 + c : kColO1 + (c - 128));
              uint32_t orr[32];
              tmem_ld32(tmem + lane_base + col, orr);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) orr[j] = __float_as_uint(__uint_as_float(orr[j]) * alpha);
              tmem_st32(tmem + lane_base + col, orr);
            }
            tmem_wait_st();
          }
          return true;
        };
        // the probabilities are formed while the previous PV runs; only
        // their stores into P wait for it
        uint32_t pk_lo[32], pk_hi[32];
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[32];
          probs(q, pk);
          if (q == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) pk_lo[j] = pk[j];
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) pk_hi[j] = pk[j];
          }
        }
        release_s();
        // P is handed over in two halves, so that the tile's PV MMAs start as
        // soon as the previous tile's end: warps 0-1 (key positions 0 and
        // 1) overwrite theirs once the MMAs of those positions are done, halfway
        // through the previous tile's; warps 2-3 once all are.  The first
        // half's barrier also says that every warp has rescaled its part of
        // O, which waits for all of the previous tile's MMAs where it happens.
        // A failed wait is agreed on at the next tile's (or the epilogue's).
        const bool resc = __any_sync(0xffffffffu, rescale);
        if (resc) ok = wait_pv_rescale();
        tc_fence_before();
        __syncwarp();  // lane 0 arrives for all: every lane's part of O is rescaled
        if (half == 1 && lane == 0) mbar_arrive_cluster(leader_bar(L::P_FULL));
        if (g >= 1 && ok && !resc)
          ok = __all_sync(0xffffffffu, mbar_wait(bar(half ? L::O_DONE : L::P_FREE), (g - 1) & 1, abort_flag, p.status));
        if (ok) {
          store_p(0, pk_lo);
          store_p(1, pk_hi);
        }
        l_part = l_part * alpha + psum;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(leader_bar(half ? L::P_FULL2 : L::P_FULL));
      }
      if (!ok) break;
      // epilogue: wait for the last PV, normalise, write the split's partial
      ok = softmax_all_ok(mbar_wait(bar(L::O_DONE), (g - 1) & 1, abort_flag, p.status) && ok);
      if (!ok) break;
      tc_fence_after();
      red_l[half * 64 + hl] = l_part;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const float l_tot = l_part + red_l[(half ^ 1) * 64 + hl];
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const float inv = l_tot > 0.f ? 1.f / l_tot : 0.f;
      // O leaves, normalised and rounded to f16 (whose range the latent keeps here
      // anyway: the partials' rounding is 2^-12, not bf16's 2^-9), through the (free) P buffer
      // as 64-column x 64-head boxes stored by TMA: lanes 0-63 hold dims
      // [256j, 256j+128), lanes 64-127 dims [256j+128, 256j+256).  Four 8 KB
      // staging slots: two iterations of both halves in flight.
      {
        const bool issuer = hl == 0;  // thread 0 of each half
        // (the CTA's rows are one token's where n_heads is a multiple of 64; other
        // head counts store row by row)
        const bool boxes = n_heads % kHalfHeads == 0;
        const int orow = (int)(((size_t)(row0 / n_heads) * p.n_slots + w + s.b) * n_heads + row0 % n_heads);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int c = 64 * i;
          if (i >= 2) {
            if (issuer) bulk_wait_read<1>();
            asm volatile("bar.sync %0, 64;" ::"r"(2 + half) : "memory");
          }
          const uint32_t col = (c < 128 ? kColO0 + c : kColO1 + (c - 128));
          uint32_t orr[64];
          tmem_ld32(tmem + lane_base + col, *reinterpret_cast<uint32_t(*)[32]>(&orr[0]));
          tmem_ld32(tmem + lane_base + col + 32, *reinterpret_cast<uint32_t(*)[32]>(&orr[32]));
          tmem_wait_ld();
          uint8_t* box = smem + L::OffP + ((i & 1) * 2 + half) * 8192 + hl * 128;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v0 = __uint_as_float(orr[8 * q + 2 * e]) * inv, v1 = __uint_as_float(orr[8 * q + 2 * e + 1]) * inv;
              const __half2 v2 = __floats2half2_rn(v0, v1);
              u[e] = *reinterpret_cast<const uint32_t*>(&v2);
            }
            if (boxes)
              *reinterpret_cast<uint4*>(box + ((q ^ (hl & 7)) * 16)) = make_uint4(u[0], u[1], u[2], u[3]);
            else if (row_ok)
              *reinterpret_cast<uint4*>(reinterpret_cast<__half*>(p.o_part) + part() * kDC + (c < 128 ? 0 : 256) +
                                        128 * half + (c & 127) + 8 * q) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          fence_proxy_async();
          asm volatile("bar.sync %0, 64;" ::"r"(2 + half) : "memory");
          if (issuer && boxes && row_ok) {
            tma_store_2d(&P.map_o, (c < 128 ? 0 : 256) + 128 * half + (c & 127), orow,
                         sbase + L::OffP + ((i & 1) * 2 + half) * 8192);
            bulk_commit();
          }
        }
        // the stores have read the staging slots (the next segment writes P
        // there) and written the partials
        if (issuer) bulk_wait_all();
        asm volatile("bar.sync %0, 64;" ::"r"(2 + half) : "memory");
      }
      if (half == 0 && row_ok) p.lse_part[part()] = l_tot == 0.f ? -INFINITY : m_ref + __log2f(l_tot);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_bar(L::O_FREE));
    }
  };
  auto convert = [&]() {
    // ------------------------------------ 4-bit: conversion of both rings' units
    // One rolled loop serves the QK and the PV converters (measured: with the
    // loops apart and unrolled, a third of all warp stalls were instruction
    // fetches).  A staging slot feeds two units; thread ct takes 32 columns q
    // (two blocks) of one row in each of a unit's two 8 KB halves: the two
    // pages of a QK unit, the two 64-column atoms of a PV unit.  Eight lanes
    // take eight rows, so that the 64-byte swizzle of the staged codes and the
    // 128-byte swizzle of the operands both spread them over all banks.
    const bool pv = warp >= L::PVConvWarp;
    const int ct = (warp - (pv ? L::PVConvWarp : L::QKConvWarp)) * 32 + lane;
    const int row = (ct >> 4) * 8 + (ct & 7), q = (ct >> 3) & 1;
    const uint32_t u0 = (uint32_t)(4 * q) ^ (row & 7);
    const uint32_t st_full = bar(pv ? L::PST_FULL : L::QST_FULL), st_empty = bar(pv ? L::PST_EMPTY : L::QST_EMPTY);
    const uint32_t un_empty = bar(pv ? L::PV_EMPTY : L::QK_EMPTY);
    const uint32_t un_full = leader_bar(pv ? L::PV_FULL : L::QK_FULL);
    const int st_slots = pv ? L::PStSlots : L::QStSlots;
    constexpr int un_slots = L::QKSlots;
    static_assert(L::QKSlots == L::PVSlots, "one ring depth");
    uint8_t* const ring = smem + (pv ? L::OffPVRing : L::OffQKRing) + row * 128;
    const uint8_t* const st_base = smem + (pv ? L::OffPSt : L::OffQSt);
    const uint32_t st_bytes = pv ? L::PStBytes : kStageBytes;
    // staged codes: 16-byte piece 2 x + q of a 64-byte row, x the unit (QK) or
    // the half (PV); 4096-byte box the half (QK) or the unit (PV)
    const uint32_t x0 = (uint32_t)(q ^ ((row >> 1) & 3)) << 4, x1 = x0 ^ 32u;
    // A NaN scale stays one in the scores, which is how the rows that see the key
    // get it, and counts as 0 among the values: there a row of the group whose
    // causal limit hides the key would take 0 times NaN.
    const uint32_t nan = pv ? 0u : 0x7FFF7FFFu;
    // the two 8-byte groups of block scales: the halves' pages (QK), the units' columns (PV)
    const uint32_t scl_g = pv ? 16 : L::PageScl, ts_a = pv ? 0 : L::PageScl;
    RingPos unit, stage;
    uint32_t gt = 0;
    SegmentWalker walk(p, w, t);
    Segment s;
    bool ok = true;
    while (ok && walk.next(s)) {
      if (s.n_pages == 0) continue;
      const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
      for (int it = 0; it < n_tiles && ok; ++it, ++gt) {
        const uint8_t* const scl_t = smem + L::OffScl + (gt & 1) * L::SclBytes;
        if (!pv) {
          ok = mbar_wait(bar(L::SCL_FULL + (gt & 1)), (gt >> 1) & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);  // the warp leaves together
          if (!ok) break;
        }
        const int pg0 = s.page_lo + it * kTilePages;
        const int npg = min(kTilePages, s.n_pages - it * kTilePages);
        // pages of the k^R unit (looked up here, loaded at the tile's end)
        int kr_page[2] = {-1, -1};
        if (!pv && ct == 0)
          for (int i = 0; i < 2; ++i) {
            const int tp = tile_page(2 * (int)rank + i);
            if (tp < npg) kr_page[i] = page_of(s.b, pg0 + tp);
          }
#pragma unroll 1
        for (int c = 0; c < 4 && ok; ++c) {
          // QK: columns [128 c, 128 c + 128) of this CTA's two pages.  PV: key
          // position c (page tile_page(c)); rows past its visible keys are zero
          const int tp = tile_page(c);
          const bool live = !pv || (tp < npg && row < s.nvis - (pg0 + tp) * kPage);
          ok = mbar_wait(st_full + 8 * stage.slot, stage.phase, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);  // the warp leaves together
          if (!ok) break;
          const uint8_t* const src = st_base + stage.slot * st_bytes + row * 64;
          const uint8_t* const scl = pv ? st_base + stage.slot * st_bytes + kStageBytes : scl_t;
          const uint8_t* const sclr = scl + row * 32 + (pv ? 8 * (int)rank : 8 * c);
          const uint8_t* const tsr = scl + 2048 + row * 4;
          const uint2 g0 = *reinterpret_cast<const uint2*>(sclr), g1 = *reinterpret_cast<const uint2*>(sclr + scl_g);
          const float t0 = *reinterpret_cast<const float*>(tsr), t1 = *reinterpret_cast<const float*>(tsr + ts_a);
          // the thread's two blocks of each (unit, half)
          uint32_t s00 = block_scales(g0.x >> (16 * q), nan, t0);
          uint32_t s01 = block_scales((pv ? g0.y : g1.x) >> (16 * q), nan, t1);
          uint32_t s10 = block_scales((pv ? g1.x : g0.y) >> (16 * q), nan, t0);
          uint32_t s11 = block_scales(g1.y >> (16 * q), nan, t1);
          if (!live) s00 = s01 = s10 = s11 = 0;  // rows past the end: their bytes may be anything
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const uint4 v[2] = {*reinterpret_cast<const uint4*>(src + (pv ? u * 4096 + x0 : u ? x1 : x0)),
                                *reinterpret_cast<const uint4*>(src + (pv ? u * 4096 + x1 : 4096 + (u ? x1 : x0)))};
            const uint32_t sc[2] = {u ? s10 : s00, u ? s11 : s01};
            ok = mbar_wait(un_empty + 8 * unit.slot, unit.phase ^ 1, abort_flag, p.status);
            ok = __all_sync(0xffffffffu, ok);  // the warp leaves together
            if (!ok) break;
            uint8_t* const dst = ring + unit.slot * kUnitBytes;
#pragma unroll
            for (int a = 0; a < 2; ++a) store_e2m1x32(dst + a * 8192, u0, v[a], sc[a]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(un_full + 8 * unit.slot);
            unit.advance(un_slots);
          }
          if (!ok) break;
          if (lane == 0) mbar_arrive_local(st_empty + 8 * stage.slot);
          stage.advance(st_slots);
        }
        if (!ok) break;
        if (!pv) {
          // k^R unit: bf16 rows by TMA into the ring slot, one box per page; the
          // first warp's arrival on the leader carries both CTAs' bytes
          ok = mbar_wait(un_empty + 8 * unit.slot, unit.phase ^ 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);  // the warp leaves together
          if (!ok) break;
          if (lane == 0) {
            const uint32_t fb = un_full + 8 * unit.slot;
            if (ct == 0) {
              if (rank == 0) mbar_expect_tx(bar(L::QK_FULL + unit.slot), 2 * kUnitBytes);
              else mbar_arrive_cluster(fb);
              for (int i = 0; i < 2; ++i)
                tma_load_3d_pair(sbase + L::OffQKRing + unit.slot * kUnitBytes + i * 8192, &P.map_kr, 0, 0,
                                 kr_page[i], fb);
            } else {
              mbar_arrive_cluster(fb);
            }
            mbar_arrive_local(bar(L::SCL_EMPTY + (gt & 1)));
          }
          __syncwarp();
          unit.advance(un_slots);
        }
      }
    }
  };
  auto load_qk = [&]() {
      // -------------------------------------------------------------- TMA: Q, QK
      if (lane == 0 && !stall) {
        RingProducer ring{L::QStSlots, 1, 0};
        const uint32_t empty0 = bar(L::QST_EMPTY);
        const int y_pages = 2 * (int)rank;  // this CTA's key positions of a tile (pages tile_page(...))
        SegmentWalker walk(p, w, t);
        Segment s;
        uint32_t seg = 0, gtile = 0;
        bool ok = true;
        while (ok && walk.next(s)) {
          if (s.n_pages == 0) continue;
          // absorbed queries of this CTA's 64 heads for (b, t)
          if (seg > 0) ok = mbar_wait(bar(L::Q_EMPTY), (seg - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          // one barrier per 64-column chunk: the first tile's MMAs of unit c
          // wait only for chunk c
          if (rank == 0)
            for (int c = 0; c < kChunks; ++c) mbar_expect_tx(bar(L::Q_FULL + c), 2 * 8192);
          const int qrow = s.b * n_rows + row0;
          for (int c = 0; c < kChunks; ++c)
            tma_load_2d_pair(sbase + L::OffQ + c * 8192, &P.map_q, 64 * c, qrow, leader_bar(L::Q_FULL + c));
          const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
          for (int it = 0; it < n_tiles && ok; ++it) {
            const int pg0 = s.page_lo + it * kTilePages;
            const int npg = min(kTilePages, s.n_pages - it * kTilePages);
            // this CTA's pages; pages past the tile's end come from outside the
            // tensor (zero fill)
            int pg[2];
            for (int i = 0; i < 2; ++i) {
              const int tp = tile_page(y_pages + i);
              pg[i] = tp < npg ? page_of(s.b, pg0 + tp) : -1;
            }
            // this CTA's pages two tiles ahead (at a segment's start also one
            // ahead) go to L2 now, so that the staging loads find them there.
            // Invalid entries are skipped here and reported when their tile is loaded.
            for (int d = it == 0 ? 1 : 2; d <= 2 && it + d < n_tiles; ++d) {
              const int pgp = s.page_lo + (it + d) * kTilePages;
              const int npgp = min(kTilePages, s.n_pages - (it + d) * kTilePages);
              for (int i = 0; i < 2; ++i) {
                const int tp = tile_page(y_pages + i);
                if (tp >= npgp) continue;
                const int page = p.page_table[(size_t)s.b * p.max_pages + pgp + tp];
                if (page >= 0 && page < p.num_pages)
                  prefetch_l2(p.pool + (size_t)page * p.page_bytes, (uint32_t)p.page_bytes);
              }
            }
            // scales of this CTA's two pages (a page past the tile's end: the first
            // page's scales; its scores are masked)
            const uint32_t sb = gtile & 1;
            ok = mbar_wait(bar(L::SCL_EMPTY + sb), ((gtile >> 1) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            const uint32_t fb = bar(L::SCL_FULL + sb);
            mbar_arrive_tx_local(fb, L::SclBytes);
            for (int i = 0; i < L::SclPages; ++i)
              bulk_load(sbase + L::OffScl + sb * L::SclBytes + i * L::PageScl,
                        p.pool + (size_t)(pg[i] >= 0 ? pg[i] : page_of(s.b, pg0)) * p.page_bytes + P.scl_off, L::PageScl, fb);
            ++gtile;
            // codes of columns [64c, 64c + 128) of both pages, for two units: one staging slot
#pragma unroll 1
            for (int c = 0; c < kChunks - 1; c += 2) {
              uint32_t slot;
              if (!ring.claim(empty0, slot, ok, abort_flag, p.status)) continue;
              const uint32_t dst = sbase + L::OffQSt + slot * kStageBytes, qb = bar(L::QST_FULL + slot);
              mbar_arrive_tx_local(qb, kStageBytes);
              for (int i = 0; i < 2; ++i) tma_load_3d(dst + i * 4096, &P.map_codes, 32 * c, 0, pg[i], qb);
            }
          }
          ++seg;
        }
      }
  };
  auto load_pv = [&]() {
      // ------------------------------------------------------------------ TMA: PV
      if (lane == 0 && !stall) {
        RingProducer ring{L::PStSlots, 1, 0};
        const uint32_t empty0 = bar(L::PST_EMPTY);
        const int x_pv = 128 * (int)rank;  // this CTA's 128 columns of an N=256 half
        SegmentWalker walk(p, w, t);
        Segment s;
        bool ok = true;
        while (ok && walk.next(s)) {
          if (s.n_pages == 0) continue;
          const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
          for (int it = 0; it < n_tiles && ok; ++it) {
            const int pg0 = s.page_lo + it * kTilePages;
            const int npg = min(kTilePages, s.n_pages - it * kTilePages);
            // key position i (page tile_page(i))
#pragma unroll 1
            for (int i = 0; i < kTilePages; ++i) {
              const int tp = tile_page(i);
              const int valid = tp < npg ? min(kPage, s.nvis - (pg0 + tp) * kPage) : 0;
              const int page = valid > 0 ? page_of(s.b, pg0 + tp) : 0;
              uint32_t slot;  // holds both N-halves' codes
              if (!ring.claim(empty0, slot, ok, abort_flag, p.status)) continue;
              const uint32_t fb = bar(L::PST_FULL + slot), dst = sbase + L::OffPSt + slot * L::PStBytes;
              mbar_arrive_tx_local(fb, kStageBytes + (valid > 0 ? L::PageScl : 0));
              for (int jj = 0; jj < 2; ++jj)
                tma_load_3d(dst + jj * 4096, &P.map_codes, (256 * jj + x_pv) / 2, 0, valid > 0 ? page : -1, fb);
              if (valid > 0)  // (no key of the page visible: the converters read no scale)
                bulk_load(dst + kStageBytes, p.pool + (size_t)page * p.page_bytes + P.scl_off, L::PageScl, fb);
            }
          }
        }
      }
  };
  auto issue_qk = [&]() {
      // ----------------------------------------------------------- MMA: S = Q K^T
      if (rank == 0 && lane == 0) {
        RingConsumer ring{bar(L::QK_FULL), bar(L::QK_EMPTY), L::QKSlots};
        SegmentWalker walk(p, w, t);
        Segment s;
        uint32_t g = 0, seg = 0;
        bool ok = true;
        // descriptors advance by adding (byte offset >> 4) to the start-address field
        const uint64_t qdesc = sdesc(sbase + L::OffQ, 16, 1024);      // chunk c: + 512 c; K-step: + 2
        const uint64_t kdesc = sdesc(sbase + L::OffQKRing, 16, 1024);  // slot: + 1024 slot
        while (ok && walk.next(s)) {
          if (s.n_pages == 0) continue;
          const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
          for (int it = 0; it < n_tiles && ok; ++it, ++g) {
            ok = mbar_wait(bar(L::S_FREE + (g & 1)), ((g >> 1) & 1) ^ 1, abort_flag, p.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sd = tmem + ((g & 1) ? kColS1 : kColS0);
#pragma unroll 1
            for (int c = 0; c < kQKUnits; ++c) {
              if (it == 0) {  // the segment's queries, chunk c
                ok = mbar_wait(bar(L::Q_FULL + c), seg & 1, abort_flag, p.status);
                if (!ok) break;
              }
              ok = ring.wait_full(abort_flag, p.status);
              if (!ok) break;
              tc_fence_after();
              const uint64_t a = qdesc + 512 * c, bb = kdesc + 1024 * ring.pos.slot;
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4)  // 16 columns = 32 bytes into the swizzled rows
                tc_mma(sd, a + 2 * k4, bb + 2 * k4, c == kChunks - 1 ? kIdescQKb : kIdescQK, (c | k4) ? 1u : 0u);
              ring.release();
            }
            if (!ok) break;
            tc_commit_pair(bar(L::S_FULL + (g & 1)));
            if (it == n_tiles - 1) tc_commit_pair(bar(L::Q_EMPTY));
          }
          ++seg;
        }
        // completes, in both CTAs, once every MMA this thread issued has finished
        tc_commit_pair(bar(L::DRAIN));
      }
  };
  auto issue_pv = [&]() {
      // ---------------------------------------------------------- MMA: O += P C
      if (rank == 0 && lane == 0) {
        RingConsumer ring{bar(L::PV_FULL), bar(L::PV_EMPTY), L::PVSlots};
        SegmentWalker walk(p, w, t);
        Segment s;
        uint32_t g = 0, seg = 0;
        bool ok = true;
        const uint64_t vdesc = sdesc(sbase + L::OffPVRing, 8192, 1024);  // slot: + 1024 slot; K-step: + 128
        const uint64_t pdesc = sdesc(sbase + L::OffP, 16, 1024);         // page sub-tile: + 512 i; K-step: + 2
        while (ok && walk.next(s)) {
          if (s.n_pages == 0) continue;
          const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
          for (int it = 0; it < n_tiles && ok; ++it, ++g) {
            ok = mbar_wait(bar(L::P_FULL), g & 1, abort_flag, p.status);
            if (!ok) break;
            if (it == 0 && seg > 0) {  // O of the previous segment must be read out first
              ok = mbar_wait(bar(L::O_FREE), (seg - 1) & 1, abort_flag, p.status);
              if (!ok) break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < kTilePages && ok; ++i) {
              if (i == 2) {  // P of the upper key positions comes on its own
                ok = mbar_wait(bar(L::P_FULL2), g & 1, abort_flag, p.status);
                if (!ok) break;
                tc_fence_after();
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                ok = ring.wait_full(abort_flag, p.status);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  tc_mma(tmem + (j ? kColO1 : kColO0), pdesc + 512 * i + 2 * ks,
                         vdesc + 1024 * ring.pos.slot + 128 * ks, kIdescPV, (it == 0 && i == 0 && ks == 0) ? 0u : 1u);
                ring.release();
              }
              if (i == 1 && ok) tc_commit_pair(bar(L::P_FREE));
            }
            if (!ok) break;
            tc_commit_pair(bar(L::O_DONE));
          }
          ++seg;
        }
        tc_commit_pair(bar(L::DRAIN));
      }
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    softmax();
  } else if (warp >= L::QKConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    convert();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == L::QKProdWarp) load_qk();
    else if (warp == L::PVProdWarp) load_pv();
    else if (warp == L::QKWarp) issue_qk();
    else if (warp == L::PVWarp) issue_pv();
  }

  // teardown: every TMEM access of both CTAs is finished before deallocation
  tc_fence_before();
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  // After an abort by either CTA (whichever gave up set both flags before its
  // cluster arrival, so both CTAs read the same value here): wait, bounded,
  // for the MMAs issued so far, give bulk copies in flight time to land, and
  // meet the peer again, so that neither CTA's shared memory or tensor memory
  // goes while an operation of the pair may still use it.
  if (*abort_flag) {
    if (threadIdx.x == 0) {
      mbar_wait_for(bar(L::DRAIN), 0, kDrainLimitCycles);
      const unsigned long long t0 = global_ns();
      while (global_ns() - t0 < kCopyGraceNs) {
      }
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
  }
  tl_end_nosync(p.timeline, MLA_TRACE_ATTEND);
  if (warp == L::QKWarp) {
    // every MMA of the pair has completed (the issuers' final commits; already
    // so on the normal path, where the softmax warps waited for the last ones)
    if (lane == 0) mbar_wait_for(bar(L::DRAIN), 0, kDrainLimitCycles);
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace

cudaError_t launch_decode_tc_fp4(const DecodeParams& p, cudaStream_t st) {
  TcParams tp;
  memset(&tp, 0, sizeof(tp));
  tp.p = p;
  tp.groups = (p.n_q * p.d.n_heads + kHeads - 1) / kHeads;
  const uint64_t q_rows = (uint64_t)p.batch * p.n_q * p.d.n_heads;
  const Fp4Page f4 = fp4_page(kPage, kDC, kDR);
  tp.scl_off = f4.sc_off;
  if (!make_o_map(&tp.map_o, p.o_part, (uint64_t)p.n_q * p.n_slots * p.d.n_heads) ||
      !make_map(&tp.map_q, p.q_abs, q_rows, 64, CU_TENSOR_MAP_DATA_TYPE_FLOAT16) ||
      !make_page_map(&tp.map_codes, p.pool, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, kDC / 2, p.num_pages, p.page_bytes, 64,
                     CU_TENSOR_MAP_SWIZZLE_64B) ||
      !make_page_map(&tp.map_kr, p.pool + f4.kr_off, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, kDR, p.num_pages,
                     p.page_bytes, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e =
      cudaFuncSetAttribute(decode_tc_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_tc_fp4_kernel, dim3(2 * tp.groups * p.splits), dim3(L::Threads), L::SmemBytes, st, tp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
