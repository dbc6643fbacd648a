// Parts of the tcgen05 decode kernels (decode_tc.cu: bf16 and FP8 caches;
// decode_tc_fp4.cu: 4-bit cache): the shape, PTX helpers, the partition of the
// keys among CTA pairs, the rings, and the tensor maps.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>

#include <cstring>

#include "mla_internal.cuh"

namespace mla {

namespace {

// ---------------------------------------------------------------------------
// Fixed shape of the tcgen05 decode kernels
// ---------------------------------------------------------------------------
constexpr int kHeads = 128, kHalfHeads = 64;
constexpr int kDC = 512, kDR = 64, kD = kDC + kDR;  // 576
constexpr int kPage = 64;                             // keys per cache page
constexpr int kTilePages = 4;                         // pages per tile: 256 keys = N of the QK MMA
constexpr int kChunks = kD / 64;                      // 9 column chunks of 64 (128 B)
constexpr int kQKUnits = kChunks;                     // QK units per tile

constexpr uint32_t kUnitBytes = 16384;                // operand unit: this CTA's share of four MMAs
constexpr uint32_t kStageBytes = 8192;                // staging slot: raw page data (FP8: of one unit, 4-bit: of two)
constexpr uint32_t kQBytes = kChunks * 64 * 128;      // 73728: 64 heads x 576 (16-bit)
constexpr uint32_t kPBytes = kTilePages * 64 * 128;   // 32768: 64 heads x 256 keys (16-bit), 4 sub-tiles

// TMEM columns (per CTA, 2x2 layout): S buffers 128 columns each, O 2 x 128
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 384;

constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr long long kWaitLimitCycles = 4000000000LL;  // ~2 s
// after an abort: the bound on the wait for the issued MMAs, and the time
// given to bulk copies whose completion this CTA cannot observe (its half of a
// pair load completes on the leader's barrier); both far above the latency of
// the operation
constexpr long long kDrainLimitCycles = 20000000LL;   // ~10 ms
constexpr unsigned long long kCopyGraceNs = 200000ull;  // 200 us

// instruction descriptors (kind::f16, dense, f32 accumulator; operands bf16
// or f16, the same for A and B)
constexpr uint32_t idesc(int M, int N, bool a_mn, bool b_mn, bool f16) {
  return (1u << 4) | (f16 ? 0u : ((1u << 7) | (1u << 10))) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------------------------------
// Protocol timestamps for development builds (-DMLA_TC_TRACE): event e of
// tile g in CTA b, read back with mla_tc_trace_read.  Absent otherwise.
// ---------------------------------------------------------------------------
#ifdef MLA_TC_TRACE
constexpr int kTrCtas = 8, kTrTiles = 48, kTrEvents = 16;
__device__ unsigned long long g_tc_trace[kTrCtas * kTrTiles * kTrEvents];
__device__ __forceinline__ void tc_trace(int e, uint32_t g) {
  if (blockIdx.x < kTrCtas && g < kTrTiles) {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    g_tc_trace[(blockIdx.x * kTrTiles + g) * kTrEvents + e] = t;
  }
}
#define TC_TRACE(e, g) tc_trace((e), (g))
#define TC_TRACE_VAL(e, g, v)                                                        \
  do {                                                                               \
    if (blockIdx.x < kTrCtas && (g) < kTrTiles)                                      \
      g_tc_trace[(blockIdx.x * kTrTiles + (g)) * kTrEvents + (e)] = (unsigned long long)(v); \
  } while (0)
#else
#define TC_TRACE(e, g) ((void)0)
#define TC_TRACE_VAL(e, g, v) ((void)0)
#endif

// ---------------------------------------------------------------------------
// PTX helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// arrive on a barrier given by its shared::cluster address (own or peer CTA)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Give up the CTA pair's work: set this CTA's abort flag and the peer's (a
// distributed shared memory store), so that every role of both CTAs stops at
// its next wait instead of running into its own limit.
__device__ __forceinline__ void raise_abort(volatile int* abort_flag) {
  *abort_flag = 1;
  const uint32_t peer = map_to_rank(smem_u32((const void*)abort_flag), cluster_rank() ^ 1u);
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer), "r"(1u) : "memory");
}

// Bounded wait.  Returns false (and records MLA_ERR_TIMEOUT) if the phase does
// not complete within the limit, or false at once if a role of this CTA or of
// the peer CTA already gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      raise_abort(abort_flag);
      record_status(status, MLA_ERR_TIMEOUT);
      return false;
    }
  }
}

// Bounded wait that ignores the abort flag (the teardown after an abort).
__device__ __forceinline__ bool mbar_wait_for(uint32_t bar, uint32_t parity, long long limit_cycles) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit_cycles) return false;
  return true;
}

// The 128 softmax threads agree on a wait's outcome: true only if it succeeded
// for all of them (a barrier with an AND reduction on named barrier 1), so
// that they leave their loop together and never wait at a named barrier for a
// warp that has gone.
__device__ __forceinline__ bool softmax_all_ok(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)__all_sync(0xffffffffu, ok))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tc_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc_,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc_), "r"(accumulate)
      : "memory");
}

// arrive on the barrier at this offset in both CTAs of the pair when all
// tcgen05 operations issued so far by this thread complete
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Scores of keys at or past `nvis` (a sub-tile's visible count) set to -inf,
// so that they drop out of the max and their exponentials are 0.
__device__ __forceinline__ void mask_scores(uint32_t (&sr)[64], int nvis) {
  if (nvis < 64) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (j >= nvis) sr[j] = 0xFF800000u;
  }
}
// max of 64 scores in eight independent chains
__device__ __forceinline__ float max64(const uint32_t (&sr)[64]) {
  float m8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m8[j] = __uint_as_float(sr[j]);
#pragma unroll
  for (int j = 8; j < 64; ++j) m8[j & 7] = fmaxf(m8[j & 7], __uint_as_float(sr[j]));
  return fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
}

// Shared-memory matrix descriptor, 128-byte swizzle, sm_100 version field.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// shared -> global tensor store (bulk group of this thread)
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// arrive on a barrier of this CTA with an expected transaction count
__device__ __forceinline__ void mbar_arrive_tx_local(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------------------
// Work partition (shared by all roles): split w of query t covers global key
// tiles [w*TT/W, (w+1)*TT/W); pieces per sequence are segments.
// ---------------------------------------------------------------------------
struct Segment {
  int b, page_lo, n_pages, nvis;  // n_pages: pages with at least one visible key
};

struct SegmentWalker {
  const int32_t* ts;
  const int32_t* seq_lens;
  int batch, n_q, t, b;
  long long g, g1;
  __device__ SegmentWalker(const DecodeParams& p, int w, int t_) {
    ts = p.plan;
    seq_lens = p.seq_lens;
    batch = p.batch;
    n_q = p.n_q;
    t = t_;
    const long long TT = ts[batch];
    g = split_tile_begin(w, TT, p.splits);
    g1 = split_tile_begin(w + 1, TT, p.splits);
    b = g < g1 ? seq_of_tile(ts, batch, g) : 0;
  }
  __device__ bool next(Segment& s) {
    if (g >= g1) return false;
    while ((long long)ts[b + 1] <= g) ++b;
    const long long end = min(g1, (long long)ts[b + 1]);
    s.b = b;
    s.page_lo = (int)(g - ts[b]);
    const int page_hi = (int)(end - ts[b]);
    s.nvis = seq_lens[b] - n_q + t + 1;
    const int vis_pages = (s.nvis + kPage - 1) / kPage;
    s.n_pages = max(0, min(page_hi, vis_pages) - s.page_lo);
    g = end;
    return true;
  }
};

// Page of a tile at key position pos (0..3; the order of the S columns and
// the P sub-tiles: the leader's two pages, then the peer's): CTA r of the pair
// holds pages r and r + 2, so a tile of two pages puts one page in each CTA.
__device__ __forceinline__ int tile_page(int pos) { return (pos >> 1) + 2 * (pos & 1); }

// Bulk prefetch of [ptr, ptr + bytes) into L2 (16-byte aligned, bytes % 16 == 0).
__device__ __forceinline__ void prefetch_l2(const void* ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

// L2 prefetch of the pages of a CTA's first key tile, issued before the
// grid-dependency wait by one warp (batch <= 32).  It reads only inputs of the
// call (sequence lengths, page table), never the preceding kernel's output,
// and a prefetch cannot change a result: at worst it fetches pages that go
// unused.  The split of pages is the plan's rule; CTA `rank` of the pair
// takes pages rank and rank + 2 of the tile.
__device__ __noinline__ void prefetch_first_tile(const DecodeParams& p, int w, int rank, int lane) {
  int pages = 0;
  if (lane < p.batch) {
    const int len = p.seq_lens[lane];
    if (len >= 1 && (long long)len <= (long long)p.max_pages * kPage) pages = (len + kPage - 1) / kPage;
  }
  int incl = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const int excl = incl - pages;
  const long long TT = __shfl_sync(0xffffffffu, incl, 31);
  const long long g0 = split_tile_begin(w, TT, p.splits), g1 = split_tile_begin(w + 1, TT, p.splits);
  const unsigned own = __ballot_sync(0xffffffffu, lane < p.batch && excl <= g0 && g0 < incl);
  const int b0 = own ? __ffs(own) - 1 : 0;
  const int e0 = __shfl_sync(0xffffffffu, excl, b0), i0 = __shfl_sync(0xffffffffu, incl, b0);
  if (g0 < g1 && own && lane < 2) {
    const long long lp = g0 - e0 + tile_page(2 * rank + lane);  // page of sequence b0
    if (lp < min(g1, (long long)i0) - e0) {
      const int page = p.page_table[(size_t)b0 * p.max_pages + lp];
      if (page >= 0 && page < p.num_pages) prefetch_l2(p.pool + (size_t)page * p.page_bytes, (uint32_t)p.page_bytes);
    }
  }
}

// Position in a ring of `slots` slots: slot index and the parity of its use.
struct RingPos {
  uint32_t slot = 0, phase = 0;
  __device__ void advance(int slots) {
    if (++slot == (uint32_t)slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// Producer side of one ring: producer pid of n issues every n-th entry of the
// ring's consumption order; every producer walks the same schedule, so the
// ring position of each entry is known to all of them.
struct RingProducer {
  int slots, producers, pid;
  RingPos pos;
  uint32_t entry = 0;
  // Claim the next entry: returns true (with its slot) when this producer
  // issues it, after waiting for the slot to be free.
  __device__ bool claim(uint32_t empty0, uint32_t& slot, bool& ok, volatile int* abort_flag, int* status) {
    const bool mine = (int)(entry % (uint32_t)producers) == pid;
    const RingPos cur = pos;
    ++entry;
    pos.advance(slots);
    if (!mine || !ok) return false;
    if (!mbar_wait(empty0 + 8 * cur.slot, cur.phase ^ 1, abort_flag, status)) {
      ok = false;
      return false;
    }
    slot = cur.slot;
    return true;
  }
};

// Consumer side of one operand ring (the MMA-issuing thread of the leader).
struct RingConsumer {
  uint32_t full0, empty0;
  int slots;
  RingPos pos;
  __device__ bool wait_full(volatile int* abort_flag, int* status) {
    return mbar_wait(full0 + 8 * pos.slot, pos.phase, abort_flag, status);
  }
  // the unit's MMAs are issued: free the slot in both CTAs once they complete
  __device__ void release() {
    tc_commit_pair(empty0 + 8 * pos.slot);
    pos.advance(slots);
  }
};

// ---------------------------------------------------------------------------
// Host side: tensor maps
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

// 2-D 16-bit map over [rows][576] with a (64 columns x box_rows) box, 128-byte swizzle
inline bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows,
              CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kD, rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// 3-D map over a page sub-block: [pages][64 rows][row_elems], box
// (box_x x 64 rows x 1 page)
inline bool make_page_map(CUtensorMap* m, const void* base, CUtensorMapDataType type, uint32_t elem_bytes,
                   uint64_t row_elems, uint64_t num_pages, uint64_t page_bytes, uint32_t box_x,
                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_NONE) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {row_elems, (cuuint64_t)kPage, num_pages};
  const cuuint64_t strides[2] = {row_elems * elem_bytes, page_bytes};
  const cuuint32_t box[3] = {box_x, (cuuint32_t)kPage, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

inline bool device_is_sm100() {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  return major == 10 && minor == 0;
}

// o_part as a 2-D tensor of 16-bit values [rows][512], box 64 x 64, 128-byte swizzle
inline bool make_o_map(CUtensorMap* m, void* base, uint64_t rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kDC, rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kDC * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)kHalfHeads};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

}  // namespace mla
