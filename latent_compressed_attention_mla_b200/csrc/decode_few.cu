// S3 over the 4-bit latent cache for at most 16 query rows (heads times query
// tokens: a tensor-parallel shard's 16 heads, or 8 with two tokens): split-KV
// attention of the absorbed queries on the warp-level tensor cores.
//
// What it computes is decode_tc.cu's (scores of [q~ | q^R] against the rows
// [c | k^R], online softmax, probability-weighted sum of the latent rows; W^UV
// afterwards in the combine kernel).  With c = code * s * ts (ts the token's
// power of two, 2^e) the rows enter in units of ts:
//   S = scale (q~ . c + q^R . k^R) = scale ts (q~ . (code s) + (q^R . k^R) / ts)
//   O = sum_k 2^(S_k + e_k - r) (code s)_k,   l = sum_k 2^(S_k - r),
// S in log2 units, r the row's reference (a running maximum of S + e): code * s
// is exact in f16 whatever the latent's magnitude, and the probabilities carry
// the tokens' scales.  (l takes a probability times 2^-e, so one that ex2 flushes,
// below 2^-126, is missing in l: with the scales of a sequence within 2^100 of one
// another, a key of weight below 2^-26.)
//
// Why warp-level MMA and not tcgen05: 16 rows against 420 bytes a key are bound
// by HBM (35 kFLOP a key), and a tcgen05 operand has to lie in shared memory as
// 16-bit values: written once and read twice, 3.3 KB a key, 26 cycles of an
// SM's shared-memory bandwidth against the 19 cycles the key's bytes take from
// HBM.  Here the codes are read from shared memory as they are (twice 256
// bytes) and become MMA fragments in registers.
//
// One CTA (eight warps and a load producer) runs one split of the keys in
// tiles of 128 (two pages):
//   scores  warp (kg, dq): 32 keys x half of the columns.  The contraction
//           order is the codes' own (a thread's 32 consecutive codes of a key
//           are the B fragments of eight k-steps); the query fragments lie in
//           shared memory in that order.  The halves' sums meet in shared memory.
//   softmax warp (kg, dq) finishes 16 keys x all rows; the reference moves only
//           when a score passes it by 2^8; P goes out as f16
//   values  warp ds: 64 columns x all keys; a thread takes eight consecutive
//           codes of two keys at a time, whose interleaved nibbles convert into
//           the B fragments of eight n-tiles
// Keys of a group of eight are taken in the order n ^ (4 if n is odd), with
// which both the 16-byte and the 4-byte reads of the 128-byte-swizzled pages
// (TMA) spread over all banks; the block scales carry the 32-byte swizzle.
// A warp interleaves the scores of tile i + 1 with the values of tile i: two
// independent streams of conversions and MMAs (two warps a scheduler are too
// few to hide one stream's latencies; P is double-buffered).
//
// Measured (16 heads, this kernel's span on the device): 128 sequences of 16,385 keys
// 360 us, 2.4 TB/s of cache rows; 8 of 131,073 188 us.  HBM would allow 135 and 68;
// loads alone take 148.  Each code becomes f16 twice (scores, values): per 128 keys a
// scheduler issues 272 MMAs (8.6 cycles each), 512 conversions of two codes (2) and
// 512 multiplies, 3,900 cycles end to end of the 6,400 that a tile takes.  The rest,
// some 40%, is latency between the phases: the exchange of the score halves, the
// softmax and the barrier run with the tensor and conversion pipes (30% and 36%
// busy) idle.  Twice the warps with half the work each (+1%) and two teams of eight
// on alternate pages, one's softmax beside the other's products (+4%), did not hide
// it.  On the way: one phase for scores, one for values +32%; query fragments in
// registers, not shared memory +9%.
#include <cuda.h>

#include <cstring>

#include "mla_internal.cuh"
#include "mma_tile.cuh"

namespace mla {

namespace {

constexpr int kDC = 512, kDR = 64, kD = kDC + kDR, kPage = 64;
constexpr int kMaxRows = 16;
constexpr int kWarps = 8, kThreads = 32 * kWarps + 128;  // and a warpgroup of which one warp issues the loads
constexpr int kTilePages = 2, kTileKeys = kTilePages * kPage;
constexpr int kStages = 3;
constexpr uint32_t kCodeBytes = kPage * kDC / 2;  // codes of a page: two 8 KB boxes of 256 columns
constexpr uint32_t kKrBytes = kPage * kDR * 2;
constexpr uint32_t kSclBytes = kPage * kDC / 16, kTsBytes = kPage * 4;  // block scales, token scales
constexpr uint32_t kStageBytes = kTilePages * (kCodeBytes + kKrBytes);
constexpr int kSteps = 18;                        // k-steps of a half: 16 of codes, 2 of k^R
constexpr float kRescaleThreshold = 8.0f;         // log2 units
constexpr unsigned long long kCopyGraceNs = 200000ull;

constexpr uint32_t kOffScl = kStages * kStageBytes;                      // [kStages][kTilePages][kSclBytes]
constexpr uint32_t kOffTs = kOffScl + kStages * kTilePages * kSclBytes;  // [kStages][kTilePages][kTsBytes]
constexpr uint32_t kXBytes = kWarps * 2 * 512;                           // [kWarps][2][32 lanes] float4
constexpr uint32_t kOffX = kOffTs + kStages * kTilePages * kTsBytes;
constexpr uint32_t kPBytes = kMaxRows * kTileKeys * 2;                   // [16][128 keys] f16, 16-byte units swizzled
constexpr uint32_t kOffP = kOffX + kXBytes;                              // two of them
constexpr uint32_t kOffQ = kOffP + 2 * kPBytes;                          // [2 halves][kSteps][32 lanes] fragments
constexpr uint32_t kOffMax = kOffQ + 2 * kSteps * 512;                   // int [16]
constexpr uint32_t kOffL = kOffMax + kMaxRows * 4;                       // float [kWarps][16]
constexpr uint32_t kOffBar = kOffL + kWarps * kMaxRows * 4;
constexpr uint32_t kOffAbort = kOffBar + 2 * kStages * 8;                // barriers: full, then empty, per stage
constexpr uint32_t kSmemBytes = kOffAbort + 8 + 1024;                    // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr long long kWaitLimitCycles = 4000000000LL;  // ~2 s

struct FewParams {
  DecodeParams p;
  int rows;               // query rows of a sequence (n_q * n_heads), at most 16
  size_t ts_off;          // token scales' offset in a page
  CUtensorMap map_codes;  // [pages][64 rows][256 bytes], box 128 bytes x 64 rows, 128-byte swizzle
  CUtensorMap map_kr;     // [pages][64 rows][64] bf16, box 64 x 64 rows, 128-byte swizzle
  CUtensorMap map_scl;    // [pages][64 rows][32 bytes], box 32 bytes x 64 rows, 32-byte swizzle
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// d += a * b, m16n8k16, f16 inputs, fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order-preserving map of floats to signed integers (for atomicMax).
__device__ __forceinline__ int float_order(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; false after ~2 s, or once another warp has given up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Barriers of the eight computing warps.
__device__ __forceinline__ void sync_warps() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool sync_warps_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// Four e4m3 codes with each NaN (0x7F and 0xFF) as 0.
__device__ __forceinline__ uint32_t drop_nan_e4m3(uint32_t x) {
  const uint32_t nan = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return x & ~((nan >> 7) * 0xFFu);
}

// Key of column n of a group of eight.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n & 1) << 2); }

// The pieces of the sequences in split w.
struct Piece {
  int b, page_lo, n_pages;
  int len, end;             // keys of the sequence; first key behind the piece's pages
};
struct PieceWalker {
  const DecodeParams* p;
  int b, g, g1;  // (the plan's prefix sums are 32-bit)
  __device__ PieceWalker(const DecodeParams& p_, int w) : p(&p_) {
    const long long TT = p->plan[p->batch];
    g = (int)split_tile_begin(w, TT, p->splits);
    g1 = (int)split_tile_begin(w + 1, TT, p->splits);
    b = g < g1 ? seq_of_tile(p->plan, p->batch, g) : 0;
  }
  __device__ bool next(Piece& s) {
    if (g >= g1) return false;
    while (p->plan[b + 1] <= g) ++b;
    const int start = p->plan[b], end = min(g1, p->plan[b + 1]);
    s.b = b;
    s.len = p->seq_lens[b];
    s.page_lo = g - start;
    s.end = (end - start) * kPage;
    s.n_pages = end - g;
    g = end;
    return true;
  }
};

__global__ void __launch_bounds__(kThreads, 1) decode_few_kernel(const __grid_constant__ FewParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const DecodeParams& p = P.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int w = blockIdx.x;
  int* s_max = reinterpret_cast<int*>(smem + kOffMax);
  float* s_l = reinterpret_cast<float*>(smem + kOffL);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  auto full = [&](int s) -> uint32_t { return sbase + kOffBar + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return sbase + kOffBar + 8u * (kStages + s); };

  pdl_trigger();
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init_local(full(s), 1);
      mbar_init_local(empty(s), kWarps);
    }
  }
  if (tid < kMaxRows) s_max[tid] = float_order(-INFINITY);
  __syncthreads();
  pdl_wait();
  tl_begin(p.timeline, MLA_TRACE_ATTEND);

  bool ok = true;
  // The launch gives 168 registers a thread (64,512 in all); the computing warps
  // take 224 (57,344), the load warpgroup keeps 56 (7,168).
  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ------------------------------------------------------------ loads: lane i
    // brings page i of each tile (looked up before the wait for its stage).
    // (Self-test of failure detection: no load is issued, the waits expire.)
    if (warp == kWarps && !(p.d.flags & MLA_FLAG_SELFTEST_STALL)) {
      PieceWalker walk(p, w);
      Piece s;
      int stage = 0, page = 0;
      uint32_t phase = 1;
      while (ok && walk.next(s)) {
        for (int at = 0; at < s.n_pages && ok; at += kTilePages) {
          const int npg = min(kTilePages, s.n_pages - at);
          if (lane < npg) page = p.page_table[(size_t)s.b * p.max_pages + s.page_lo + at + lane];
          ok = __all_sync(0xffffffffu, mbar_wait(empty(stage), phase, abort_flag));
          if (!ok) break;
          if (lane == 0) mbar_expect_local(full(stage), npg * (kCodeBytes + kKrBytes + kSclBytes + kTsBytes));
          __syncwarp();
          if (lane < npg) {
            if (page < 0 || page >= p.num_pages) {
              record_status(p.status, MLA_ERR_BOUNDS);
              page = 0;
            }
            const uint32_t st = sbase + stage * kStageBytes, fb = full(stage);
            for (int h = 0; h < 2; ++h)
              tma_load_3d(st + lane * kCodeBytes + h * (kCodeBytes / 2), &P.map_codes, 128 * h, 0, page, fb);
            tma_load_3d(st + kTilePages * kCodeBytes + lane * kKrBytes, &P.map_kr, 0, 0, page, fb);
            tma_load_3d(sbase + kOffScl + (stage * kTilePages + lane) * kSclBytes, &P.map_scl, 0, 0, page, fb);
            bulk_load(sbase + kOffTs + (stage * kTilePages + lane) * kTsBytes,
                      p.pool + (size_t)page * p.page_bytes + P.ts_off, kTsBytes, fb);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      ok = true;  // (a wait that gave up is the computing warps' to report)
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int kg = warp >> 1, dq = warp & 1;  // scores, softmax
    const int ds = warp;                      // values
    // This thread's places in a staged tile; the loops add multiples of eight
    // rows, which leave the swizzle as it is.
    const int qk_key = (32 * kg & 63) + key_of(g);  // scores: row of page kg / 2, + 8 nt
    const uint32_t qk_row = (uint32_t)((kg >> 1) * kCodeBytes + dq * (kCodeBytes / 2) + qk_key * 128);
    const uint32_t qk_codes0 = qk_row + ((q ^ (qk_key & 7)) << 4), qk_codes1 = qk_row + (((4 + q) ^ (qk_key & 7)) << 4);
    const uint32_t qk_kr = (uint32_t)(kTilePages * kCodeBytes + (kg >> 1) * kKrBytes + qk_key * 128 +
                                      (((2 * q + dq) ^ (qk_key & 7)) << 4));
    const uint32_t qk_scl = (uint32_t)((kg >> 1) * kSclBytes + qk_key * 32 + ((dq ^ ((qk_key >> 2) & 1)) << 4) + 2 * q);
    const uint32_t qk_ts = (uint32_t)((kg >> 1) * kTsBytes + (32 * kg & 63) * 4);
    const int k0 = 2 * q, k1 = key_of(2 * q + 1);   // keys of an accumulator's columns, of a value fragment's halves
    const uint32_t pv_col = (ds & 3) * 2 + (g >> 2);
    const uint32_t pv_box = (uint32_t)((ds >> 2) * (kCodeBytes / 2) + (g & 3) * 4);
    const uint32_t pv_codes0 = pv_box + k0 * 128 + ((pv_col ^ k0) << 4), pv_codes1 = pv_box + k1 * 128 + ((pv_col ^ k1) << 4);
    const uint32_t pv_scl0 = ((4 * ds + (g >> 1)) & 15) + k0 * 32 + (((ds >> 2) ^ ((k0 >> 2) & 1)) << 4);
    const uint32_t pv_scl1 = ((4 * ds + (g >> 1)) & 15) + k1 * 32 + (((ds >> 2) ^ ((k1 >> 2) & 1)) << 4);
    int qk_stage = 0, pv_stage = 0;
    uint32_t qk_phase = 0;
    PieceWalker walk(p, w);
    Piece s;
    while (ok && walk.next(s)) {
      // keys before the piece's end that the first and the last query token see
      const int nvis_lo = min(s.len - p.n_q + 1, s.end), nvis_hi = min(s.len, s.end);
      // Query fragments.  Step st < 16: contraction indexes 2q, 2q + 1 / 2q + 8,
      // 2q + 9 are columns 256 dq + 128 (st / 8) + 32 q + 4 (st % 8) + {0, 1} /
      // {2, 3}; steps 16, 17: k^R columns 16 q + 8 dq + 4 (st % 2) + {0, 1} / {2, 3} (bf16).
      // (The warps of kg 0 write both halves'; read after the barrier below.)
      const uint4* const qf = reinterpret_cast<const uint4*>(smem + kOffQ) + dq * kSteps * 32 + lane;
      if (kg == 0) {
        uint4* const qw = reinterpret_cast<uint4*>(smem + kOffQ) + dq * kSteps * 32 + lane;
        const __half* qa = static_cast<const __half*>(p.q_abs) + ((size_t)s.b * P.rows + g) * kD;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const int col = st < 16 ? 256 * dq + 128 * (st >> 3) + 32 * q + 4 * (st & 7)
                                  : kDC + 16 * q + 8 * dq + 4 * (st & 1);
          const uint2 lo = g < P.rows ? *reinterpret_cast<const uint2*>(qa + col) : make_uint2(0, 0);
          const uint2 hi = g + 8 < P.rows ? *reinterpret_cast<const uint2*>(qa + 8 * kD + col) : make_uint2(0, 0);
          qw[32 * st] = make_uint4(lo.x, hi.x, lo.y, hi.y);
        }
      }
      sync_warps();
      float o[8][4], m_ref[2] = {-INFINITY, -INFINITY}, l_sum[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
      for (int i = -1; i < n_tiles; ++i) {
        const bool more = i + 1 < n_tiles;
        const int key0 = (s.page_lo + (i + 1) * kTilePages) * kPage;  // tile i + 1
        if (more) {
          ok = mbar_wait(full(qk_stage), qk_phase, abort_flag) && ok;
          const int n_keys = nvis_hi - key0;
          if (n_keys < kTileKeys) {
            // keys that no row sees count as zero, whatever the page holds there
            for (int k = tid >> 2; k < kTileKeys; k += 8 * kWarps)
              if (k >= n_keys) {
                *reinterpret_cast<uint2*>(smem + kOffScl + qk_stage * kTilePages * kSclBytes + k * 32 + 8 * (tid & 3)) =
                    make_uint2(0, 0);
                if ((tid & 3) == 0)
                  *reinterpret_cast<float*>(smem + kOffTs + qk_stage * kTilePages * kTsBytes + k * 4) = 1.0f;
              }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later load overwrites them
            sync_warps();
          }
        }
        // -------------------------- scores of tile i + 1, values of tile i
        float acc[4][4];  // scores of four n-tiles of eight keys: two for the other half's warp, then its own
        const uint8_t* const q_st = smem + qk_stage * kStageBytes;
        const uint8_t* const q_scl = smem + kOffScl + qk_stage * kTilePages * kSclBytes + qk_scl;
        const uint32_t* const q_ts =
            reinterpret_cast<const uint32_t*>(smem + kOffTs + qk_stage * kTilePages * kTsBytes + qk_ts);
        auto work = [&](auto scores, auto values) {
          constexpr bool kScores = decltype(scores)::value, kValues = decltype(values)::value;
          const uint8_t* const v_st = smem + pv_stage * kStageBytes;
          const uint8_t* const v_scl = smem + kOffScl + pv_stage * kTilePages * kSclBytes;
          const uint32_t pa_addr = sbase + kOffP + (i & 1) * kPBytes + (lane & 15) * 256;
          uint4 v[4];
          uint32_t sc[4][2];
          if constexpr (kScores) {
            const uint4 q16 = qf[16 * 32], q17 = qf[17 * 32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int nt = (2 * dq + 2 + j) & 3;
              const uint4 kr = *reinterpret_cast<const uint4*>(q_st + qk_kr + nt * 1024);
              // (q^R . k^R) / ts of the accumulator's two keys
              const float i0 = __uint_as_float(0x7F000000u - q_ts[8 * nt + k0]);
              const float i1 = __uint_as_float(0x7F000000u - q_ts[8 * nt + k1]);
              acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
              mma_bf16(acc[j], *reinterpret_cast<const uint32_t(*)[4]>(&q16), kr.x, kr.y);
              mma_bf16(acc[j], *reinterpret_cast<const uint32_t(*)[4]>(&q17), kr.z, kr.w);
              acc[j][0] *= i0;
              acc[j][1] *= i1;
              acc[j][2] *= i0;
              acc[j][3] *= i1;
            }
          }
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            if constexpr (kScores) {
              // columns half t / 4; eight codes of each key: two k-steps
              if (t % 4 == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int nt = (2 * dq + 2 + j) & 3;
                  v[j] = *reinterpret_cast<const uint4*>(q_st + (t ? qk_codes1 : qk_codes0) + nt * 1024);
                  const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(q_scl + nt * 256 + 2 * t));
                  sc[j][0] = dup_lo(s2);
                  sc[j][1] = dup_hi(s2);
                }
              }
              const uint4 qa = qf[2 * t * 32], qb = qf[(2 * t + 1) * 32];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t c[4];
                e2m1x8_to_f16x2(t % 4 == 0 ? v[j].x : t % 4 == 1 ? v[j].y : t % 4 == 2 ? v[j].z : v[j].w, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = mul_f16x2(c[e], sc[j][(t % 4) >> 1]);
                mma_f16(acc[j], qa, c[0], c[1]);
                mma_f16(acc[j], qb, c[2], c[3]);
              }
            }
            if constexpr (kValues) {
              // columns 64 ds + 8 g .. + 7 of keys 16 t + {k0, k1} and 8 more; the codes of
              // the two keys are interleaved, so that a byte converts into the f16
              // pair of one column, and the pair of scales multiplies it
              const uint32_t kc = (t >> 2) * kCodeBytes + (t & 3) * 2048, ks = (t >> 2) * kSclBytes + (t & 3) * 512;
              uint4 pa;
              ldsm_x4(pa_addr + (((2 * t + (lane >> 4)) ^ (lane & 7)) << 4), pa.x, pa.y, pa.z, pa.w);
              uint32_t b[2][8];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w0 = *reinterpret_cast<const uint32_t*>(v_st + pv_codes0 + kc + h * 1024);
                const uint32_t w1 = *reinterpret_cast<const uint32_t*>(v_st + pv_codes1 + kc + h * 1024);
                const uint32_t s2 =
                    e4m3x2_to_f16x2(v_scl[pv_scl0 + ks + h * 256] | (uint32_t)v_scl[pv_scl1 + ks + h * 256] << 8);
                uint32_t he[4], ho[4];  // columns 0, 2, 4, 6 and 1, 3, 5, 7
                e2m1x8_to_f16x2((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), he);
                e2m1x8_to_f16x2(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), ho);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  b[h][2 * m] = mul_f16x2(he[m], s2);
                  b[h][2 * m + 1] = mul_f16x2(ho[m], s2);
                }
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) mma_f16(o[j], pa, b[0][j], b[1][j]);
            }
          }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (i < 0) work(Yes(), No());
        else if (more) work(Yes(), Yes());
        else work(No(), Yes());
        if (i >= 0) {
          __syncwarp();  // every lane has read tile i
          if (lane == 0) mbar_arrive(empty(pv_stage));
          pv_stage = pv_stage + 1 == kStages ? 0 : pv_stage + 1;
        }
        if (!more) break;
        // the other half's sums of the keys this warp finishes
        float4* const X = reinterpret_cast<float4*>(smem + kOffX) + lane;
#pragma unroll
        for (int j = 0; j < 2; ++j) X[warp * 64 + 32 * j] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        asm volatile("bar.sync %0, 64;" ::"r"(2 + kg) : "memory");  // the two halves of key group kg
        // ------------------------------------------------ softmax of tile i + 1
        // keys 32 kg + 16 dq + 8 h + {k0, k1}; rows g, g + 8
        float x[2][4], p4[2][4], inv_ts[2][2];
        bool over = false;  // a score passes its row's reference by more than the threshold
        uint8_t* const Pb = smem + kOffP + ((i + 1) & 1) * kPBytes;
        auto probabilities = [&]() {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float m = m_ref[r] == -INFINITY ? 0.f : m_ref[r];  // a row that sees no key yet
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              p4[h][2 * r] = fast_exp2(x[h][2 * r] - m);
              p4[h][2 * r + 1] = fast_exp2(x[h][2 * r + 1] - m);
              *reinterpret_cast<__half2*>(Pb + (8 * r + g) * 256 + (((4 * kg + 2 * dq + h) ^ g) << 4) + 4 * q) =
                  __floats2half2_rn(p4[h][2 * r], p4[h][2 * r + 1]);
            }
          }
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 y = X[(warp ^ 1) * 64 + 32 * h];
          const float f[4] = {acc[2 + h][0] + y.x, acc[2 + h][1] + y.y, acc[2 + h][2] + y.z, acc[2 + h][3] + y.w};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t u = q_ts[16 * dq + 8 * h + (c ? k1 : k0)];
            const float a = __uint_as_float(u) * p.scale_log2, e = (float)((int)(u >> 23) - 127);
            inv_ts[h][c] = __uint_as_float(0x7F000000u - u);
            x[h][c] = fmaf(f[c], a, e);
            x[h][2 + c] = fmaf(f[2 + c], a, e);
          }
        }
        if (key0 + kTileKeys > nvis_lo) {  // some key of the tile is hidden from some row
          // A NaN scale of such a key counts as 0 among the values: the rows that see
          // the key have the NaN in their scores, and for the others 0 times NaN
          // would not be 0.  (Each warp has read the scales that it rewrites: its
          // keys, its half of the columns.)  Clearing NaNs where the values are read
          // costs every tile its instructions: 387 -> 391 us on 128 x 16,385 keys.
          const int row = (32 * kg & 63) + lane;
          if (key0 + 32 * kg + lane >= nvis_lo) {
            uint4* const sp = reinterpret_cast<uint4*>(smem + kOffScl + (qk_stage * kTilePages + (kg >> 1)) * kSclBytes +
                                                       row * 32 + ((dq ^ ((row >> 2) & 1)) << 4));
            uint4 v = *sp;
            v.x = drop_nan_e4m3(v.x);
            v.y = drop_nan_e4m3(v.y);
            v.z = drop_nan_e4m3(v.z);
            v.w = drop_nan_e4m3(v.w);
            *sp = v;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later load overwrites them
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int row = min(g + 8 * (c >> 1), P.rows - 1);  // t * n_heads + h
            const int nvis = min(s.len - p.n_q + row / p.d.n_heads + 1, s.end);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (key0 + 32 * kg + 16 * dq + 8 * h + ((c & 1) ? k1 : k0) >= nvis) x[h][c] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c) over |= x[h][c] > m_ref[c >> 1] + kRescaleThreshold;
        probabilities();
        if (++qk_stage == kStages) {
          qk_stage = 0;
          qk_phase ^= 1;
        }
        // P of tile i + 1 is published
        if (sync_warps_or(over || !ok)) {
          ok = !sync_warps_or(!ok);
          if (!ok) break;
          // rare: the rows' maxima over the tile move the references
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (q == 0) atomicMax(&s_max[8 * r + g], float_order(mx));
          }
          sync_warps();
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float t_max = order_float(s_max[8 * r + g]);
            if (t_max > m_ref[r] + kRescaleThreshold) {
              const float alpha = fast_exp2(m_ref[r] - t_max);
              m_ref[r] = t_max;
              l_sum[r] *= alpha;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                o[j][2 * r] *= alpha;
                o[j][2 * r + 1] *= alpha;
              }
            }
          }
          probabilities();
          sync_warps();
          if (tid < kMaxRows) s_max[tid] = float_order(-INFINITY);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            l_sum[r] = fmaf(p4[h][2 * r], inv_ts[h][0], fmaf(p4[h][2 * r + 1], inv_ts[h][1], l_sum[r]));
      }
      if (!ok) break;
      // ------------------------------------------------------------- epilogue
      // l over the warps' keys; columns of this thread: 64 ds + 16 q .. + 15
      // (n-tile j, column n: 8 n + j)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = l_sum[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (q == 0) s_l[warp * kMaxRows + 8 * r + g] = l;
      }
      sync_warps();
      {
        float l[2] = {0.f, 0.f};
#pragma unroll
        for (int wv = 0; wv < kWarps; ++wv) {
          l[0] += s_l[wv * kMaxRows + g];
          l[1] += s_l[wv * kMaxRows + 8 + g];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = g + 8 * r, t = row / p.d.n_heads;
          if (row >= P.rows) continue;
          const size_t part = ((size_t)t * p.n_slots + (w + s.b)) * p.d.n_heads + (row - t * p.d.n_heads);
          const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
          // (few rows: fp32 partials cost nothing that shows)
          float4* dst = reinterpret_cast<float4*>(p.o_part + part * kDC + 64 * ds + 16 * q);
#pragma unroll
          for (int c = 0; c < 2; ++c)  // columns 16 q + 8 c + j
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              dst[2 * c + j / 4] = make_float4(o[j][2 * r + c] * inv, o[j + 1][2 * r + c] * inv, o[j + 2][2 * r + c] * inv,
                                               o[j + 3][2 * r + c] * inv);
          if (ds == 0 && q == 0) p.lse_part[part] = l[r] == 0.f ? -INFINITY : m_ref[r] + __log2f(l[r]);
        }
      }
      sync_warps();  // s_l is rewritten by the next piece
    }
  }
  if (!ok) {
    // a wait gave up: report it, and let copies in flight land before the shared memory goes
    if (tid == 0) record_status(p.status, MLA_ERR_TIMEOUT);
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < kCopyGraceNs) {
    }
  }
  tl_end(p.timeline, MLA_TRACE_ATTEND);
}

}  // namespace

bool decode_few_supported(const mla_dims& d, int n_q) {
  return d.cache_dtype == MLA_FP4_E2M1 && d.act_dtype == MLA_BF16 && d.d_c == kDC && d.d_rope == kDR &&
         d.page_size == kPage && d.d_v == 128 && n_q >= 1 && (long long)n_q * d.n_heads <= kMaxRows;
}

int decode_few_auto_splits(int num_sms) { return num_sms; }

cudaError_t launch_decode_few(const DecodeParams& p, cudaStream_t st) {
  FewParams fp;
  memset(&fp, 0, sizeof(fp));
  fp.p = p;
  fp.rows = p.n_q * p.d.n_heads;
  const Fp4Page f4 = fp4_page(kPage, kDC, kDR);
  fp.ts_off = f4.ts_off;
  if (!make_page_map_swizzled(&fp.map_codes, p.pool, false, kDC / 2, kPage, p.num_pages, p.page_bytes, 128) ||
      !make_page_map_swizzled(&fp.map_kr, p.pool + f4.kr_off, true, kDR, kPage, p.num_pages, p.page_bytes, kDR) ||
      !make_page_map_swizzled(&fp.map_scl, p.pool + f4.sc_off, false, kDC / 16, kPage, p.num_pages, p.page_bytes,
                              kDC / 16))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(decode_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(decode_few_kernel, dim3(p.splits), dim3(kThreads), kSmemBytes, st, fp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mla
