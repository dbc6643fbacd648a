// S3 over the 4-bit latent cache for few query rows: split-KV attention of the
// absorbed queries of any number of heads (a tensor-parallel shard's 8 to 64,
// times the step's query tokens) on the warp-level tensor cores.
//
// What it computes is decode_tc.cu's (scores of [q~ | q^R] against the rows
// [c | k^R], online softmax, probability-weighted sum of the latent rows; W^UV
// afterwards in the combine kernel).  With c = code * s * ts (ts the token's
// power of two, 2^e) the rows enter in units of ts:
//   S = scale (q~ . c + q^R . k^R) = scale ts (q~ . (code s) + (q^R . k^R) / ts)
//   O = sum_k 2^(S_k + e_k - r) (code s)_k,   l = sum_k 2^(S_k - r),
// S in log2 units, r the row's reference (a running maximum of S + e): code * s
// is exact in f16 whatever the latent's magnitude, and the probabilities carry
// the tokens' scales.
//
// Why warp-level MMA and not tcgen05: 16 rows against 420 bytes a key are bound
// by HBM (16 rows: 35 kFLOP a key), and a tcgen05 operand has to lie in shared
// memory as 16-bit values: written once and read twice, 3.3 KB a key, 26 cycles
// of an SM's shared-memory bandwidth against the 19 cycles the key's bytes take
// from HBM.  Here the codes are read from shared memory as they are (twice 256
// bytes) and become MMA fragments in registers.
//
// One CTA (16 warps) runs one split of the keys for a group of 16 MT rows, in
// tiles of 128 keys (two pages):
//   scores  warp (kg, dq): 32 keys x a quarter of the columns; the contraction
//           order is the codes' own (a thread's 32 consecutive codes of a key
//           are the B fragments of eight k-steps), the query fragments are
//           stored in that order; the quarters' sums meet in shared memory
//   softmax warp (kg, dq) finishes 8 keys x all rows; the reference moves only
//           when a tile's maximum passes it by 2^8; P goes out as f16
//   values  warp (ds, kh): 64 columns x half of the keys; a thread takes eight
//           consecutive codes of four keys, whose halves, paired over keys by
//           byte permutes, are the B fragments of eight n-tiles
// Keys of a group of eight are taken in the order n ^ (4 if n is odd), with
// which both the 16-byte and the 4-byte reads of the 128-byte-swizzled pages
// (TMA) spread over all banks.
#include <cuda.h>

#include <cstring>

#include "mla_internal.cuh"
#include "mma_tile.cuh"

namespace mla {

namespace {

constexpr int kDC = 512, kDR = 64, kD = kDC + kDR, kPage = 64;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kTilePages = 2, kTileKeys = kTilePages * kPage;
constexpr uint32_t kCodeBytes = kPage * kDC / 2;             // codes of a page: two 8 KB boxes of 256 columns
constexpr uint32_t kKrBytes = kPage * kDR * 2;
constexpr uint32_t kSclBytes = kPage * kDC / 16 + kPage * 4;  // block scales, then token scales
constexpr uint32_t kStageBytes = kTilePages * (kCodeBytes + kKrBytes);
constexpr int kSteps = 9;                                    // k-steps of a quarter: 8 of codes, 1 of k^R
constexpr float kRescaleThreshold = 8.0f;                    // log2 units
constexpr unsigned long long kCopyGraceNs = 200000ull;

template <int MT>
struct Layout {
  static constexpr int Rows = 16 * MT;
  static constexpr int Stages = MT == 1 ? 3 : 2;
  static constexpr uint32_t OffStage = 0;
  static constexpr uint32_t OffScl = OffStage + Stages * kStageBytes;        // [Stages][kTilePages][kSclBytes]
  static constexpr uint32_t OffQ = OffScl + Stages * kTilePages * kSclBytes;  // [MT][4 dq][kSteps][32 lanes] fragments
  static constexpr uint32_t OffX = OffQ + MT * 4 * kSteps * 512;             // [MT][kWarps][4][32 lanes] float4
  static constexpr uint32_t OffP = OffX + MT * kWarps * 4 * 512;             // [Rows][128 keys] f16, 16-byte units swizzled
  static constexpr uint32_t OffMax = OffP + Rows * kTileKeys * 2;            // int [Rows]
  static constexpr uint32_t OffL = OffMax + Rows * 4;                    // float [kWarps][Rows]
  static constexpr uint32_t OffBar = OffL + kWarps * Rows * 4;
  static constexpr uint32_t Bytes = OffBar + Stages * 8 + 1024;              // + alignment slack
};
static_assert(Layout<1>::Bytes <= 232448 && Layout<2>::Bytes <= 232448, "shared memory");

struct FewParams {
  DecodeParams p;
  int rows, groups;       // query rows of a sequence (n_q * n_heads), groups of 16 MT of them
  size_t scl_off;         // scales' offset in a page
  CUtensorMap map_codes;  // [pages][64 rows][256 bytes], box 128 bytes x 64 rows, 128-byte swizzle
  CUtensorMap map_kr;     // [pages][64 rows][64] bf16, box 64 x 64 rows, 128-byte swizzle
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
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Order-preserving map of floats to signed integers (for atomicMax).
__device__ __forceinline__ int float_order(float x) {
  const int i = __float_as_int(x);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// Key of column n of a group of eight.
__device__ __forceinline__ int key_of(int n) { return n ^ ((n & 1) << 2); }

// The pieces of the sequences in split w, for query tokens up to t_hi.
struct Piece {
  int b, page_lo, n_pages;  // n_pages: pages with a key visible to token t_hi
  int len, end;             // keys of the sequence; first key behind the piece's pages
};
struct PieceWalker {
  const DecodeParams* p;
  int t_hi, b;
  long long g, g1;
  __device__ PieceWalker(const DecodeParams& p_, int w, int t_hi_) : p(&p_), t_hi(t_hi_) {
    const long long TT = p->plan[p->batch];
    g = split_tile_begin(w, TT, p->splits);
    g1 = split_tile_begin(w + 1, TT, p->splits);
    b = g < g1 ? seq_of_tile(p->plan, p->batch, g) : 0;
  }
  __device__ bool next(Piece& s) {
    if (g >= g1) return false;
    while ((long long)p->plan[b + 1] <= g) ++b;
    const long long end = min(g1, (long long)p->plan[b + 1]);
    s.b = b;
    s.len = p->seq_lens[b];
    s.page_lo = (int)(g - p->plan[b]);
    s.end = (int)(end - p->plan[b]) * kPage;
    const int vis_pages = (s.len - p->n_q + t_hi + 1 + kPage - 1) / kPage;
    s.n_pages = max(0, min((int)(end - p->plan[b]), vis_pages) - s.page_lo);
    g = end;
    return true;
  }
};

// MT: 16-row tiles of query rows per CTA.
template <int MT>
__global__ void __launch_bounds__(kThreads, 1) decode_few_kernel(const __grid_constant__ FewParams P) {
  using L = Layout<MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const DecodeParams& p = P.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int grp = blockIdx.x % P.groups, w = blockIdx.x / P.groups;
  const int row0 = grp * L::Rows;  // first row (t * n_heads + h) of this CTA
  const int t_hi = min(P.rows - 1, row0 + L::Rows - 1) / p.d.n_heads, t_lo = row0 / p.d.n_heads;
  int* s_max = reinterpret_cast<int*>(smem + L::OffMax);
  float* s_l = reinterpret_cast<float*>(smem + L::OffL);
  auto bar = [&](int s) -> uint32_t { return sbase + L::OffBar + 8u * s; };

  pdl_trigger();
  if (tid == 0)
    for (int s = 0; s < L::Stages; ++s) mbar_init_local(bar(s), 1);
  if (tid < L::Rows) s_max[tid] = float_order(-INFINITY);
  __syncthreads();
  pdl_wait();
  tl_begin(p.timeline, MLA_TRACE_ATTEND);

  // loads: lane i of warp 0 brings page i of a tile; the walker runs ahead of the tiles
  PieceWalker lwalk(p, w, t_hi);
  Piece lp;
  int l_at = 0, l_stage = 0, l_page = 0;
  lp.n_pages = 0;
  const bool stall = (p.d.flags & MLA_FLAG_SELFTEST_STALL) != 0;
  // the next tile's page of this lane (looked up one load ahead)
  auto look_up = [&]() {
    while (l_at >= lp.n_pages) {
      lp.n_pages = 0;
      l_at = 0;
      if (!lwalk.next(lp)) return;
    }
    if (lane < min(kTilePages, lp.n_pages - l_at))
      l_page = p.page_table[(size_t)lp.b * p.max_pages + lp.page_lo + l_at + lane];
  };
  auto load_next = [&]() {  // warp 0
    if (lp.n_pages == 0) return;  // no tile left
    const int npg = min(kTilePages, lp.n_pages - l_at);
    if (!stall) {
      if (lane == 0) mbar_expect_local(bar(l_stage), npg * (kCodeBytes + kKrBytes + kSclBytes));
      __syncwarp();
      if (lane < npg) {
        int page = l_page;
        if (page < 0 || page >= p.num_pages) {
          record_status(p.status, MLA_ERR_BOUNDS);
          page = 0;
        }
        const uint32_t st = sbase + L::OffStage + l_stage * kStageBytes, fb = bar(l_stage);
        for (int h = 0; h < 2; ++h)
          tma_load_3d(st + lane * kCodeBytes + h * (kCodeBytes / 2), &P.map_codes, 128 * h, 0, page, fb);
        tma_load_3d(st + kTilePages * kCodeBytes + lane * kKrBytes, &P.map_kr, 0, 0, page, fb);
        bulk_load(sbase + L::OffScl + (l_stage * kTilePages + lane) * kSclBytes,
                  p.pool + (size_t)page * p.page_bytes + P.scl_off, kSclBytes, fb);
      }
      __syncwarp();
    }
    l_at += npg;
    if (++l_stage == L::Stages) l_stage = 0;
    look_up();
  };
  if (warp == 0) look_up();
  if (warp == 0)
    for (int s = 0; s < L::Stages; ++s) load_next();

  const int kg = warp >> 2, dq = warp & 3;  // scores, softmax
  const int ds = warp & 7, kh = warp >> 3;  // values
  // This thread's places in a staged tile; the loops add multiples of eight
  // rows, which leave the swizzle as it is.
  const int qk_key = (32 * kg & 63) + key_of(g);  // scores: row of page kg / 2, + 8 nt
  const uint32_t qk_codes = (uint32_t)((kg >> 1) * kCodeBytes + (dq >> 1) * (kCodeBytes / 2) + qk_key * 128 +
                                       ((((dq & 1) * 4 + q) ^ (qk_key & 7)) << 4));
  const uint32_t qk_kr = (uint32_t)(kTilePages * kCodeBytes + (kg >> 1) * kKrBytes + qk_key * 128 +
                                    (((2 * q + (dq >> 1)) ^ (qk_key & 7)) << 4) + (dq & 1) * 8);
  const uint32_t qk_scl = (uint32_t)((kg >> 1) * kSclBytes + qk_key * 32 + 8 * dq + 2 * q);
  const uint32_t qk_ts = (uint32_t)((kg >> 1) * kSclBytes + kPage * kDC / 16 + (32 * kg & 63) * 4);
  const int k0 = 2 * q, k1 = key_of(2 * q + 1);   // keys of an accumulator's columns, of a value fragment's halves
  const uint32_t pv_col = (ds & 3) * 2 + (g >> 2);
  const uint32_t pv_box = (uint32_t)(kh * kCodeBytes + (ds >> 2) * (kCodeBytes / 2) + (g & 3) * 4);
  const uint32_t pv_codes0 = pv_box + k0 * 128 + ((pv_col ^ k0) << 4), pv_codes1 = pv_box + k1 * 128 + ((pv_col ^ k1) << 4);
  const uint32_t pv_scl = (uint32_t)(kh * kSclBytes + 4 * ds + (g >> 1));
  int qk_stage = 0, pv_stage = 0;
  uint32_t qk_phase = 0;
  bool ok = true;
  PieceWalker walk(p, w, t_hi);
  Piece s;
  while (ok && walk.next(s)) {
    const size_t slot0 = (size_t)(w + s.b);
    auto part_row = [&](int r) -> size_t {  // row r (t * n_heads + h) among the split partials
      return ((size_t)(r / p.d.n_heads) * p.n_slots + slot0) * p.d.n_heads + r % p.d.n_heads;
    };
    __nv_bfloat16* o_part = reinterpret_cast<__nv_bfloat16*>(p.o_part);
    if (s.n_pages == 0) {
      for (int i = tid; i < L::Rows * (kDC / 8); i += kThreads) {
        const int r = row0 + i / (kDC / 8);
        if (r < P.rows) *reinterpret_cast<uint4*>(o_part + part_row(r) * kDC + 8 * (i % (kDC / 8))) = make_uint4(0, 0, 0, 0);
      }
      if (tid < L::Rows && row0 + tid < P.rows) p.lse_part[part_row(row0 + tid)] = -INFINITY;
      continue;
    }
    // Query fragments.  Quarter dq, step st < 8: contraction index 2q, 2q + 1 /
    // 2q + 8, 2q + 9 are columns 128 dq + 32 q + 4 st + {0, 1} / {2, 3}; step 8:
    // k^R columns 16 q + 4 dq + {0, 1} / {2, 3}.
    for (int i = tid; i < MT * 4 * kSteps * 32; i += kThreads) {
      const int ln = i & 31, st = (i >> 5) % kSteps, d4 = (i >> 5) / kSteps % 4, mt = (i >> 5) / (4 * kSteps);
      const int col = st < 8 ? 128 * d4 + 32 * (ln & 3) + 4 * st : kDC + 16 * (ln & 3) + 4 * d4;
      const int r = row0 + 16 * mt + (ln >> 2);
      const __half* src = static_cast<const __half*>(p.q_abs) + ((size_t)s.b * P.rows + r) * kD + col;
      const uint2 lo = r < P.rows ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
      const uint2 hi = r + 8 < P.rows ? *reinterpret_cast<const uint2*>(src + 8 * kD) : make_uint2(0, 0);
      *reinterpret_cast<uint4*>(smem + L::OffQ + (size_t)i * 16) = make_uint4(lo.x, hi.x, lo.y, hi.y);
    }
    __syncthreads();
    float o[MT][8][4], m_ref[MT][2], l_sum[MT][2];
    int nvis[MT][2];  // keys before the piece's end that this thread's rows see
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m_ref[mt][r] = -INFINITY;
        l_sum[mt][r] = 0.f;
        nvis[mt][r] = min(s.len - p.n_q + min(row0 + 16 * mt + 8 * r + g, P.rows - 1) / p.d.n_heads + 1, s.end);
      }
    }
    const int nvis_lo = min(s.len - p.n_q + t_lo + 1, s.end), nvis_hi = min(s.len - p.n_q + t_hi + 1, s.end);
    const int n_tiles = (s.n_pages + kTilePages - 1) / kTilePages;
    // Pipeline: the scores of tile i + 1 and the values of tile i share a phase
    // (either's latencies lie under the other's work), the softmax of i + 1 follows.
    for (int i = -1; i < n_tiles; ++i) {
      const bool more = i + 1 < n_tiles;
      const int key0 = (s.page_lo + (i + 1) * kTilePages) * kPage;  // tile i + 1
      const bool tail = key0 + kTileKeys > nvis_lo;  // some key of it is hidden from some row
      float4* X = reinterpret_cast<float4*>(smem + L::OffX);
      // ------------------------------------------------ scores of tile i + 1
      if (more) {
        const uint8_t* st = smem + L::OffStage + qk_stage * kStageBytes;
        uint8_t* scl = smem + L::OffScl + qk_stage * kTilePages * kSclBytes;
        ok = mbar_wait_bounded(bar(qk_stage), qk_phase) && ok;
        if (tail) {
          // keys that no row sees count as zero, whatever the page holds there
          const int n_keys = nvis_hi - key0;
          for (int k = tid >> 2; k < kTileKeys; k += kThreads / 4)
            if (k >= n_keys) {
              uint8_t* ps = scl + (k >> 6) * kSclBytes;
              *reinterpret_cast<uint2*>(ps + (k & 63) * 32 + 8 * (tid & 3)) = make_uint2(0, 0);
              if ((tid & 3) == 0) *reinterpret_cast<float*>(ps + kPage * kDC / 16 + (k & 63) * 4) = 1.0f;
            }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a later load overwrites them
          __syncthreads();
        }
        float acc[MT][4][4];
        uint4 v[4];
        __half2 sc[4][2];
        const uint4* qf = reinterpret_cast<const uint4*>(smem + L::OffQ) + dq * kSteps * 32 + lane;
        uint4 qr[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) qr[mt] = qf[(mt * 4 * kSteps + 8) * 32];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const uint2 kr = *reinterpret_cast<const uint2*>(st + qk_kr + nt * 1024);
          v[nt] = *reinterpret_cast<const uint4*>(st + qk_codes + nt * 1024);
          const __half2 s2 = __half2(__nv_cvt_fp8x2_to_halfraw2(
              *reinterpret_cast<const uint16_t*>(scl + qk_scl + nt * 256), __NV_E4M3));
          sc[nt][0] = __low2half2(s2);
          sc[nt][1] = __high2half2(s2);
          // (q^R . k^R) / ts of the accumulator's two keys
          const uint32_t* ts = reinterpret_cast<const uint32_t*>(scl + qk_ts) + 8 * nt;
          const float i0 = __uint_as_float(0x7F000000u - ts[k0]), i1 = __uint_as_float(0x7F000000u - ts[k1]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
            mma_bf16(acc[mt][nt], *reinterpret_cast<const uint32_t(*)[4]>(&qr[mt]), kr.x, kr.y);
            acc[mt][nt][0] *= i0;
            acc[mt][nt][1] *= i1;
            acc[mt][nt][2] *= i0;
            acc[mt][nt][3] *= i1;
          }
        }
#pragma unroll
        for (int wi = 0; wi < 4; ++wi) {  // eight codes of each key: two k-steps
          uint4 qa[MT][2];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            qa[mt][0] = qf[(mt * 4 * kSteps + 2 * wi) * 32];
            qa[mt][1] = qf[(mt * 4 * kSteps + 2 * wi + 1) * 32];
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            __half2 h[4];
            e2m1x8_to_half2(wi == 0 ? v[nt].x : wi == 1 ? v[nt].y : wi == 2 ? v[nt].z : v[nt].w, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = __hmul2(h[e], sc[nt][wi >> 1]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(acc[mt][nt], qa[mt][0], as_u32(h[0]), as_u32(h[1]));
              mma_f16(acc[mt][nt], qa[mt][1], as_u32(h[2]), as_u32(h[3]));
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
            X[((mt * kWarps + warp) * 4 + nt) * 32 + lane] =
                make_float4(acc[mt][nt][0], acc[mt][nt][1], acc[mt][nt][2], acc[mt][nt][3]);
      }
      // ---------------------------------------------------- values of tile i
      if (i >= 0) {
        const uint8_t* st = smem + L::OffStage + pv_stage * kStageBytes;
        const uint8_t* scl = smem + L::OffScl + pv_stage * kTilePages * kSclBytes;
        // thread: columns 64 ds + 8 g .. + 7 of keys 16 kb + {k0, k1} and 8 more; the
        // codes of the two keys are interleaved, so that a byte converts into
        // the f16 pair of one column, and the pair of scales multiplies it
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          uint4 pa[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int r = 16 * mt + (lane & 15), u = 8 * kh + 2 * kb + (lane >> 4);
            ldsm_x4(sbase + L::OffP + r * 256 + ((u ^ (r & 7)) << 4), pa[mt].x, pa[mt].y, pa[mt].z, pa[mt].w);
          }
          uint32_t b0[8], b1[8];
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // keys 16 kb + 8 h + {k0, k1}
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(st + pv_codes0 + kb * 2048 + h * 1024);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(st + pv_codes1 + kb * 2048 + h * 1024);
            const uint32_t s0 = scl[pv_scl + k0 * 32 + kb * 512 + h * 256], s1 = scl[pv_scl + k1 * 32 + kb * 512 + h * 256];
            const __half2 s2 = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(s0 | (s1 << 8)), __NV_E4M3));
            __half2 he[4], ho[4];  // columns 0, 2, 4, 6 and 1, 3, 5, 7
            e2m1x8_to_half2((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), he);
            e2m1x8_to_half2(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), ho);
            uint32_t* bb = h ? b1 : b0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              bb[2 * m] = as_u32(__hmul2(he[m], s2));
              bb[2 * m + 1] = as_u32(__hmul2(ho[m], s2));
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][j], pa[mt], b0[j], b1[j]);
        }
      }
      // every warp is done with tile i (its stage and P are free) and has
      // published its scores of tile i + 1
      ok = __syncthreads_and(ok);
      if (!ok) break;
      if (i >= 0) {
        pv_stage = pv_stage + 1 == L::Stages ? 0 : pv_stage + 1;
        if (warp == 0) load_next();
      }
      if (!more) break;
      // ----------------------------------------------- softmax of tile i + 1
      // keys 32 kg + 8 dq + {k0, k1}; rows 16 mt + g, + 8
      float x[MT][4], p4[MT][4], inv_ts[2];
      {
        const int k8 = 32 * kg + 8 * dq;
        const uint32_t* ts =
            reinterpret_cast<const uint32_t*>(smem + L::OffScl + qk_stage * kTilePages * kSclBytes + qk_ts) + 8 * dq;
        const int kk[2] = {k0, k1};
        float a[2], e[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t u = ts[kk[c]];
          a[c] = __uint_as_float(u) * p.scale_log2;
          e[c] = (float)((int)(u >> 23) - 127);
          inv_ts[c] = __uint_as_float(0x7F000000u - u);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float4 f = X[((mt * kWarps + 4 * kg) * 4 + dq) * 32 + lane];
#pragma unroll
          for (int d4 = 1; d4 < 4; ++d4) {
            const float4 y = X[((mt * kWarps + 4 * kg + d4) * 4 + dq) * 32 + lane];
            f.x += y.x;
            f.y += y.y;
            f.z += y.z;
            f.w += y.w;
          }
          x[mt][0] = fmaf(f.x, a[0], e[0]);
          x[mt][1] = fmaf(f.y, a[1], e[1]);
          x[mt][2] = fmaf(f.z, a[0], e[0]);
          x[mt][3] = fmaf(f.w, a[1], e[1]);
          if (tail) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key0 + k8 + kk[c & 1] >= nvis[mt][c >> 1]) x[mt][c] = -INFINITY;
          }
        }
      }
      auto probabilities = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float m = m_ref[mt][r] == -INFINITY ? 0.f : m_ref[mt][r];  // a row that sees no key yet
            p4[mt][2 * r] = fast_exp2(x[mt][2 * r] - m);
            p4[mt][2 * r + 1] = fast_exp2(x[mt][2 * r + 1] - m);
            const int row = 16 * mt + 8 * r + g;
            *reinterpret_cast<__half2*>(smem + L::OffP + row * 256 + (((4 * kg + dq) ^ (row & 7)) << 4) + 4 * q) =
                __floats2half2_rn(p4[mt][2 * r], p4[mt][2 * r + 1]);
          }
      };
      bool over = false;  // a score passes its row's reference by more than the threshold
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int c = 0; c < 4; ++c) over |= x[mt][c] > m_ref[mt][c >> 1] + kRescaleThreshold;
      probabilities();
      if (__syncthreads_or(over)) {
        // rare: the rows' maxima over the tile move the references
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float mx = fmaxf(x[mt][2 * r], x[mt][2 * r + 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            if (q == 0) atomicMax(&s_max[16 * mt + 8 * r + g], float_order(mx));
          }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float t_max = order_float(s_max[16 * mt + 8 * r + g]);
            if (t_max > m_ref[mt][r] + kRescaleThreshold) {
              const float alpha = fast_exp2(m_ref[mt][r] - t_max);
              m_ref[mt][r] = t_max;
              l_sum[mt][r] *= alpha;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                o[mt][j][2 * r] *= alpha;
                o[mt][j][2 * r + 1] *= alpha;
              }
            }
          }
        probabilities();
        __syncthreads();
        if (tid < L::Rows) s_max[tid] = float_order(-INFINITY);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          l_sum[mt][r] = fmaf(p4[mt][2 * r], inv_ts[0], fmaf(p4[mt][2 * r + 1], inv_ts[1], l_sum[mt][r]));
      if (++qk_stage == L::Stages) {
        qk_stage = 0;
        qk_phase ^= 1;
      }
    }
    if (!ok) break;
    // ------------------------------------------------------------- epilogue
    // l over the warps' keys, O over the two key halves; columns of this
    // thread: 64 ds + 16 q .. + 15 (n-tile j, column n: 8 n + j)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = l_sum[mt][r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (q == 0) s_l[warp * L::Rows + 16 * mt + 8 * r + g] = l;
      }
    float4* X = reinterpret_cast<float4*>(smem + L::OffX);  // (its scores were read before the last barrier)
    if (kh == 1)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          X[((mt * 8 + ds) * 8 + j) * 32 + lane] = make_float4(o[mt][j][0], o[mt][j][1], o[mt][j][2], o[mt][j][3]);
    __syncthreads();
    if (kh == 0) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float l[2] = {0.f, 0.f};
#pragma unroll
        for (int wv = 0; wv < kWarps; ++wv) {
          l[0] += s_l[wv * L::Rows + 16 * mt + g];
          l[1] += s_l[wv * L::Rows + 16 * mt + 8 + g];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 y = X[((mt * 8 + ds) * 8 + j) * 32 + lane];
          o[mt][j][0] += y.x;
          o[mt][j][1] += y.y;
          o[mt][j][2] += y.z;
          o[mt][j][3] += y.w;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = row0 + 16 * mt + 8 * r + g;
          if (row >= P.rows) continue;
          const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
          uint32_t u[8];
#pragma unroll
          for (int c = 0; c < 2; ++c)  // columns 16 q + 8 c + j
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const __nv_bfloat162 v2 = __floats2bfloat162_rn(o[mt][j][2 * r + c] * inv, o[mt][j + 1][2 * r + c] * inv);
              u[4 * c + j / 2] = *reinterpret_cast<const uint32_t*>(&v2);
            }
          uint4* dst = reinterpret_cast<uint4*>(o_part + part_row(row) * kDC + 64 * ds + 16 * q);
          dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
          dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
          if (ds == 0 && q == 0) p.lse_part[part_row(row)] = l[r] > 0.f ? m_ref[mt][r] + __log2f(l[r]) : -INFINITY;
        }
      }
    }
    __syncthreads();
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

template <int MT>
cudaError_t launch_few(FewParams& fp, cudaStream_t st) {
  fp.groups = (fp.rows + 16 * MT - 1) / (16 * MT);
  auto kernel = decode_few_kernel<MT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<MT>::Bytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(fp.p.splits * fp.groups), dim3(kThreads), Layout<MT>::Bytes, st, fp);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// 16-row tiles per CTA: two from 17 rows on, so that a page's codes are
// converted once for 32 rows.
int few_tiles(int rows) { return rows > 16 ? 2 : 1; }

}  // namespace

bool decode_few_supported(const mla_dims& d, int n_q) {
  return d.cache_dtype == MLA_FP4_E2M1 && d.act_dtype == MLA_BF16 && d.d_c == kDC && d.d_rope == kDR &&
         d.page_size == kPage && d.d_v == 128 && n_q >= 1 && (long long)n_q * d.n_heads <= 65536;
}

int decode_few_auto_splits(const mla_dims& d, int num_sms, int n_q) {
  const int rows = n_q * d.n_heads, per = 16 * few_tiles(rows), groups = (rows + per - 1) / per;
  const int w = num_sms / groups;
  return w > 0 ? w : 1;
}

cudaError_t launch_decode_few(const DecodeParams& p, cudaStream_t st) {
  FewParams fp;
  memset(&fp, 0, sizeof(fp));
  fp.p = p;
  fp.rows = p.n_q * p.d.n_heads;
  const Fp4Page f4 = fp4_page(kPage, kDC, kDR);
  fp.scl_off = f4.sc_off;
  if (!make_page_map_swizzled(&fp.map_codes, p.pool, false, kDC / 2, kPage, p.num_pages, p.page_bytes, 128) ||
      !make_page_map_swizzled(&fp.map_kr, p.pool + f4.kr_off, true, kDR, kPage, p.num_pages, p.page_bytes, kDR))
    return cudaErrorInvalidValue;
  return few_tiles(fp.rows) == 2 ? launch_few<2>(fp, st) : launch_few<1>(fp, st);
}

}  // namespace mla
