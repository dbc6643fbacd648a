// Rows of the paged latent cache, written from and read back as values:
//   mla_append_rows  [c | k^R] rows that the caller has already projected (a
//                    fused down-projection's output) go into the cache:
//                    optional RMSNorm of c, RoPE of k^R at the token's
//                    position, rounding to the cache type, paged store, in one
//                    pass over the rows
//   mla_read_rows    cache rows back as c and k^R values
// and the quantiser that ends mla_append_latent on a 4-bit cache.  They have
// no counterpart of their own in the articles: their append projects inside
// ("1. Low-Rank Key-Value Compression", "3. Decoupled RoPE and Matrix
// Absorption"), and this is the same store for a projection made elsewhere.
//
// One warp takes a token; a lane holds blocks of 16 consecutive elements of c,
// so a 4-bit block's maximum needs no exchange, an 8-bit tile's (128 elements)
// three shuffles, the norm's sum and the token's maximum five.  Every input
// byte is read once and every output byte written once (V3 dims, bf16 in, 4-bit
// out: 1,152 + 420 bytes a token).  Measured on 32,792 tokens, where HBM would
// allow 7.9 us each way: append with norm 26.6 us (2.0 TB/s), without 20.4, read 10.9
// (4.7 TB/s).  To an 8-bit cache (floor 9.1) 29.4, 22.5 and 11.0 us, to a bf16 one
// (11.5) 19.3, 13.9 and 12.9.  The append is bound by issue (65% of the slots; 600
// instructions a token: 64-bit norm, angles, quotients), so its warps load the next
// row while they work on one (30 -> 26 us); the read by latency, so a warp takes four
// tokens at a time and stores whole sectors (18 -> 11).  Calls of up to some thousand
// tokens take 3 to 7 us on the device, less than their launch costs the host.
#include <math.h>

#include "mla_internal.cuh"

namespace mla {

int* device_status_word();
size_t cache_page_bytes(const mla_dims& d);

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxHalf = 64;  // RoPE frequencies passed by value; wider k^R computes its own

struct RowsArgs {
  const void* c;       // [n][c_stride]
  long long c_stride;  // elements
  const void* kr;      // [n][kr_stride]
  long long kr_stride;
  const void* norm_w;  // [d_c] or null
  double norm_eps, inv_dc;
  int n_tokens;
  const int32_t* seq_idx;
  const int32_t* pos;
  const int32_t* page_table;
  int batch, max_pages;
  uint8_t* pool;
  int num_pages;
  size_t page_bytes;
  int d_c, d_rope, page_size, page_shift;  // page_shift: log2 of page_size, or -1
  float rope_base;
  int* status;
  unsigned long long* timeline;
  double inv_freq[kMaxHalf];
};

// Physical (page, row) of token n, or page -1 (recorded) if out of range.
template <typename A>
__device__ __forceinline__ int row_slot(const A& a, int b, int p, int* row, bool record) {
  const int lp = a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size;
  const bool ok = b >= 0 && b < a.batch && p >= 0 && lp < a.max_pages;
  const int page = ok ? a.page_table[(size_t)b * a.max_pages + lp] : -1;
  *row = p - lp * a.page_size;
  if (page < 0 || page >= a.num_pages) {
    if (record) record_status(a.status, MLA_ERR_BOUNDS);
    return -1;
  }
  return page;
}

// 16 consecutive elements as fp32
template <bool VEC>
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
  if (VEC) {
    load8(p, x);
    load8(p + 8, x + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = p[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
  if (VEC) {
    load8(p, x);
    load8(p + 8, x + 8);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __bfloat162float(p[e]);
  }
}
template <bool VEC>
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
  if (VEC) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = x[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
  if (VEC) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = __float2bfloat16_rn(x[e]);
  }
}

// of values >= 0, whose bit patterns are ordered as they are
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// 16 elements as they lie in memory, for a load ahead of its use
template <typename T>
struct Raw16 {
  uint4 v[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
}
template <typename T>
__device__ __forceinline__ void unpack16(const Raw16<T>& r, float (&x)[16]) {
  load16<true>(reinterpret_cast<const T*>(r.v), x);
}

// RMSNorm of one token's c, held 16 elements per lane and block: y = c w r,
// r = 1 / sqrt(mean(c^2) + eps).  The quantisers cut y into codes whose
// borders bf16 inputs meet exactly, so y is the correctly rounded fp32 value up to
// an error of 2^-48: the sum and r are formed in 64 bits, c w as a product and
// its remainder, r as the sum of two floats.  Where the mean square lies beyond
// 2^+-100, a power of two goes from r to c first, so that neither c w (beyond fp32's
// range) nor the remainders (subnormal) lose anything.
template <typename T, int NB, bool VEC, bool AHEAD>
__device__ __forceinline__ void rms_norm(const RowsArgs& a, int lane, int nb, const Raw16<T>& w0, float (&x)[NB][16]) {
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const double v = (double)x[j][e];
      ss = fma(v, v, ss);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double ms = fma(ss, a.inv_dc, a.norm_eps);  // the same in every lane
  double r = rsqrt(ms);
  if (ms > 0x1p100 || ms < 0x1p-100) {
    const float f = ms > 1.0 ? 0x1p-50f : 0x1p50f;
    r *= ms > 1.0 ? 0x1p50 : 0x1p-50;
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[j][e] *= f;
  }
  const float r_hi = (float)r, r_lo = (float)(r - (double)r_hi);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int b = lane + 32 * j;
    if (b < nb) {
      float w[16];
      if (AHEAD) unpack16(w0, w);
      else load16<VEC>(static_cast<const T*>(a.norm_w) + 16 * b, w);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float p = x[j][e] * w[e];
        const float p_lo = std::is_same<T, float>::value ? fmaf(x[j][e], w[e], -p) : 0.f;  // bf16 products are exact
        x[j][e] = fmaf(p, r_hi, fmaf(p, r_lo, p_lo * r_hi));
      }
    }
  }
}

// Codes, block scales and token scale of one row of a 4-bit cache.
template <int NB>
__device__ __forceinline__ void store_fp4(uint8_t* pg, const Fp4Page& f4, int prow, int d_c, int lane, int nb,
                                          const float (&x)[NB][16], float kr_max) {
  float amax[NB], c_max = 0.f;
  bool finite[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    float m = 0.f, z = 0.f;  // z: 0 unless an element is not finite
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      m = fmaxf(m, fabsf(x[j][e]));
      z = fmaf(x[j][e], 0.f, z);
    }
    finite[j] = z == 0.f;
    if (!finite[j]) {
      m = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, finite_abs(x[j][e], finite[j]));
    }
    amax[j] = m;
    c_max = fmaxf(c_max, m);
  }
  const float ts = fp4_token_scale(warp_max(c_max), kr_max);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int b = lane + 32 * j;
    if (b < nb) {
      const uint32_t sc = fp4_block_scale(amax[j], ts, finite[j]);
      const float step = e4m3_to_float((uint8_t)sc) * ts;
      const float inv = fp4_inverse(step);
      uint32_t w[2] = {0u, 0u};
      if (inv > 0.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= fp4_pair(x[j][2 * e], x[j][2 * e + 1], step, inv) << (8 * (e & 3));
      }
      *reinterpret_cast<uint2*>(pg + (size_t)prow * (d_c / 2) + 8 * b) = make_uint2(w[0], w[1]);
      pg[f4.sc_off + (size_t)prow * (d_c / 16) + b] = (uint8_t)sc;
    }
  }
  if (lane == 0) reinterpret_cast<float*>(pg + f4.ts_off)[prow] = ts;
}

// T: type of the rows; CACHE: cache type; NB: blocks per lane (d_c <= 512 NB);
// VEC: rows, weights and unquantised cache rows allow 16-byte accesses.
template <typename T, int CACHE, int NB, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) append_rows_kernel(const __grid_constant__ RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  tl_begin(a.timeline, MLA_TRACE_APPEND_FINALIZE);
  using CT = typename std::conditional<CACHE == MLA_F32, float, __nv_bfloat16>::type;  // k^R (and plain c) in the cache
  const int lane = threadIdx.x & 31, nb = a.d_c / 16, half = a.d_rope >> 1;
  const double inv0 = lane < half ? (half <= kMaxHalf ? a.inv_freq[lane & (kMaxHalf - 1)]
                                                      : rope_inv_freq(lane, half, a.rope_base))
                                  : 0.0;
  // bf16 rows of at most 512 elements: the weights stay in registers, and the
  // next token's row is loaded while this one is computed
  constexpr bool kAhead = VEC && NB == 1 && sizeof(T) == 2;
  const int stride = gridDim.x * kWarps, last = a.n_tokens - 1;
  int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (n > last) return tl_end(a.timeline, MLA_TRACE_APPEND_FINALIZE);
  Raw16<T> raw = {}, w0 = {};
  T k1 = from_f<T>(0.f), k2 = k1;
  auto fetch = [&](int m) {
    if (kAhead && lane < nb) load_raw(static_cast<const T*>(a.c) + (long long)m * a.c_stride + 16 * lane, raw);
    if (lane < half) {
      const T* p = static_cast<const T*>(a.kr) + (long long)m * a.kr_stride;
      k1 = p[lane];
      k2 = p[lane + half];
    }
  };
  if (kAhead && a.norm_w && lane < nb) load_raw(static_cast<const T*>(a.norm_w) + 16 * lane, w0);
  fetch(n);
  int position = a.pos[n], prow;
  int page = row_slot(a, a.seq_idx[n], position, &prow, lane == 0);
  for (; n <= last; n += stride) {
    float x[NB][16];
    if (kAhead) {
      unpack16(raw, x[0]);
    } else {
      const T* src = static_cast<const T*>(a.c) + (long long)n * a.c_stride;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int b = lane + 32 * j;
        if (b < nb) {
          load16<VEC>(src + 16 * b, x[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[j][e] = 0.f;
        }
      }
    }
    const float x1_0 = to_f(k1), x2_0 = to_f(k2);
    // the next token's row, position and sequence; its page after this row
    const int m = min(n + stride, last), m_pos = a.pos[m], m_seq = a.seq_idx[m];
    fetch(m);
    if (page >= 0) {
      uint8_t* pg = a.pool + (size_t)page * a.page_bytes;
      CT* kr = CACHE == MLA_F32 || CACHE == MLA_BF16
                   ? reinterpret_cast<CT*>(pg) + (size_t)prow * (a.d_c + a.d_rope) + a.d_c
                   : reinterpret_cast<CT*>(pg + coded_kr_off(CACHE, a.page_size, a.d_c, a.d_rope)) + (size_t)prow * a.d_rope;
      const T* krs = static_cast<const T*>(a.kr) + (long long)n * a.kr_stride;
      float kr_max = 0.f;
      for (int i = lane; i < half; i += 32) {
        const double inv = i == lane ? inv0
                           : half <= kMaxHalf ? a.inv_freq[i & (kMaxHalf - 1)]
                                              : rope_inv_freq(i, half, a.rope_base);
        float cs, sn;
        rope_cos_sin_at(position, inv, &cs, &sn);
        const float x1 = i == lane ? x1_0 : to_f(krs[i]), x2 = i == lane ? x2_0 : to_f(krs[i + half]);
        const CT y1 = from_f<CT>(x1 * cs - x2 * sn), y2 = from_f<CT>(x2 * cs + x1 * sn);
        kr[i] = y1;
        kr[i + half] = y2;
        bool f = true;
        kr_max = fmaxf(kr_max, fmaxf(finite_abs(to_f(y1), f), finite_abs(to_f(y2), f)));
      }
      if (a.norm_w) rms_norm<T, NB, VEC, kAhead>(a, lane, nb, w0, x);
      if (CACHE == MLA_FP4_E2M1) {
        store_fp4<NB>(pg, fp4_page(a.page_size, a.d_c, a.d_rope), prow, a.d_c, lane, nb, x, warp_max(kr_max));
      } else if (CACHE == MLA_FP8_E4M3) {
        // tiles of 128 columns: eight lanes each, the quantiser of the FP8 append
        const Fp8Page fp = fp8_page(a.page_size, a.d_c, a.d_rope);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int b = lane + 32 * j;
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[j][e]));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const float scale = amax > 0.f ? amax / kE4M3Max : 1.0f;
          if (b < nb) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[q] = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[q] |= (uint32_t)__nv_cvt_float_to_fp8(x[j][4 * q + e] / scale, __NV_SATFINITE, __NV_E4M3) << (8 * e);
            }
            *reinterpret_cast<uint4*>(pg + (size_t)prow * a.d_c + 16 * b) = make_uint4(w[0], w[1], w[2], w[3]);
            if ((b & 7) == 0) reinterpret_cast<float*>(pg + fp.sc_off)[(size_t)prow * (a.d_c / 128) + b / 8] = scale;
          }
        }
      } else {
        CT* dst = reinterpret_cast<CT*>(pg) + (size_t)prow * (a.d_c + a.d_rope);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const int b = lane + 32 * j;
          if (b < nb) store16<VEC>(dst + 16 * b, x[j]);
        }
      }
    }
    position = m_pos;
    page = n + stride <= last ? row_slot(a, m_seq, m_pos, &prow, lane == 0) : -1;
  }
  tl_end(a.timeline, MLA_TRACE_APPEND_FINALIZE);
}

// The end of mla_append_latent on a 4-bit cache: c rows from the fp32 scratch,
// k^R from the page, where the projection stored it.
template <int NB>
__global__ void __launch_bounds__(kThreads) append_fp4_finalize_kernel(const __grid_constant__ RowsArgs a) {
  pdl_trigger();
  pdl_wait();
  tl_begin(a.timeline, MLA_TRACE_APPEND_FINALIZE);
  const int lane = threadIdx.x & 31, nb = a.d_c / 16;
  const int n = blockIdx.x * kWarps + (threadIdx.x >> 5);
  int prow;
  const int page = n < a.n_tokens ? row_slot(a, a.seq_idx[n], a.pos[n], &prow, lane == 0) : -1;
  if (page >= 0) {
    const Fp4Page f4 = fp4_page(a.page_size, a.d_c, a.d_rope);
    uint8_t* pg = a.pool + (size_t)page * a.page_bytes;
    const __nv_bfloat16* kr = reinterpret_cast<const __nv_bfloat16*>(pg + f4.kr_off) + (size_t)prow * a.d_rope;
    float kr_max = 0.f, x[NB][16];
    bool f = true;
    for (int i = lane; i < a.d_rope; i += 32) kr_max = fmaxf(kr_max, finite_abs(__bfloat162float(kr[i]), f));
    const float* src = static_cast<const float*>(a.c) + (long long)n * a.c_stride;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int b = lane + 32 * j;
      if (b < nb) {
        load16<true>(src + 16 * b, x[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[j][e] = 0.f;
      }
    }
    store_fp4<NB>(pg, f4, prow, a.d_c, lane, nb, x, warp_max(kr_max));
  }
  tl_end(a.timeline, MLA_TRACE_APPEND_FINALIZE);
}

struct ReadArgs {
  const uint8_t* pool;
  int num_pages;
  size_t page_bytes;
  const int32_t* page_table;
  int batch, max_pages;
  const int32_t* seq_idx;
  const int32_t* pos;
  int n_tokens, d_c, d_rope, page_size, page_shift;
  void* c_out;   // [n][d_c]
  void* kr_out;  // [n][d_rope]
  int* status;
};

__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(v);
}

// Eight elements of a cache row: their bytes, then their values.  A lane takes
// eight, not a block of 16, so that a warp's 16-byte stores fill whole sectors.
template <int CACHE, bool VEC>
struct CacheUnit {
  using CT = typename std::conditional<CACHE == MLA_F32, float, __nv_bfloat16>::type;
  float x[8];
  __device__ __forceinline__ void load(const ReadArgs& a, const uint8_t* pg, int prow, int b) {
    const CT* p = reinterpret_cast<const CT*>(pg) + (size_t)prow * (a.d_c + a.d_rope) + 8 * b;
    if (VEC) {
      load8(p, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = to_f(p[e]);
    }
  }
  __device__ __forceinline__ void values(float (&y)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e];
  }
};
template <bool VEC>
struct CacheUnit<MLA_FP8_E4M3, VEC> {
  uint2 w;
  float s;
  __device__ __forceinline__ void load(const ReadArgs& a, const uint8_t* pg, int prow, int b) {
    w = *reinterpret_cast<const uint2*>(pg + (size_t)prow * a.d_c + 8 * b);
    s = reinterpret_cast<const float*>(pg + fp8_page(a.page_size, a.d_c, a.d_rope).sc_off)[(size_t)prow * (a.d_c / 128) + b / 16];
  }
  __device__ __forceinline__ void values(float (&y)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = e4m3_to_float((uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)))) * s;
  }
};
template <bool VEC>
struct CacheUnit<MLA_FP4_E2M1, VEC> {
  uint32_t w;
  float ts;
  uint8_t sc;
  __device__ __forceinline__ void load(const ReadArgs& a, const uint8_t* pg, int prow, int b) {
    const Fp4Page f4 = fp4_page(a.page_size, a.d_c, a.d_rope);
    w = *reinterpret_cast<const uint32_t*>(pg + (size_t)prow * (a.d_c / 2) + 4 * b);
    sc = pg[f4.sc_off + (size_t)prow * (a.d_c / 16) + b / 2];
    ts = reinterpret_cast<const float*>(pg + f4.ts_off)[prow];
  }
  __device__ __forceinline__ void values(float (&y)[8]) const {
    const float s = e4m3_to_float(sc) * ts;
    uint32_t h[4];
    e2m1x8_to_f16x2(w, h);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = f16x2_to_float2(h[e]);
      y[2 * e] = f.x * s;
      y[2 * e + 1] = f.y * s;
    }
  }
};
template <bool VEC>
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  if (VEC) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = x[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  if (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __float2bfloat16_rn(x[e]);
  }
}

// A warp takes U consecutive tokens of the list: their slots are resolved side
// by side, one lane each, and all their loads are issued before the first is used.
template <typename TO, int CACHE, bool VEC, int U>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ ReadArgs a) {
  pdl_trigger();
  pdl_wait();
  using CT = typename std::conditional<CACHE == MLA_F32, float, __nv_bfloat16>::type;
  const int lane = threadIdx.x & 31, nu = a.d_c / 8;
  constexpr bool kCoded = CACHE == MLA_FP8_E4M3 || CACHE == MLA_FP4_E2M1;
  const size_t kr_off = kCoded ? coded_kr_off(CACHE, a.page_size, a.d_c, a.d_rope) : (size_t)a.d_c * sizeof(CT);
  const int kr_row = kCoded ? a.d_rope : a.d_c + a.d_rope;
  for (long long n0 = (long long)(blockIdx.x * kWarps + (threadIdx.x >> 5)) * U; n0 < a.n_tokens;
       n0 += (long long)gridDim.x * kWarps * U) {
    int my_page = -1, my_row = 0;
    if (lane < U && n0 + lane < a.n_tokens) my_page = row_slot(a, a.seq_idx[n0 + lane], a.pos[n0 + lane], &my_row, true);
    const uint8_t* pg[U];
    int prow[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int page = __shfl_sync(0xffffffffu, my_page, u);
      prow[u] = __shfl_sync(0xffffffffu, my_row, u);
      ok[u] = page >= 0;
      pg[u] = a.pool + (size_t)(ok[u] ? page : 0) * a.page_bytes;
    }
    for (int i = VEC ? 2 * lane : lane; i < a.d_rope; i += VEC ? 64 : 32) {
      float2 k[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ok[u]) {
          const CT* p = reinterpret_cast<const CT*>(pg[u] + kr_off) + (size_t)prow[u] * kr_row + i;
          if (VEC) k[u] = load2(p);
          else k[u].x = to_f(*p);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ok[u]) {
          TO* p = static_cast<TO*>(a.kr_out) + (size_t)(n0 + u) * a.d_rope + i;
          if (VEC) store2(p, k[u]);
          else *p = from_f<TO>(k[u].x);
        }
    }
    for (int b = lane; b < nu; b += 64) {
      CacheUnit<CACHE, VEC> unit[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (ok[u] && b + 32 * j < nu) unit[u][j].load(a, pg[u], prow[u], b + 32 * j);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (ok[u] && b + 32 * j < nu) {
            float y[8];
            unit[u][j].values(y);
            store8<VEC>(static_cast<TO*>(a.c_out) + (size_t)(n0 + u) * a.d_c + 8 * (b + 32 * j), y);
          }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// One warp per per_warp tokens, up to `most` CTAs per SM, then every warp loops.
int rows_grid(int n_tokens, int per_warp, int most) {
  const int ctas = (n_tokens - 1) / (kWarps * per_warp) + 1;
  return ctas < most * device_sm_count() ? ctas : most * device_sm_count();
}

// log2 of a page size that is a power of two, else -1.
int page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size && s < 30) ++s;
  return (1 << s) == page_size ? s : -1;
}

template <typename T, int CACHE>
cudaError_t launch_rows_typed(const RowsArgs& a, bool vec, cudaStream_t st) {
  auto kernel = a.d_c <= 512 ? (vec ? append_rows_kernel<T, CACHE, 1, true> : append_rows_kernel<T, CACHE, 1, false>)
                             : (vec ? append_rows_kernel<T, CACHE, 2, true> : append_rows_kernel<T, CACHE, 2, false>);
  return launch_pdl(kernel, dim3(rows_grid(a.n_tokens, 1, 3)), dim3(kThreads), 0, st, a);
}

template <typename TO, int CACHE>
cudaError_t launch_read_typed(const ReadArgs& a, bool vec, cudaStream_t st) {
  // four tokens a warp once that still gives every SM four CTAs (32,792 tokens of a
  // 4-bit cache: 11.1 us, one token a warp 12.2; 4,096 tokens: one a warp, 3.5)
  if (a.n_tokens >= 4 * 4 * kWarps * device_sm_count()) {
    auto kernel = vec ? read_rows_kernel<TO, CACHE, true, 4> : read_rows_kernel<TO, CACHE, false, 4>;
    return launch_pdl(kernel, dim3(rows_grid(a.n_tokens, 4, 32)), dim3(kThreads), 0, st, a);
  }
  auto kernel = vec ? read_rows_kernel<TO, CACHE, true, 1> : read_rows_kernel<TO, CACHE, false, 1>;
  return launch_pdl(kernel, dim3(rows_grid(a.n_tokens, 1, 32)), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_append_fp4_finalize(const mla_dims& d, const float* raw, int n_tokens, const int32_t* seq_idx,
                                       const int32_t* pos, const int32_t* page_table, int batch, int max_pages,
                                       void* pool, int num_pages, size_t page_bytes, int* status, cudaStream_t st) {
  RowsArgs a = {};
  a.c = raw;
  a.c_stride = d.d_c;
  a.n_tokens = n_tokens;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.page_table = page_table;
  a.batch = batch;
  a.max_pages = max_pages;
  a.pool = static_cast<uint8_t*>(pool);
  a.num_pages = num_pages;
  a.page_bytes = page_bytes;
  a.d_c = d.d_c;
  a.d_rope = d.d_rope;
  a.page_size = d.page_size;
  a.page_shift = page_shift(d.page_size);
  a.status = status;
  a.timeline = timeline_ptr();
  auto kernel = d.d_c <= 512 ? append_fp4_finalize_kernel<1> : append_fp4_finalize_kernel<2>;
  return launch_pdl(kernel, dim3((n_tokens + kWarps - 1) / kWarps), dim3(kThreads), 0, st, a);
}

}  // namespace mla

using namespace mla;

extern "C" int mla_append_rows(const mla_dims* dims, const void* c, int64_t c_stride, const void* k_rope,
                               int64_t k_stride, const void* norm_weight, float norm_eps, int n_tokens,
                               const int32_t* seq_idx, const int32_t* pos, const int32_t* page_table, int batch,
                               int max_pages, void* cache_pool, int num_pages, void* stream) {
  int rc = mla_check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (n_tokens < 0 || batch < 1 || max_pages < 1 || num_pages < 1 || c_stride < dims->d_c || k_stride < dims->d_rope)
    return MLA_ERR_INVALID_ARG;
  if (norm_weight && !(norm_eps > 0.f && isfinite(norm_eps))) return MLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!c || (!k_rope && dims->d_rope > 0) || !seq_idx || !pos || !page_table || !cache_pool) return MLA_ERR_INVALID_ARG;
  if (!aligned16(cache_pool)) return MLA_ERR_ALIGNMENT;
  RowsArgs a = {};
  a.c = c;
  a.c_stride = c_stride;
  a.kr = k_rope;
  a.kr_stride = k_stride;
  a.norm_w = norm_weight;
  a.norm_eps = (double)norm_eps;
  a.inv_dc = 1.0 / (double)dims->d_c;
  a.n_tokens = n_tokens;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.page_table = page_table;
  a.batch = batch;
  a.max_pages = max_pages;
  a.pool = static_cast<uint8_t*>(cache_pool);
  a.num_pages = num_pages;
  a.page_bytes = cache_page_bytes(*dims);
  a.d_c = dims->d_c;
  a.d_rope = dims->d_rope;
  a.page_size = dims->page_size;
  a.page_shift = page_shift(dims->page_size);
  a.rope_base = dims->rope_base;
  a.status = device_status_word();
  a.timeline = timeline_ptr();
  const int half = dims->d_rope / 2;
  const double log_base = log((double)dims->rope_base);
  for (int i = 0; i < half && i < kMaxHalf; ++i) a.inv_freq[i] = exp(-log_base * (double)i / (double)half);
  const size_t es = dims->act_dtype == MLA_F32 ? 4 : 2, cs = dims->cache_dtype == MLA_F32 ? 4 : 2;
  bool vec = aligned16(c) && (size_t)c_stride * es % 16 == 0 && aligned16(norm_weight);
  // unquantised rows lie d_c + d_rope elements apart
  if (!is_coded_cache(*dims))
    vec = vec && (size_t)(dims->d_c + dims->d_rope) * cs % 16 == 0 && a.page_bytes % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  trace_record(MLA_TRACE_APPEND_PROJECT, false, st);
  trace_record(MLA_TRACE_APPEND_PROJECT, true, st);
  trace_record(MLA_TRACE_APPEND_FINALIZE, false, st);
  cudaError_t e;
  const bool f32 = dims->act_dtype == MLA_F32;
  switch (dims->cache_dtype) {
    case MLA_F32: e = launch_rows_typed<float, MLA_F32>(a, vec, st); break;
    case MLA_BF16:
      e = f32 ? launch_rows_typed<float, MLA_BF16>(a, vec, st) : launch_rows_typed<__nv_bfloat16, MLA_BF16>(a, vec, st);
      break;
    case MLA_FP4_E2M1:
      e = f32 ? launch_rows_typed<float, MLA_FP4_E2M1>(a, vec, st)
              : launch_rows_typed<__nv_bfloat16, MLA_FP4_E2M1>(a, vec, st);
      break;
    default:
      e = f32 ? launch_rows_typed<float, MLA_FP8_E4M3>(a, vec, st)
              : launch_rows_typed<__nv_bfloat16, MLA_FP8_E4M3>(a, vec, st);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  trace_record(MLA_TRACE_APPEND_FINALIZE, true, st);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH;
}

extern "C" int mla_read_rows(const mla_dims* dims, const void* cache_pool, int num_pages, const int32_t* page_table,
                             int batch, int max_pages, const int32_t* seq_idx, const int32_t* pos, int n_tokens,
                             void* c_out, void* k_out, void* stream) {
  int rc = mla_check_dims(dims);
  if (rc != MLA_OK) return rc;
  if (n_tokens < 0 || batch < 1 || max_pages < 1 || num_pages < 1) return MLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return MLA_OK;
  if (!cache_pool || !page_table || !seq_idx || !pos || !c_out || (!k_out && dims->d_rope > 0))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(cache_pool)) return MLA_ERR_ALIGNMENT;
  ReadArgs a = {};
  a.pool = static_cast<const uint8_t*>(cache_pool);
  a.num_pages = num_pages;
  a.page_bytes = cache_page_bytes(*dims);
  a.page_table = page_table;
  a.batch = batch;
  a.max_pages = max_pages;
  a.seq_idx = seq_idx;
  a.pos = pos;
  a.n_tokens = n_tokens;
  a.d_c = dims->d_c;
  a.d_rope = dims->d_rope;
  a.page_size = dims->page_size;
  a.page_shift = page_shift(dims->page_size);
  a.c_out = c_out;
  a.kr_out = k_out;
  a.status = device_status_word();
  // output rows of c are d_c (a multiple of 16) elements apart
  const size_t cs = dims->cache_dtype == MLA_F32 ? 4 : 2;
  bool vec = aligned16(c_out) && aligned16(k_out) && dims->d_rope % 2 == 0;
  if (!is_coded_cache(*dims))
    vec = vec && (size_t)(dims->d_c + dims->d_rope) * cs % 16 == 0 && a.page_bytes % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  const bool f32 = dims->act_dtype == MLA_F32;
  switch (dims->cache_dtype) {
    case MLA_F32: e = launch_read_typed<float, MLA_F32>(a, vec, st); break;
    case MLA_BF16:
      e = f32 ? launch_read_typed<float, MLA_BF16>(a, vec, st) : launch_read_typed<__nv_bfloat16, MLA_BF16>(a, vec, st);
      break;
    case MLA_FP4_E2M1:
      e = f32 ? launch_read_typed<float, MLA_FP4_E2M1>(a, vec, st)
              : launch_read_typed<__nv_bfloat16, MLA_FP4_E2M1>(a, vec, st);
      break;
    default:
      e = f32 ? launch_read_typed<float, MLA_FP8_E4M3>(a, vec, st)
              : launch_read_typed<__nv_bfloat16, MLA_FP8_E4M3>(a, vec, st);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? MLA_OK : MLA_ERR_LAUNCH;
}
