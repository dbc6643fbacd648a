// Internal declarations shared by the libmla translation units (device helpers,
// workspace layout, kernel launchers).  Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/mla.h"

namespace mla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kE4M3Max = 448.0f;

// ----------------------------------------------------------------------------
// Device status word: kernels record errors that depend on device-resident
// values (bad page index, short sequence, expired bounded wait) here.
// ----------------------------------------------------------------------------
__device__ __forceinline__ void record_status(int* status, int code) {
  if (status) atomicMax(status, code);
}

// ----------------------------------------------------------------------------
// FP8 cache page: [page_size][d_c] e4m3 codes, then [page_size][d_rope] bf16
// k^R, then [page_size][d_c/128] fp32 scales, each sub-block 128-byte aligned.
// ----------------------------------------------------------------------------
struct Fp8Page {
  size_t kr_off, sc_off;
};
__host__ __device__ inline size_t a128(size_t x) { return (x + 127) / 128 * 128; }
__host__ __device__ inline Fp8Page fp8_page(int page_size, int d_c, int d_rope) {
  Fp8Page p;
  p.kr_off = a128((size_t)page_size * d_c);
  p.sc_off = a128(p.kr_off + (size_t)page_size * d_rope * 2);
  return p;
}

// ----------------------------------------------------------------------------
// 4-bit cache page: [page_size][d_c/2] bytes of e2m1 code pairs (element 2i in
// the low half of byte i), [page_size][d_rope] bf16 k^R, [page_size][d_c/16]
// e4m3 block scales, [page_size] fp32 token scales (powers of two), each
// sub-block 128-byte aligned.  c = code * block scale * token scale.
// ----------------------------------------------------------------------------
struct Fp4Page {
  size_t kr_off, sc_off, ts_off, bytes;
};
__host__ __device__ inline Fp4Page fp4_page(int page_size, int d_c, int d_rope) {
  Fp4Page p;
  p.kr_off = a128((size_t)page_size * (d_c / 2));
  p.sc_off = a128(p.kr_off + (size_t)page_size * d_rope * 2);
  p.ts_off = a128(p.sc_off + (size_t)page_size * (d_c / 16));
  p.bytes = a128(p.ts_off + (size_t)page_size * 4);
  return p;
}
// Offset of the bf16 k^R rows in a page of a quantised cache.
__host__ __device__ inline size_t coded_kr_off(int cache_dtype, int page_size, int d_c, int d_rope) {
  return cache_dtype == MLA_FP4_E2M1 ? fp4_page(page_size, d_c, d_rope).kr_off
                                     : fp8_page(page_size, d_c, d_rope).kr_off;
}

// ----------------------------------------------------------------------------
// Programmatic dependent launch.  The tensor-core kernels are launched with
// programmatic stream serialization: a kernel may start while the previous
// one drains, stages what does not depend on it (weights), and then waits.
// Every such kernel calls pdl_wait() before it reads or writes anything the
// previous kernels of the stream touch, so it also completes after them (the
// ordering stays transitive along the stream).
// ----------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// 2-D bf16 TMA tensor map with the 128-byte swizzle (box_cols * 2 == 128),
// written into `map` (a 64-byte aligned CUtensorMap).  False if the driver
// entry point is missing or the encoder rejects the shape.
bool make_tile_map_bf16(void* map, const void* base, uint64_t cols, uint64_t rows, uint64_t row_bytes,
                        uint32_t box_cols, uint32_t box_rows);

// 3-D map over a sub-block of the cache pages, [pages][rows][row_elems] of bytes
// or bf16, one page's rows x box_cols per box; a box row is 128 or 32 bytes and
// the swizzle the one of that width.
bool make_page_map_swizzled(void* map, const void* base, bool bf16, uint64_t row_elems, uint64_t rows, uint64_t pages,
                            uint64_t page_bytes, uint32_t box_cols);

// ----------------------------------------------------------------------------
// Element access
// ----------------------------------------------------------------------------
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// Load 8 consecutive bf16 (one 16-byte vector) as floats.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* f) {
  uint4 v = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
// Load 8 consecutive floats (two 16-byte vectors).
__device__ __forceinline__ void load8(const float* p, float* f) {
  float4 a = *reinterpret_cast<const float4*>(p);
  float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ float e4m3_to_float(uint8_t code) {
  __nv_fp8_e4m3 v;
  v.__x = code;
  return float(v);
}

// ----------------------------------------------------------------------------
// The 4-bit quantiser.  A token's scale ts is a power of two taken from
// a = max(max|c|, max|k^R| / 64), a block's e4m3 scale s from its own maximum,
// so that every decision below is one fp32 division rounded to the target
// type; s * ts is exact in fp32.  Dividing k^R into the token scale keeps
// k^R / ts inside f16 (at most 2^12) for the attention kernel that scores in
// units of ts.  Non-finite elements take no part in the maxima; their block's
// scale is the e4m3 NaN, so the row's values there read as NaN.
// ----------------------------------------------------------------------------
constexpr int kFp4MinExp = -100;        // smallest token scale 2^-100
constexpr uint32_t kE4M3NaN = 0x7Fu;
__device__ __forceinline__ float fp4_token_scale(float amax_c, float amax_kr) {
  const float a = fmaxf(amax_c, amax_kr * 0.015625f);
  // floor(log2 a) from the exponent field (a subnormal lands below the limit)
  const int k = max((int)(__float_as_uint(a) >> 23) - 127 - 5, kFp4MinExp);
  return a > 0.f ? __uint_as_float((uint32_t)(k + 127) << 23) : 1.0f;
}
__device__ __forceinline__ uint32_t fp4_block_scale(float amax, float ts, bool finite) {
  // amax / (6 ts): the power of two first, exactly, then the sixth with one
  // residual correction (the code is that of the correctly rounded quotient, as
  // at fp4_pair: an e4m3 border has five significant bits, six times it seven)
  const float z = amax * __uint_as_float((254u << 23) - __float_as_uint(ts));
  const float q = z * (1.0f / 6.0f);
  const uint32_t code = (uint32_t)__nv_cvt_float_to_fp8(fmaf(fmaf(-6.0f, q, z), 1.0f / 6.0f, q), __NV_SATFINITE,
                                                        __NV_E4M3);
  return finite ? code : kE4M3NaN;
}
// codes of two elements, the first in the low half; step = block scale * ts,
// inv its correctly rounded reciprocal (0 where step is 0 or NaN: code 0).  The
// quotient is v * inv and one correction by its residual, which is within 2^-44
// of v / step before its last rounding.  That gives the code of the correctly
// rounded quotient: codes change only at m = .25, .75, 1.25, 1.75, 2.5, 3.5 and
// 5.  step has four significant bits, so m step is a float; where v equals it,
// the correction ends on m, and elsewhere v / step is away from m by v's last
// place at least, 2^-23 / 1.97 of m, more than half of the quotient's last place
// (2^-24).  Steps lie in [2^-109, 2^126], so near a border nothing underflows.
__device__ __forceinline__ float fp4_inverse(float step) { return step > 0.f ? __frcp_rn(step) : 0.f; }
__device__ __forceinline__ uint32_t fp4_pair(float v0, float v1, float step, float inv) {
  const float q0 = v0 * inv, q1 = v1 * inv;
  const float c0 = fmaf(fmaf(-q0, step, v0), inv, q0), c1 = fmaf(fmaf(-q1, step, v1), inv, q1);
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(c0, c1), __NV_E2M1, cudaRoundNearest);
}
// |v| for the maxima: non-finite elements count as 0 and clear `finite`
__device__ __forceinline__ float finite_abs(float v, bool& finite) {
  const float x = fabsf(v);
  const bool f = x < INFINITY;
  finite = finite && f;
  return f ? x : 0.f;
}
// Eight codes (one 32-bit word, first code in the low bits) as exact f16 pairs.
// (The bytes are taken apart inside the asm block: the conversion reads them
// in place.  cuda_fp4.h's one-byte conversions cost an extraction each:
// measured 47 against 96 codes per cycle and SM with 16 warps.)
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// f16 pairs held as 32-bit words
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// the larger of each two; of a NaN and a number the number
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// two e4m3 codes (low byte first) as an f16 pair
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t s) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(s));
  return d;
}
__device__ __forceinline__ uint32_t dup_lo(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t h) { return __byte_perm(h, h, 0x3232); }
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// RoPE frequency of rotation pair i of a d_rope-wide vector: base^(-i/half),
// in double precision.
__device__ __forceinline__ double rope_inv_freq(int i, int half, float base) {
  return exp(-log((double)base) * (double)i / (double)half);
}

// cos / sin of the RoPE angle pos * inv_freq.  The angle is formed in double
// precision (positions reach 1.3e5, where a float angle is off by ~1e-2 rad),
// brought into [-pi, pi] by Cody-Waite reduction against 2*pi held as the sum
// of two doubles, and the reduced angle is evaluated in float (|error| of a
// few 1e-7).
__device__ __forceinline__ void rope_cos_sin_at(int pos, double inv_freq, float* c, float* s) {
  constexpr double kTwoPiHi = 6.283185307179586232;    // 2*pi rounded to double
  constexpr double kTwoPiLo = 2.4492935982947064e-16;  // 2*pi - kTwoPiHi
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double ang = (double)pos * inv_freq;
  const double k = rint(ang * kInvTwoPi);
  const double r = fma(-k, kTwoPiLo, fma(-k, kTwoPiHi, ang));
  sincosf((float)r, s, c);
}

__device__ __forceinline__ void rope_cos_sin(int pos, int i, int half, float base, float* c, float* s) {
  rope_cos_sin_at(pos, rope_inv_freq(i, half, base), c, s);
}

// ----------------------------------------------------------------------------
// Decode workspace layout (shared by mla_decode and mla_combine)
//   plan  : int32 [batch + 1] first key tile of each sequence (prefix sum of
//           ceil(seq_len / page_size)), then int32 [4] {total tiles, splits,
//           batch, n_q}, then int32 [batch][2] {first split, split count}
//           overlapping each sequence
//   q_abs : [batch, n_q, n_heads, d_c + d_rope] act type (absorbed queries,
//           rotated q^R appended)
//   o_part: [n_q, n_slots, n_heads, d_c] per-split normalised latent sums in
//           rows of the decode kernel's PartType (16-bit rows in the first half
//           of the region)
//   lse   : float32 [n_q, n_slots, n_heads] per-split log2-sum-exp2 of the scores
//           scaled by softmax_scale*log2(e) (-inf for an empty split, NaN for one
//           with a visible key whose score is NaN)
// A split w covers global key tiles [w*TT/W, (w+1)*TT/W) of the concatenated
// sequences; its piece of sequence b goes to slot w + b (n_slots = batch + W - 1).
// ----------------------------------------------------------------------------
struct DecodeLayout {
  size_t off_plan, off_q, off_o, off_lse, total;
  int splits, n_slots;
};

inline bool is_coded_cache(const mla_dims& d) {
  return d.cache_dtype == MLA_FP8_E4M3 || d.cache_dtype == MLA_FP4_E2M1;
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline DecodeLayout decode_layout(const mla_dims& d, int batch, int n_q, int splits) {
  DecodeLayout L;
  L.splits = splits;
  L.n_slots = batch + splits - 1;
  size_t act = d.act_dtype == MLA_F32 ? 4 : 2;
  size_t D = (size_t)d.d_c + d.d_rope;
  size_t off = 0;
  L.off_plan = off;
  off = align_up(off + sizeof(int32_t) * ((size_t)batch + 1 + 4 + 2 * (size_t)batch), 256);
  L.off_q = off;
  off = align_up(off + act * (size_t)batch * n_q * d.n_heads * D, 256);
  L.off_o = off;
  off = align_up(off + 4 * (size_t)n_q * L.n_slots * d.n_heads * d.d_c, 256);
  L.off_lse = off;
  off = align_up(off + 4 * (size_t)n_q * L.n_slots * d.n_heads, 256);
  L.total = off;
  return L;
}

// Tile range of split w: [w*TT/W, (w+1)*TT/W).
__host__ __device__ __forceinline__ long long split_tile_begin(int w, long long TT, int W) {
  return (long long)w * TT / W;
}

// Index of the sequence that owns global tile g: the largest b with tile_start[b] <= g.
__device__ __forceinline__ int seq_of_tile(const int32_t* tile_start, int batch, long long g) {
  int lo = 0, hi = batch;  // tile_start[0] = 0 <= g
  while (hi - lo > 1) {
    int mid = (lo + hi) >> 1;
    if ((long long)tile_start[mid] <= g) lo = mid; else hi = mid;
  }
  return lo;
}

struct DecodeParams {
  mla_dims d;
  const void* q_abs;       // workspace q_abs
  const uint8_t* pool;     // cache pool
  size_t page_bytes;
  int num_pages;
  const int32_t* page_table;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* plan;     // tile_start [batch+1], then {TT, W, batch, n_q}
  float* o_part;
  float* lse_part;
  int batch, n_q, splits, n_slots;
  float scale_log2;        // softmax_scale * log2(e)
  int* status;
  unsigned long long* timeline;  // device timeline (null: off)
};

// Tracing hook: events installed by mla_set_trace_events (may be null).
void trace_record(int kernel, bool end, cudaStream_t st);

// Device timeline installed by mla_set_timeline (null when off): the
// launchers copy it into each kernel's arguments.  Per kernel k (MLA_TRACE_*),
// thread 0 of every CTA keeps in [2k] the earliest %globaltimer at which a CTA
// passed its grid-dependency wait and in [2k + 1] the latest at which one
// finished, so a graph replay of a step gives each kernel's span on the device.
unsigned long long* timeline_ptr();

__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void tl_begin(unsigned long long* tl, int k) {
  if (tl && threadIdx.x == 0) atomicMin(tl + 2 * k, global_ns());
}
// at the end of a CTA: the CTA's other threads are done first (tl is uniform
// over the grid, so the barrier is taken by all threads or none)
__device__ __forceinline__ void tl_end(unsigned long long* tl, int k) {
  if (tl) {
    __syncthreads();
    if (threadIdx.x == 0) atomicMax(tl + 2 * k + 1, global_ns());
  }
}
// at the end of a CTA whose threads have already synchronised
__device__ __forceinline__ void tl_end_nosync(unsigned long long* tl, int k) {
  if (tl && threadIdx.x == 0) atomicMax(tl + 2 * k + 1, global_ns());
}

// ----------------------------------------------------------------------------
// Launchers (host side), each returning cudaError_t of the launch.
// ----------------------------------------------------------------------------
cudaError_t launch_append(const mla_dims& d, const void* h, int n_tokens, const int32_t* seq_idx,
                          const int32_t* pos, const void* W_dkv, const void* W_kr,
                          const int32_t* page_table, int batch, int max_pages, void* pool,
                          int num_pages, size_t page_bytes, float* raw, size_t raw_floats, int* status,
                          cudaStream_t st);
// fp32 scratch (floats) with which launch_append takes its split-K path for
// these dims and token count, or 0 when that path does not apply
size_t append_splitk_floats(const mla_dims& d, int n_tokens);

// 4-bit caches: c rows of fp32 scratch -> codes and scales of the rows whose
// k^R the projection has already stored
cudaError_t launch_append_fp4_finalize(const mla_dims& d, const float* raw, int n_tokens, const int32_t* seq_idx,
                                       const int32_t* pos, const int32_t* page_table, int batch, int max_pages,
                                       void* pool, int num_pages, size_t page_bytes, int* status, cudaStream_t st);

// absorb + split plan (+ empty-split initialisation of the lse slots)
cudaError_t launch_absorb_and_plan(const mla_dims& d, const void* q_nope, const void* q_rope, const void* W_uk,
                                   const int32_t* seq_lens, int batch, int n_q, int max_pages, int splits,
                                   void* q_abs, bool q_abs_f16, bool q_rope_bf16, int32_t* plan, float* lse_part, size_t lse_count,
                                   int* status, cudaStream_t st);

cudaError_t launch_decode_simt(const DecodeParams& p, cudaStream_t st);

bool decode_tc_supported(const mla_dims& d, int n_q);
// the tensor-core path for this cache reads the absorbed queries as f16
bool decode_tc_wants_f16_queries(const mla_dims& d);
// ... but for the rotated q^R, which it reads as bf16 beside a bf16 k^R
bool decode_tc_wants_bf16_q_rope(const mla_dims& d);
// multiprocessor count of the current device (cached per device)
int device_sm_count();

// Timeline stamps for latency studies, compiled in only with MLA_TC_TRACE:
// per event slot, the earliest and latest %globaltimer over the CTAs whose
// thread 0 reaches it.  Each translation unit keeps its own table and exports
// mla_stamps_<unit>(host, reset) to read (and re-arm) it.
#ifdef MLA_TC_TRACE
namespace {
__device__ unsigned long long g_stamps[16][2];
}
__device__ __forceinline__ void mla_stamp_now(int e) {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  atomicMin(&g_stamps[e][0], t);
  atomicMax(&g_stamps[e][1], t);
}
#define MLA_STAMP(e)                          \
  do {                                        \
    if (threadIdx.x == 0) mla_stamp_now(e);   \
  } while (0)
#define MLA_STAMP_ANY(e) mla_stamp_now(e)
#define MLA_STAMP_EXPORT(unit)                                                                  \
  extern "C" int mla_stamps_##unit(unsigned long long* host, int reset) {                       \
    if (host && cudaMemcpyFromSymbol(host, mla::g_stamps, sizeof(mla::g_stamps)) != cudaSuccess) \
      return 1;                                                                                 \
    if (reset) {                                                                                \
      unsigned long long init[16][2];                                                           \
      for (int i = 0; i < 16; ++i) {                                                            \
        init[i][0] = ~0ull;                                                                     \
        init[i][1] = 0ull;                                                                      \
      }                                                                                         \
      if (cudaMemcpyToSymbol(mla::g_stamps, init, sizeof(init)) != cudaSuccess) return 1;       \
    }                                                                                           \
    return 0;                                                                                   \
  }
#else
#define MLA_STAMP(e) ((void)0)
#define MLA_STAMP_ANY(e) ((void)0)
#define MLA_STAMP_EXPORT(unit)
#endif
cudaError_t launch_decode_tc(const DecodeParams& p, cudaStream_t st);
cudaError_t launch_decode_tc_fp4(const DecodeParams& p, cudaStream_t st);
// few query rows over a 4-bit cache, warp-level tensor cores (decode_few.cu)
bool decode_few_supported(const mla_dims& d, int n_q);
int decode_few_auto_splits(int num_sms);
cudaError_t launch_decode_few(const DecodeParams& p, cudaStream_t st);
int decode_tc_auto_splits(const mla_dims& d, int num_sms, int n_q);

// The split partials' rows as the decode kernels write them: fp32 (CUDA cores;
// warp-level MMA over a 4-bit cache), bf16 (tcgen05, bf16 and FP8 caches), f16
// (tcgen05, 4-bit cache).  two_terms: the combine's product takes the merged
// latent sum as two bf16 terms, not one rounded to bf16.
enum PartType { kPartF32 = 0, kPartBf16 = 1, kPartF16 = 2 };
cudaError_t launch_combine(const mla_dims& d, const void* W_uv, int batch, int n_q, const int32_t* plan,
                           const float* o_part, PartType part, bool two_terms, const float* lse_part, void* out, float* lse_out,
                           int* status, cudaStream_t st);

}  // namespace mla
