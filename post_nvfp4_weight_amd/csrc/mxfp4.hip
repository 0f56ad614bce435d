// Microscaled 4-bit floating point (MXFP4: E2M1 elements, one power of two per
// 32 of them along k) and its product:
//   quantize:  E = clamp(floor(log2 max|x|) - 2, -127, 127) per block, codes the nearest E2M1 of x 2^-E
//   product:   Y = Xq Wq^T, both operands MXFP4, on the block-scaled matrix cores
// The matrix cores read the codes and the scale bytes as they are stored, so
// nothing is expanded: v_mfma_scale_f32_*_f8f6f4 takes 32 codes (16 bytes)
// and one scale byte per lane and accumulates in fp32.  Products of two E2M1
// values are exact.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace nvq {

namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---- quantization -------------------------------------------------------------
// A block's scale byte from its largest magnitude's exponent field e (of bf16
// and fp32 alike): floor(log2 a) = e - 127 for normal a, so the byte is e - 2,
// and 0 (2^-127) for everything smaller, zero too; 255 (NaN) for a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t e) { return e == 255 ? 255 : max(e, 2u) - 2; }
// What the conversions divide by: they take the exponent field alone, 0 for 2^-127.
__device__ __forceinline__ float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }
// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

// (By value: a bit cast of a vector's element itself reads the vector's first.)
__device__ __forceinline__ bf16x2 pair_of(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// Eight values as loaded.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *(const u32x4_a2*)p; }
  __device__ __forceinline__ uint32_t top_exponent() const {   // of the largest magnitude
    u16x2 a{0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) a = __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    return max(a.x, a.y) >> 7;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(v[3]), s, 3);
  }
};
template <>
struct Eight<float> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *(const f32x4_a4*)p;
    v[1] = *(const f32x4_a4*)(p + 4);
  }
  __device__ __forceinline__ uint32_t top_exponent() const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i >> 2][i & 3]) & 0x7FFFFFFFu);
    return a >> 23;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0][0], v[0][1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0][2], v[0][3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[1][0], v[1][1], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[1][2], v[1][3], s, 3);
  }
};

constexpr int QU = 4;   // units of eight values per thread

// Four lanes per block, eight values each.  FLAT: rows without gaps, so that a
// unit's place is its number.
template <typename T, bool FLAT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ X, int64_t units, int64_t upr, int64_t ldx,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  for (int64_t base = (int64_t)blockIdx.x * (256 * QU); base < units; base += (int64_t)gridDim.x * (256 * QU)) {
    Eight<T> x[QU];
#pragma unroll
    for (int j = 0; j < QU; ++j) {
      const int64_t u = base + j * 256 + threadIdx.x;
      if (u >= units) continue;
      if (FLAT) {
        x[j].load(X + 8 * u);
      } else {
        const int64_t row = units <= 0xFFFFFFFFll ? (int64_t)((uint32_t)u / (uint32_t)upr) : u / upr;
        x[j].load(X + row * ldx + 8 * (u - row * upr));
      }
    }
#pragma unroll
    for (int j = 0; j < QU; ++j) {
      const int64_t u = base + j * 256 + threadIdx.x;
      if (u >= units) continue;   // whole blocks: their number of units is a multiple of 4
      uint32_t e = x[j].top_exponent();
      e = max(e, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)e, 0xB1, 0xF, 0xF, false));   // lanes 1, 0, 3, 2
      e = max(e, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)e, 0x4E, 0xF, 0xF, false));   // lanes 2, 3, 0, 1
      const uint32_t byte = scale_byte(e);
      ((uint32_t*)codes)[u] = byte == 255 ? 0u : x[j].codes(scale_operand(byte));
      if ((threadIdx.x & 3) == 0) scales[u >> 2] = (uint8_t)byte;
    }
  }
}

// VPT values per thread, 16 bytes of output.
template <int OUT_BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                            int64_t units, void* __restrict__ out) {
  constexpr int VPT = OUT_BF16 ? 8 : 4;
  for (int64_t base = (int64_t)blockIdx.x * (256 * QU); base < units; base += (int64_t)gridDim.x * (256 * QU)) {
    uint32_t w[QU], b[QU];
#pragma unroll
    for (int j = 0; j < QU; ++j) {
      const int64_t u = base + j * 256 + threadIdx.x;
      if (u >= units) continue;
      w[j] = OUT_BF16 ? ((const uint32_t*)codes)[u] : ((const uint16_t*)codes)[u];
      b[j] = scales[u * VPT / 32];
    }
#pragma unroll
    for (int j = 0; j < QU; ++j) {
      const int64_t u = base + j * 256 + threadIdx.x;
      if (u >= units) continue;
      const float s = scale_value(b[j]);
      const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 1);
      if (OUT_BF16) {   // (two significant bits: exact in bf16, below its normal range too)
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 3);
        ((bf16x8*)out)[u] = bf16x8{(__bf16)(p0.x * s), (__bf16)(p0.y * s), (__bf16)(p1.x * s), (__bf16)(p1.y * s),
                                   (__bf16)(p2.x * s), (__bf16)(p2.y * s), (__bf16)(p3.x * s), (__bf16)(p3.y * s)};
      } else {
        ((f32x4*)out)[u] = f32x4{p0.x * s, p0.y * s, p1.x * s, p1.y * s};
      }
    }
  }
}

// ---- the product ----------------------------------------------------------------

__device__ __forceinline__ i32x8 fragment(u32x4 v) { return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0}; }

// A lane's 32 values of one block, to codes and scale byte; the bits of mx_quantize_kernel.
template <typename T>
__device__ __forceinline__ void quantize_block(const T* __restrict__ p, u32x4& w, uint32_t& byte) {
  Eight<T> x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j].load(p + 8 * j);
  byte = scale_byte(max(max(x[0].top_exponent(), x[1].top_exponent()), max(x[2].top_exponent(), x[3].top_exponent())));
  const float s = scale_operand(byte);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = byte == 255 ? 0u : x[j].codes(s);
}

// Few rows: 16 CG output channels per workgroup, the eight waves each a part
// of k, all rows in NG groups of 16.
//   v_mfma_scale_f32_16x16x128_f8f6f4, A = 16 channels, B = 16 rows: lane
//   (c = l % 16, q = l / 16) holds block q of a step of 128 k, of channel c and of row c.
// A wave takes chunks of 512 k (four steps: a channel's 16 scale bytes in one
// load) in turn with the other waves.  Rows that are not quantized yet are
// quantized by the lane that multiplies them: its fragment is one block.  The
// waves' partial sums are added in wave order through LDS.
constexpr int FW = 8;

// XT: uint8_t (codes, with scales), uint16_t (bf16) or float.
template <typename XT, int NG, int CG, int OUT_BF16>
__global__ __launch_bounds__(64 * FW) void mx_few_kernel(const XT* __restrict__ X, const uint8_t* __restrict__ xscales,
                                                         int64_t n, int64_t k, int64_t ldx,
                                                         const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t m,
                                                         void* __restrict__ Y, int64_t ldy) {
  constexpr bool kCodes = sizeof(XT) == 1;
  __shared__ __attribute__((aligned(16))) float part[FW][16 * NG][16 * CG + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int64_t kb = k / 32, o0 = (int64_t)blockIdx.x * (16 * CG);
  const uint8_t *wc[CG], *wsc[CG];
#pragma unroll
  for (int f = 0; f < CG; ++f) {
    const int64_t o = min(o0 + 16 * f + c, m - 1);   // (channels past m repeat the last one and are not stored)
    wc[f] = codes + o * (k / 2) + 16 * q;
    wsc[f] = scales + o * kb;
  }
  const XT* xr[NG];
  const uint8_t* xs[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int64_t t = min((int64_t)(16 * g + c), n - 1);
    xr[g] = X + (kCodes ? t * (k / 2) + 16 * q : t * ldx + 32 * q);
    xs[g] = kCodes ? xscales + t * kb : nullptr;
  }
  f32x4 acc[NG][CG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int f = 0; f < CG; ++f) acc[g][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Chunk {
    u32x4 w[CG][4], s[CG];
  };
  auto load_chunk = [&](int64_t ch, Chunk& x) {
#pragma unroll
    for (int f = 0; f < CG; ++f) {
      x.s[f] = *(const u32x4_any*)(wsc[f] + 16 * ch);
#pragma unroll
      for (int j = 0; j < 4; ++j) x.w[f][j] = *(const u32x4*)(wc[f] + 256 * ch + 64 * j);
    }
  };
  auto step = [&](const u32x4 (&w)[CG], const uint32_t (&s)[CG], int g, u32x4 xv, uint32_t xsc) {
#pragma unroll
    for (int f = 0; f < CG; ++f)
      acc[g][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fragment(w[f]), fragment(xv), acc[g][f], 4, 4, 0, (int)s[f], 0, (int)xsc);
  };
  const int64_t whole = k / 512;
  Chunk next;
  if (wave < whole) load_chunk(wave, next);
  for (int64_t ch = wave; ch < whole; ch += FW) {
    const Chunk cur = next;
    if (ch + FW < whole) load_chunk(ch + FW, next);
    u32x4 xsv[NG];
    if (kCodes)
#pragma unroll
      for (int g = 0; g < NG; ++g) xsv[g] = *(const u32x4_any*)(xs[g] + 16 * ch);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 w[CG];
      uint32_t s[CG];
#pragma unroll
      for (int f = 0; f < CG; ++f) {
        w[f] = cur.w[f][j];
        s[f] = cur.s[f][j] >> (8 * q);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        u32x4 xv;
        uint32_t xb;
        if constexpr (kCodes) {
          xv = *(const u32x4*)(xr[g] + 256 * ch + 64 * j);
          xb = xsv[g][j] >> (8 * q);
        } else {
          quantize_block(xr[g] + 512 * ch + 128 * j, xv, xb);
        }
        step(w, s, g, xv, xb);
      }
    }
  }
  // The rest of k, less than a chunk: blocks past k as zero codes under scale 1.
  if (wave == whole % FW) {
    for (int64_t b0 = 16 * whole; b0 < kb; b0 += 4) {
      const bool in = b0 + q < kb;
      u32x4 w[CG];
      uint32_t s[CG];
#pragma unroll
      for (int f = 0; f < CG; ++f) {
        w[f] = in ? *(const u32x4*)(wc[f] + 16 * b0) : u32x4{0u, 0u, 0u, 0u};
        s[f] = in ? wsc[f][b0 + q] : 127u;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        u32x4 xv{0u, 0u, 0u, 0u};
        uint32_t xb = 127;
        if (in) {
          if constexpr (kCodes) {
            xv = *(const u32x4*)(xr[g] + 16 * b0);
            xb = xs[g][b0 + q];
          } else {
            quantize_block(xr[g] + 32 * b0, xv, xb);
          }
        }
        step(w, s, g, xv, xb);
      }
    }
  }
  // Accumulator register r of lane l: channel 4 q + r, row c.
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int f = 0; f < CG; ++f) *(f32x4*)&part[wave][16 * g + c][16 * f + 4 * q] = acc[g][f];
  __syncthreads();
  for (int i = tid; i < 256 * NG * CG; i += 64 * FW) {
    const int r = i / (16 * CG), o = i % (16 * CG);
    if (r >= n || o0 + o >= m) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < FW; ++w) v += part[w][r][o];
    const int64_t at = r * ldy + o0 + o;
    if (OUT_BF16) ((__bf16*)Y)[at] = (__bf16)v;
    else ((float*)Y)[at] = v;
  }
}

// Many rows: tiles of 32 FA WM output channels x 32 FB WN rows per workgroup of
// WM x WN waves, each 32 FA channels x 32 FB rows.
//   v_mfma_scale_f32_32x32x64_f8f6f4, A = 32 channels, B = 32 rows: lane
//   (r = l % 32, h = l / 32) holds one block of channel r and of row r.
//   k goes in stages of 256, four products deep: a row's 128 bytes of codes
//   and 8 scale bytes.  Product s takes block s for h = 0 and block 4 + s for
//   h = 1 (the order of k in the sum is free, as long as both operands agree),
//   so that the lane's four scale bytes are one word whose byte s the
//   instruction selects.
//   Codes are copied to LDS directly, one stage ahead, 16-byte pieces swizzled
//   by (row / 2) % 8: the 16 rows that are read at once then touch all 64
//   banks.  Scales go through registers (they may start at any byte).
template <int WM, int WN, int FA, int FB>
struct MxTile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kM = 32 * FA * WM, kN = 32 * FB * WN, kAll = kM + kN;
  static constexpr int kWLoads = kM / 8 / kWaves, kXLoads = kN / 8 / kWaves;
  static constexpr int kWBuf = kM * 128, kXBuf = kN * 128, kSBuf = kAll * 8;
  static constexpr int kLds = 2 * (kWBuf + kXBuf + kSBuf);
  static constexpr int kSPer = (kAll + kThreads - 1) / kThreads;   // rows of scales per thread
  static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0, "whole copies per wave");
};

__device__ __forceinline__ constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// NL copies of 1024 bytes to LDS (16 per lane), from `src` + off[q]; offsets at or past the bound bring zeros.
template <int NL, int STRIDE>
__device__ __forceinline__ void copy_rows(char* __restrict__ dst, const void* src, uint32_t bound, const uint32_t (&off)[NL],
                                          uint32_t add, bool in) {
#if __HIP_DEVICE_COMPILE__
  __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, (short)0, bound, 0x00020000);
#pragma unroll
  for (int q = 0; q < NL; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + q * STRIDE), 16,
                                             in ? off[q] + add : 0xFFFFFFF0u, 0, 0, 0);
#endif
}

// One stage: four products deep from wb, xb (codes) and sw, sx (scales); the
// buffers that the copies in flight fill are others, which the restrict
// qualifiers state, so that reads need not wait for them.
template <int S, int FA, int FB>
__device__ __forceinline__ void mx_product(const u32x4 (&a)[FA], const u32x4 (&b)[FB], const uint32_t (&sa)[FA],
                                           const uint32_t (&sb)[FB], f32x16 (&acc)[FA][FB]) {
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fragment(a[i]), fragment(b[j]), acc[i][j], 4, 4, S, (int)sa[i], S,
                                                                  (int)sb[j]);
}
template <int FA, int FB>
__device__ __forceinline__ void mx_stage(const char* __restrict__ wb, const char* __restrict__ xb, const char* __restrict__ sw,
                                         const char* __restrict__ sx, const int (&rd)[4], f32x16 (&acc)[FA][FB]) {
  uint32_t sa[FA], sb[FB];
#pragma unroll
  for (int i = 0; i < FA; ++i) sa[i] = *(const uint32_t*)(sw + i * 256);
#pragma unroll
  for (int j = 0; j < FB; ++j) sb[j] = *(const uint32_t*)(sx + j * 256);
  u32x4 a[2][FA], b[2][FB];
  auto read = [&](int s, int p) {
#pragma unroll
    for (int i = 0; i < FA; ++i) a[p][i] = *(const u32x4*)(wb + i * 4096 + rd[s]);
#pragma unroll
    for (int j = 0; j < FB; ++j) b[p][j] = *(const u32x4*)(xb + j * 4096 + rd[s]);
  };
  read(0, 0);
  read(1, 1);
  mx_product<0, FA, FB>(a[0], b[0], sa, sb, acc);
  read(2, 0);
  mx_product<1, FA, FB>(a[1], b[1], sa, sb, acc);
  read(3, 1);
  mx_product<2, FA, FB>(a[0], b[0], sa, sb, acc);
  mx_product<3, FA, FB>(a[1], b[1], sa, sb, acc);
}

// A row's 8 scale bytes of the stage, `left` blocks to the end of k (zeros
// stand for what is behind it: its codes are zeros too).
__device__ __forceinline__ u32x2 stage_scales(const uint8_t* __restrict__ p, int64_t left) {
  if (left >= 8) return *(const u32x2_any*)p;
  u32x2 v{0u, 0u};
#pragma unroll
  for (int b = 0; b < 8; ++b)
    if (b < left) v[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
  return v;
}

template <int WM, int WN, int FA, int FB, int OUT_BF16>
__global__ __launch_bounds__(64 * WM * WN) void mx_tile_kernel(const uint8_t* __restrict__ xcodes,
                                                               const uint8_t* __restrict__ xscales, int64_t n, int64_t k,
                                                               const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t m,
                                                               void* __restrict__ Y, int64_t ldy) {
  using TL = MxTile<WM, WN, FA, FB>;
  constexpr int NW = TL::kWaves;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, wm = wave / WN, wn = wave % WN;

  // The tiles are dealt to the 8 XCDs (blockIdx.x mod 8) in contiguous runs of
  // an order that walks 8 row tiles, then the next channel tile, so that the
  // tiles that run together in an XCD share operands in its L2.
  const uint32_t ntm = (uint32_t)((m + TL::kM - 1) / TL::kM), ntn = (uint32_t)((n + TL::kN - 1) / TL::kN);
  const uint64_t all = (uint64_t)ntm * ntn, per = (all + 7) / 8;
  const uint64_t id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || id >= all) return;
  const uint64_t panel = id / (8ull * ntm), in_panel = id - panel * 8 * ntm;
  const uint32_t high = (uint32_t)min((uint64_t)8, ntn - panel * 8);
  const int64_t o0 = (int64_t)(in_panel / high) * TL::kM, t0 = (int64_t)(panel * 8 + in_panel % high) * TL::kN;

  const int64_t kh = k / 2, kb = k / 32;
  const int64_t om = min((int64_t)TL::kM, m - o0), tn = min((int64_t)TL::kN, n - t0);   // channels and rows that are there
  codes += o0 * kh;
  scales += o0 * kb;
  xcodes += t0 * kh;
  xscales += t0 * kb;
  const uint32_t wbound = (uint32_t)(om * kh), xbound = (uint32_t)(tn * kh);   // (below 2^32: checked on the host)

  // Copy q of a stage: rows 8 (NW q + wave) + lane / 8, piece (lane % 8) ^ (row / 2) % 8.
  const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
  uint32_t woff[TL::kWLoads], xoff[TL::kXLoads];
#pragma unroll
  for (int q = 0; q < TL::kWLoads; ++q) {
    const int row = 8 * (NW * q + wave) + (lane >> 3);
    woff[q] = row < om ? (uint32_t)(row * kh) + 16 * piece : 0xC0000000u;
  }
#pragma unroll
  for (int q = 0; q < TL::kXLoads; ++q) {
    const int row = 8 * (NW * q + wave) + (lane >> 3);
    xoff[q] = row < tn ? (uint32_t)(row * kh) + 16 * piece : 0xC0000000u;
  }
  char *w0 = smem, *w1 = w0 + TL::kWBuf, *x0 = w1 + TL::kWBuf, *x1 = x0 + TL::kXBuf, *s0 = x1 + TL::kXBuf, *s1 = s0 + TL::kSBuf;
  const int64_t nst = (k + 255) / 256;
  auto copy = [&](int64_t st, char* w, char* x) {
    const bool in = st * 128 + 16 * piece < kh;
    copy_rows<TL::kWLoads, NW * 1024>(w + wave * 1024, codes, wbound, woff, (uint32_t)(st * 128), in);
    copy_rows<TL::kXLoads, NW * 1024>(x + wave * 1024, xcodes, xbound, xoff, (uint32_t)(st * 128), in);
  };
  u32x2 sreg[TL::kSPer];
  auto load_scales = [&](int64_t st) {
#pragma unroll
    for (int q = 0; q < TL::kSPer; ++q) {
      const int row = q * TL::kThreads + tid;
      if (row >= TL::kAll) continue;
      const uint8_t* p = row < TL::kM ? scales + min((int64_t)row, om - 1) * kb : xscales + min((int64_t)(row - TL::kM), tn - 1) * kb;
      sreg[q] = stage_scales(p + 8 * st, kb - 8 * st);
    }
  };
  auto store_scales = [&](char* s) {
#pragma unroll
    for (int q = 0; q < TL::kSPer; ++q) {
      const int row = q * TL::kThreads + tid;
      if (row < TL::kAll) *(u32x2*)(s + row * 8) = sreg[q];
    }
  };
  int rd[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) rd[s] = r * 128 + (((4 * h + s) ^ ((r >> 1) & 7)) * 16);
  const int wrow = wm * 32 * FA, xrow = wn * 32 * FB;

  f32x16 acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  load_scales(0);
  copy(0, w0, x0);
  store_scales(s0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
  asm volatile("s_barrier" ::: "memory");
  for (int64_t st = 0; st < nst; ++st) {
    if (st + 1 < nst) {
      load_scales(st + 1);
      copy(st + 1, w1, x1);
    }
    __builtin_amdgcn_sched_barrier(0);
    mx_stage<FA, FB>(w0 + wrow * 128, x0 + xrow * 128, s0 + (wrow + r) * 8 + 4 * h, s0 + (TL::kM + xrow + r) * 8 + 4 * h, rd, acc);
    __builtin_amdgcn_sched_barrier(0);
    if (st + 1 < nst) store_scales(s1);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    asm volatile("s_barrier" ::: "memory");
    char* t = w0;
    w0 = w1;
    w1 = t;
    t = x0;
    x0 = x1;
    x1 = t;
    t = s0;
    s0 = s1;
    s1 = t;
  }

  // Accumulator: lane l, register e -> channel 8 (e / 4) + 4 h + e % 4, row r.
  // 32 rows at a time go through LDS of the wave's own, so that a row's
  // channels leave in 16-byte pieces side by side.
  constexpr int ES = OUT_BF16 ? 2 : 4, ROW = 32 * FA * ES + 16, PR = 32 * FA * ES / 16;
  static_assert(NW * 32 * ROW <= TL::kLds, "output staging");
  char* stage = smem + wave * 32 * ROW;
  const int64_t oc = o0 + wrow;
#pragma unroll
  for (int j = 0; j < FB; ++j) {
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        char* p = stage + r * ROW + (32 * i + 8 * e4 + 4 * h) * ES;
        const float v0 = acc[i][j][4 * e4], v1 = acc[i][j][4 * e4 + 1], v2 = acc[i][j][4 * e4 + 2], v3 = acc[i][j][4 * e4 + 3];
        if (OUT_BF16) {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          *(bf16x4*)p = bf16x4{(__bf16)v0, (__bf16)v1, (__bf16)v2, (__bf16)v3};
        } else {
          *(f32x4*)p = f32x4{v0, v1, v2, v3};
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int q = 0; q < 32 * PR / 64; ++q) {
      const int e = q * 64 + lane, row = e / PR, pc = e % PR;
      const u32x4 v = *(const u32x4*)(stage + row * ROW + pc * 16);
      const int64_t t = t0 + xrow + 32 * j + row, o = oc + pc * (16 / ES);
      if (t >= n) continue;
      if (o + 16 / ES <= m) {
        *(u32x4_a2*)((char*)Y + (t * ldy + o) * ES) = v;
      } else {
#pragma unroll
        for (int x = 0; x < 16 / ES; ++x)
          if (o + x < m) {
            if (OUT_BF16) ((uint16_t*)Y)[t * ldy + o + x] = (uint16_t)(v[x >> 1] >> (16 * (x & 1)));
            else ((uint32_t*)Y)[t * ldy + o + x] = v[x];
          }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

}  // namespace

hipError_t mxfp4_quantize_launch(const void* X, int bf16, int64_t n, int64_t k, int64_t ldx, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  const int64_t upr = k / 8, units = n * upr;
  const bool flat = ldx == k || n == 1;
  const unsigned blocks = (unsigned)std::min<int64_t>((units + 256 * QU - 1) / (256 * QU), 1 << 20);
#define NVQ_Q(T, FLAT) hipLaunchKernelGGL((mx_quantize_kernel<T, FLAT>), dim3(blocks), dim3(256), 0, s, (const T*)X, units, upr, ldx, codes, scales)
  if (bf16) {
    if (flat) NVQ_Q(uint16_t, true);
    else NVQ_Q(uint16_t, false);
  } else {
    if (flat) NVQ_Q(float, true);
    else NVQ_Q(float, false);
  }
#undef NVQ_Q
  return hipGetLastError();
}

hipError_t mxfp4_dequantize_launch(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, void* out, int out_bf16,
                                   hipStream_t s) {
  const int64_t units = n * k / (out_bf16 ? 8 : 4);
  const unsigned blocks = (unsigned)std::min<int64_t>((units + 256 * QU - 1) / (256 * QU), 1 << 20);
  if (out_bf16) hipLaunchKernelGGL((mx_dequantize_kernel<1>), dim3(blocks), dim3(256), 0, s, codes, scales, units, out);
  else hipLaunchKernelGGL((mx_dequantize_kernel<0>), dim3(blocks), dim3(256), 0, s, codes, scales, units, out);
  return hipGetLastError();
}

// Rows that are not quantized yet are quantized within the product's kernel up to this many.
constexpr int64_t kFusedRows = 16;
constexpr int64_t kFewRows = 64;

size_t mxfp4_gemm_workspace(int x_codes, int64_t n, int64_t k, int64_t m) {
  return x_codes || n <= kFusedRows ? 0 : (size_t)n * (k / 2) + (size_t)n * (k / 32);
}

hipError_t mxfp4_gemm_launch(const void* X, int x_codes, int x_bf16, const uint8_t* xscales, int64_t n, int64_t k, int64_t ldx,
                             const uint8_t* codes, const uint8_t* scales, int64_t m, void* Y, int out_bf16, int64_t ldy,
                             void* ws, hipStream_t s) {
#define NVQ_FEW_(XT, NG, CG, OUT)                                                                                              \
  hipLaunchKernelGGL((mx_few_kernel<XT, NG, CG, OUT>), dim3((unsigned)((m + 16 * CG - 1) / (16 * CG))), dim3(64 * FW), 0, s,   \
                     (const XT*)X, xscales, n, k, ldx, codes, scales, m, Y, ldy)
#define NVQ_FEW(XT, NG)                  \
  do {                                   \
    if (out_bf16) NVQ_FEW_(XT, NG, 1, 1); \
    else NVQ_FEW_(XT, NG, 1, 0);          \
    return hipGetLastError();            \
  } while (0)
  if (!x_codes && n <= kFusedRows) {
    if (x_bf16) NVQ_FEW(uint16_t, 1);
    NVQ_FEW(float, 1);
  }
  if (!x_codes) {
    uint8_t* xc = (uint8_t*)ws;
    uint8_t* xsc = xc + (size_t)n * (k / 2);
    const hipError_t e = mxfp4_quantize_launch(X, x_bf16, n, k, ldx, xc, xsc, s);
    if (e != hipSuccess) return e;
    X = xc;
    xscales = xsc;
  }
  if (n <= 16) NVQ_FEW(uint8_t, 1);
  if (n <= 32) NVQ_FEW(uint8_t, 2);
  if (n <= kFewRows) NVQ_FEW(uint8_t, 4);
#define NVQ_TILE(WM, WN, FA, FB)                                                                                              \
  do {                                                                                                                        \
    using TL = MxTile<WM, WN, FA, FB>;                                                                                        \
    const int64_t tiles = ((m + TL::kM - 1) / TL::kM) * ((n + TL::kN - 1) / TL::kN), blocks = (tiles + 7) / 8 * 8;            \
    if (blocks > kMaxThreads / TL::kThreads) return kTooManyTiles;                                                            \
    if (out_bf16)                                                                                                             \
      hipLaunchKernelGGL((mx_tile_kernel<WM, WN, FA, FB, 1>), dim3((unsigned)blocks), dim3(TL::kThreads), 0, s,               \
                         (const uint8_t*)X, xscales, n, k, codes, scales, m, Y, ldy);                                         \
    else                                                                                                                      \
      hipLaunchKernelGGL((mx_tile_kernel<WM, WN, FA, FB, 0>), dim3((unsigned)blocks), dim3(TL::kThreads), 0, s,               \
                         (const uint8_t*)X, xscales, n, k, codes, scales, m, Y, ldy);                                         \
    return hipGetLastError();                                                                                                 \
  } while (0)
  if (((m + 255) / 256) * ((n + 255) / 256) >= 192) NVQ_TILE(2, 4, 4, 2);
  NVQ_TILE(2, 2, 2, 2);
#undef NVQ_TILE
#undef NVQ_FEW
#undef NVQ_FEW_
}

}  // namespace nvq
