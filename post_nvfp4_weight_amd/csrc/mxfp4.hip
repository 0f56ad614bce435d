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
#include "quads.h"

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

// Units of eight values per thread.  us with 1 / 2 / 4 / 8: 8192 x 28672 fp32 there and
// back 423 / 401 / 401 / 425 (5.3 TB/s), 53 x 14336 bf16 with its product 12.3 / 12.6 / 13.5 / 14.9.
constexpr int QU = 2;

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

// A lane's block of 32 of a row, as loaded, and as codes under a scale byte: with
// the bits of mx_quantize_kernel, or as they are (T = uint8_t: codes).
template <typename T>
struct Block {
  Eight<T> x[4];
  __device__ __forceinline__ void load(const T* row, const uint8_t*, int64_t block) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j].load(row + 32 * block + 8 * j);
  }
  __device__ __forceinline__ void quantize(u32x4& w, uint32_t& byte) const {
    byte = scale_byte(max(max(x[0].top_exponent(), x[1].top_exponent()), max(x[2].top_exponent(), x[3].top_exponent())));
    const float s = scale_operand(byte);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = byte == 255 ? 0u : x[j].codes(s);
  }
};
template <>
struct Block<uint8_t> {
  u32x4 w;
  uint8_t s;
  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* scales, int64_t block) {
    w = *(const u32x4*)(row + 16 * block);
    s = scales[block];
  }
  __device__ __forceinline__ void quantize(u32x4& v, uint32_t& byte) const {
    v = w;
    byte = s;
  }
};

// Few rows: 16 output channels per workgroup, the eight waves each a part of k,
// all rows in NG groups of 4.
//   v_mfma_scale_f32_16x16x128_f8f6f4: a lane's operand is 32 codes under one
//   scale byte, which is one piece of quads.h, and one block.
// A wave takes chunks of 512 k in turn with the other waves.  Rows that are not
// quantized yet are quantized by the lane that multiplies them.  The waves'
// partial sums are added in wave order through LDS.
// Pieces past k: the rows' are zero codes under scale 1, the channels' are read
// at their row's start (a NaN there makes the channel NaN, as it does in its place).
constexpr int FW = 8;

// XT: uint8_t (codes, with scales), uint16_t (bf16) or float.
template <typename XT, int NG, int OUT_BF16>
__global__ __launch_bounds__(64 * FW, NG == 1 && sizeof(XT) < 4 ? 4 : 2) void mx_few_kernel(const XT* __restrict__ X, const uint8_t* __restrict__ xscales,
                                                            int64_t n, int64_t k, int64_t ldx,
                                                            const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t m,
                                                            void* __restrict__ Y, int64_t ldy) {
  constexpr bool kCodes = sizeof(XT) == 1;
  __shared__ float part[FW][4 * NG][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int piece = quad_piece(lane), col = quad_column(lane);
  const int64_t kb = k / 32, o0 = (int64_t)blockIdx.x * 16;
  codes += o0 * (k / 2);
  scales += o0 * kb;
  uint32_t row[4], srow[4];   // the lane's channels' first code and scale (channels past m repeat the last one and are not stored)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t o = (uint32_t)min((int64_t)(4 * col + i), m - 1 - o0);
    row[i] = o * (uint32_t)(k / 2);
    srow[i] = o * (uint32_t)kb;
  }
  const XT* xr[NG];
  const uint8_t* xs[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int64_t t = min((int64_t)(4 * g + col), n - 1);   // (likewise)
    xr[g] = X + (kCodes ? t * (k / 2) : t * ldx);
    xs[g] = kCodes ? xscales + t * kb : nullptr;
  }
  const int chunks = (int)((kb + 15) / 16), mine = chunks > wave ? (chunks - wave + FW - 1) / FW : 0;

  struct Chunk {
    u32x4 w[4];
    uint8_t s[4];
  };
  // (the same loads on every path, behind the last chunk the last one's)
  auto load_chunk = [&](int i, Chunk& x) __attribute__((always_inline)) {
    const int block = 16 * (wave + FW * min(i, mine - 1)) + piece;
    const uint32_t at = block < kb ? block : 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x.w[c] = *(const u32x4*)(codes + (row[c] + 16 * at));
      x.s[c] = scales[srow[c] + at];
    }
  };
  f32x4 acc[NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[g][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  Block<XT> x[NG];
  auto load_x = [&](int i) __attribute__((always_inline)) {
    const int block = 16 * (wave + FW * min(i, mine - 1)) + piece, at = block < kb ? block : 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) x[g].load(xr[g], xs[g], at);
  };
  if (mine > 0) {
    // Loads return in the order of their issue: a chunk's activations go out
    // ahead of the next chunk's weights.
    Chunk buf[2];
    load_chunk(0, buf[0]);
    auto consume = [&](int i, const Chunk& w, Chunk& next) __attribute__((always_inline)) {
      load_x(i);
      __builtin_amdgcn_sched_barrier(0);
      load_chunk(i + 1, next);
      __builtin_amdgcn_sched_barrier(0);
      const bool in = 16 * (wave + FW * i) + piece < kb;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        u32x4 xv;
        uint32_t xb;
        x[g].quantize(xv, xb);
#pragma unroll
        for (int e = 0; e < 4; ++e) xv[e] = in ? xv[e] : 0u;
        xb = in ? xb : 127u;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[g][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fragment(w.w[c]), fragment(xv), acc[g][c], 4, 4, 0, (int)w.s[c], 0,
                                                                       (int)xb);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    int i = 0;
    for (; i + 2 <= mine; i += 2) {
      consume(i, buf[0], buf[1]);
      consume(i + 1, buf[1], buf[0]);
    }
    if (i < mine) consume(i, buf[0], buf[1]);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) part[wave][4 * g + col][4 * (lane >> 4) + (lane & 3)] = quad_sum(acc[g], lane);
  __syncthreads();
  for (int i = tid; i < 64 * NG; i += 64 * FW) {
    const int r = i >> 4, o = i & 15;
    if (r >= n || o0 + o >= m) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < FW; ++w) v += part[w][r][o];
    const int64_t at = r * ldy + o0 + o;
    if (OUT_BF16) ((__bf16*)Y)[at] = (__bf16)v;
    else ((float*)Y)[at] = v;
  }
}

// Tiles of 32 FA WM output channels x 32 FB WN rows per workgroup of WM x WN
// waves, each 32 FA channels x 32 FB rows.
//   v_mfma_scale_f32_32x32x64_f8f6f4, A = 32 channels, B = 32 rows: lane
//   (r = l % 32, h = l / 32) holds one block of channel r and of row r.
//   k goes in stages of 256, four products deep: a row's 128 bytes of codes
//   and 8 scale bytes.  Product s takes block s for h = 0 and block 4 + s for
//   h = 1 (the order of k in the sum is free, as long as both operands agree),
//   so that the lane's four scale bytes are one word whose byte s the
//   instruction selects.
//   Codes are copied to LDS directly, R - 1 stages ahead into a ring of R, 16-byte
//   pieces swizzled by (row / 2) % 8: the 16 rows that are read at once then touch
//   all 64 banks.  Scales (which may start at any byte) go through registers, for
//   GS stages at a time, one such group ahead.
// BF16: both operands bf16 (the gradient on weights that were expanded before):
// a row's 128 bytes are 64 k, a piece 8 k of v_mfma_f32_32x32x16_bf16; no scales.
template <int WM, int WN, int FA, int FB, int R, int GS, bool BF16 = false>
struct MxTile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kM = 32 * FA * WM, kN = 32 * FB * WN, kAll = kM + kN;
  static constexpr int kWLoads = kM / 8 / kWaves, kXLoads = kN / 8 / kWaves, kLoads = kWLoads + kXLoads;
  static constexpr int kBuf = kAll * 128, kSBuf = BF16 ? 0 : kAll * 8;   // codes and scales of a stage; the channels' first
  static constexpr int kRing = R * kBuf + 2 * GS * kSBuf, kOut = kWaves * 32 * (32 * FA * 4 + 16), kLds = kRing > kOut ? kRing : kOut;
  static_assert(kM % (8 * kWaves) == 0 && kN % (8 * kWaves) == 0 && kWaves % 2 == 0, "whole copies per wave");
  static_assert(kAll <= kThreads && (GS == 2 || GS == 4), "a thread per row of scales");
};

// The workgroup's tile of TM channels x TN rows: its first channel and row, false
// if there is none.  The tiles are dealt to the 8 XCDs (blockIdx.x mod 8) in
// contiguous runs of an order that walks 8 row tiles, then the next channel tile, so
// that the tiles that run together in an XCD share operands in its L2.
__device__ __forceinline__ bool tile_of(int64_t m, int64_t n, int tm, int tn, int64_t& o0, int64_t& t0) {
  const uint32_t ntm = (uint32_t)((m + tm - 1) / tm), ntn = (uint32_t)((n + tn - 1) / tn);
  const uint64_t all = (uint64_t)ntm * ntn, per = (all + 7) / 8;
  const uint64_t id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || id >= all) return false;
  const uint64_t panel = id / (8ull * ntm), in_panel = id - panel * 8 * ntm;
  const uint32_t high = (uint32_t)min((uint64_t)8, ntn - panel * 8);
  o0 = (int64_t)(in_panel / high) * tm;
  t0 = (int64_t)(panel * 8 + in_panel % high) * tn;
  return true;
}

__device__ __forceinline__ constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
__device__ __forceinline__ constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// NL copies of 1024 bytes to LDS (16 per lane), from `src` + off[q] + add; offsets at or past the bound bring zeros.
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

// One stage, from wb, xb (codes) and sw, sx (scales); the buffers that the copies
// in flight fill are others, which the restrict qualifiers state, so that reads
// need not wait for them.
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
template <int S, int FA, int FB, bool BF16>
__device__ __forceinline__ void multiply(const u32x4 (&a)[FA], const u32x4 (&b)[FB], const uint32_t (&sa)[FA], const uint32_t (&sb)[FB],
                                         f32x16 (&acc)[FA][FB]) {
  if constexpr (!BF16) {
    mx_product<S, FA, FB>(a, b, sa, sb, acc);
  } else {
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a[i]), __builtin_bit_cast(bf16x8, b[j]), acc[i][j],
                                                            0, 0, 0);
  }
}
template <int FA, int FB, bool BF16>
__device__ __forceinline__ void mx_stage(const char* __restrict__ wb, const char* __restrict__ xb, const char* __restrict__ sw,
                                         const char* __restrict__ sx, const int (&rd)[4], f32x16 (&acc)[FA][FB]) {
  uint32_t sa[FA], sb[FB];
  if (!BF16) {
#pragma unroll
    for (int i = 0; i < FA; ++i) sa[i] = *(const uint32_t*)(sw + i * 256);
#pragma unroll
    for (int j = 0; j < FB; ++j) sb[j] = *(const uint32_t*)(sx + j * 256);
  }
  u32x4 a[2][FA], b[2][FB];
  auto read = [&](int s, int p) {
#pragma unroll
    for (int i = 0; i < FA; ++i) a[p][i] = *(const u32x4*)(wb + i * 4096 + rd[s]);
#pragma unroll
    for (int j = 0; j < FB; ++j) b[p][j] = *(const u32x4*)(xb + j * 4096 + rd[s]);
  };
  read(0, 0);
  read(1, 1);
  multiply<0, FA, FB, BF16>(a[0], b[0], sa, sb, acc);
  read(2, 0);
  multiply<1, FA, FB, BF16>(a[1], b[1], sa, sb, acc);
  read(3, 1);
  multiply<2, FA, FB, BF16>(a[0], b[0], sa, sb, acc);
  multiply<3, FA, FB, BF16>(a[1], b[1], sa, sb, acc);
}

// A row's 8 GS scale bytes of a group, `left` blocks to the end of k (zeros stand
// for what is behind it: its codes are zeros too).
template <int GS>
__device__ __forceinline__ void group_scales(const uint8_t* __restrict__ p, int64_t left, u32x4 (&v)[GS / 2]) {
  if (left >= 8 * GS) {
#pragma unroll
    for (int i = 0; i < GS / 2; ++i) v[i] = *(const u32x4_any*)(p + 16 * i);
    return;
  }
#pragma unroll
  for (int i = 0; i < GS / 2; ++i)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t x = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (16 * i + 4 * w + b < left) x |= (uint32_t)p[16 * i + 4 * w + b] << (8 * b);
      v[i][w] = x;
    }
}

// kbytes: bytes of a row that are multiplied; xs, ws (BF16): from one row to the next.
template <int WM, int WN, int FA, int FB, int R, int GS, bool BF16, int OUT_BF16>
__global__ __launch_bounds__(64 * WM * WN) void mx_tile_kernel(const uint8_t* __restrict__ xcodes, int64_t xs,
                                                               const uint8_t* __restrict__ xscales, int64_t n, int64_t kbytes,
                                                               const uint8_t* __restrict__ codes, int64_t ws,
                                                               const uint8_t* __restrict__ scales, int64_t m,
                                                               void* __restrict__ Y, int64_t ldy) {
  using TL = MxTile<WM, WN, FA, FB, R, GS, BF16>;
  constexpr int NW = TL::kWaves;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, wm = wave / WN, wn = wave % WN;
  int64_t o0, t0;
  if (!tile_of(m, n, TL::kM, TL::kN, o0, t0)) return;

  const int64_t kb = BF16 ? 0 : kbytes / 16, xstride = BF16 ? xs : kbytes, wstride = BF16 ? ws : kbytes;
  const int64_t om = min((int64_t)TL::kM, m - o0), tn = min((int64_t)TL::kN, n - t0);   // channels and rows that are there
  codes += o0 * wstride;
  xcodes += t0 * xstride;
  if (!BF16) {
    scales += o0 * kb;
    xscales += t0 * kb;
  }
  const uint32_t wbound = (uint32_t)((om - 1) * wstride + kbytes), xbound = (uint32_t)((tn - 1) * xstride + kbytes);   // (below 0xC0000000: checked on the host)

  // Copy q of a stage: rows 8 (NW q + wave) + lane / 8, piece (lane % 8) ^ (row / 2) % 8.
  const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
  uint32_t woff[TL::kWLoads], xoff[TL::kXLoads];
#pragma unroll
  for (int q = 0; q < TL::kWLoads; ++q) {
    const int row = 8 * (NW * q + wave) + (lane >> 3);
    woff[q] = row < om ? (uint32_t)(row * wstride) + 16 * piece : 0xC0000000u;
  }
#pragma unroll
  for (int q = 0; q < TL::kXLoads; ++q) {
    const int row = 8 * (NW * q + wave) + (lane >> 3);
    xoff[q] = row < tn ? (uint32_t)(row * xstride) + 16 * piece : 0xC0000000u;
  }
  const int nst = (int)((kbytes + 127) / 128);
  char* const ring = smem;
  char* const sring = smem + R * TL::kBuf;   // [group % 2][stage in it][row][8]
  auto copy = [&](int st, int slot) {   // (past the last stage: zeros that nothing is fetched for)
    const bool in = (int64_t)st * 128 + 16 * piece < kbytes;
    char* to = ring + slot * TL::kBuf + wave * 1024;
    copy_rows<TL::kWLoads, NW * 1024>(to, codes, wbound, woff, (uint32_t)st * 128, in);
    copy_rows<TL::kXLoads, NW * 1024>(to + TL::kM * 128, xcodes, xbound, xoff, (uint32_t)st * 128, in);
  };
  u32x4 sreg[GS / 2];
  const uint8_t* const srow =
      BF16 ? nullptr : tid < TL::kM ? scales + min((int64_t)tid, om - 1) * kb : xscales + min((int64_t)min(tid, TL::kAll - 1) - TL::kM, tn - 1) * kb;
  auto load_scales = [&](int grp) { group_scales<GS>(srow + (int64_t)grp * 8 * GS, kb - (int64_t)grp * 8 * GS, sreg); };
  auto store_scales = [&](int grp) {
    if (tid < TL::kAll)
#pragma unroll
      for (int s = 0; s < GS; ++s)
        *(u32x2*)(sring + ((grp & 1) * GS + s) * TL::kSBuf + tid * 8) = u32x2{sreg[s / 2][2 * (s & 1)], sreg[s / 2][2 * (s & 1) + 1]};
  };
  int rd[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) rd[s] = r * 128 + (((4 * h + s) ^ ((r >> 1) & 7)) * 16);
  const int wrow = wm * 32 * FA, xrow = TL::kM + wn * 32 * FB;
  // A wave without a channel or a row only copies.  In the large tile the branch also
  // keeps the compiler from moving reads of the next stage up, for which it spilled
  // (578 us with it, 682 without, at 8192 rows x 28672 x 4096); the small ones are a
  // twentieth faster without (8.3 us against 8.9 at 1537 x 1003 x 1056).
  const bool live = FA * FB < 8 || (wrow < om && wn * 32 * FB < tn);

  f32x16 acc[FA][FB];
#pragma unroll
  for (int i = 0; i < FA; ++i)
#pragma unroll
    for (int j = 0; j < FB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  if (!BF16) load_scales(0);
#pragma unroll
  for (int s = 0; s < R - 1; ++s) copy(s, s);
  if (!BF16) store_scales(0);
  int slot = 0;
  for (int st = 0; st < nst; st += GS) {
    const int grp = st / GS;
#pragma unroll
    for (int s = 0; s < GS; ++s) {
      if (s > 0 && st + s >= nst) break;
      // Stage st + s is there once at most R - 2 stages of copies are in flight,
      // and every wave is through with the stage before, whose place is filled next.
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((R - 2) * TL::kLoads));
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      if (!BF16 && s == 0 && st + GS < nst) load_scales(grp + 1);
      copy(st + s + R - 1, slot == 0 ? R - 1 : slot - 1);
      __builtin_amdgcn_sched_barrier(0);
      const char* b = ring + slot * TL::kBuf;
      const char* sc = sring + ((grp & 1) * GS + s) * TL::kSBuf + 4 * h;
      if (live) mx_stage<FA, FB, BF16>(b + wrow * 128, b + xrow * 128, sc + (wrow + r) * 8, sc + (xrow + r) * 8, rd, acc);
      slot = slot + 1 == R ? 0 : slot + 1;
      if (!BF16 && s == GS - 1) store_scales(grp + 1);
    }
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
  asm volatile("s_barrier" ::: "memory");

  // Accumulator: lane l, register e -> channel 8 (e / 4) + 4 h + e % 4, row r.
  constexpr int ES = OUT_BF16 ? 2 : 4;
  // 32 rows at a time go through LDS of the wave's own, so that a row's
  // channels leave in 16-byte pieces side by side.
  constexpr int ROW = 32 * FA * ES + 16, PR = 32 * FA * ES / 16;
  static_assert(NW * 32 * ROW <= TL::kLds, "output staging");
  char* stage = smem + wave * 32 * ROW;
  const int64_t oc = o0 + wrow, tr = t0 + wn * 32 * FB;
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
      const int64_t t = tr + 32 * j + row, o = oc + pc * (16 / ES);
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

// W [m x k] to bf16 W^T [k x m]: 64 m x 64 k per workgroup, through LDS.
// Thread (row tid / 4, quarter tid % 4) expands 16 codes of a row under one scale
// and writes them down a column of LDS; 16 m of a column leave as two vectors.
__global__ __launch_bounds__(256) void mx_transpose_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                           int64_t m, int64_t k, uint16_t* __restrict__ out) {
  constexpr int LD = 64 + 8;   // (rows apart by 36 banks)
  __shared__ __attribute__((aligned(16))) uint16_t t[64][LD];
  const int64_t m0 = (int64_t)blockIdx.x * 64, k0 = (int64_t)blockIdx.y * 64;
  const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
  if (m0 + row < m && k0 + 16 * part < k) {
    const u32x2 w = *(const u32x2*)(codes + (m0 + row) * (k / 2) + k0 / 2 + 8 * part);
    const float s = scale_value(scales[(m0 + row) * (k / 32) + k0 / 32 + part / 2]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w[i];
      const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 3)};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __bf16 b = (__bf16)((e & 1 ? p[e / 2].y : p[e / 2].x) * s);
        t[16 * part + 8 * i + e][row] = __builtin_bit_cast(uint16_t, b);
      }
    }
  }
  __syncthreads();
  if (k0 + row < k) {   // column `row` of the tile, m 16 part ..
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t mm = m0 + 16 * part + 8 * i;   // (m is a multiple of 8)
      if (mm < m) *(u32x4*)(out + (k0 + row) * m + mm) = *(const u32x4*)&t[row][16 * part + 8 * i];
    }
  }
}

// The gradient of one or two rows: dX[t][c] = sum_m dY[t][m] W[m][c], bound by reading W.
// A lane holds 16 columns (8 bytes of codes under one scale), a wave 1024, and
// adds row after row of W, expanded in fp32, to its sums for NR rows of dX;
// the 8 waves of a workgroup take the rows of its part of m in turn, DB at a time,
// and add their sums in wave order.  The parts' sums go to `out` [part][row][k] and
// are added in their order by the second kernel, or with one part are the result.
// us with this / on the matrix cores' tiles of 64 rows, which want W transposed: one
// row x 4096 x 4096 8.5 / 12.9, 28672 x 4096 21 / 31, 1000 x 1056 6.8 / 8.9; two rows 9.9 /
// 13.5, 26 / 32; four, for which each code is expanded once too, 13.5 / 13.4, 36 / 33.
constexpr int DB = 8, kDxPart = 1024;   // rows of W at a time; most of a part

template <int NR, int OUT>   // OUT: 0 fp32, 1 bf16
__global__ __launch_bounds__(512) void mx_dx_few_kernel(const uint16_t* __restrict__ dY, int64_t m, int64_t lddy,
                                                        const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t k,
                                                        int64_t mper, void* __restrict__ out, int64_t ldo) {
  __shared__ float dy[NR][kDxPart];
  __shared__ __attribute__((aligned(16))) float part[8][1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t c0 = (int64_t)blockIdx.x * 1024 + 16 * lane, m0 = (int64_t)blockIdx.y * mper;
  const int rows = (int)min(mper, m - m0);
  const bool in = c0 < k;
  const uint8_t* cp = codes + m0 * (k / 2) + (in ? c0 / 2 : 0);
  const uint8_t* sp = scales + m0 * (k / 32) + (in ? c0 / 32 : 0);
#pragma unroll
  for (int t = 0; t < NR; ++t)
    for (int r = tid; r < rows; r += 512) dy[t][r] = __uint_as_float((uint32_t)dY[t * lddy + m0 + r] << 16);
  float acc[NR][16];
#pragma unroll
  for (int t = 0; t < NR; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[t][e] = 0.0f;
  u32x2 w[DB];
  uint8_t s[DB];
  auto load = [&](int r0) __attribute__((always_inline)) {   // (rows past the part repeat its last one, under scale 0)
#pragma unroll
    for (int j = 0; j < DB; ++j) {
      const int64_t r = min(r0 + 8 * j, rows - 1);
      w[j] = *(const u32x2*)(cp + r * (k / 2));
      s[j] = sp[r * (k / 32)];
    }
  };
  load(wave);
  __syncthreads();
  for (int r0 = wave; r0 < rows; r0 += 8 * DB) {
#pragma unroll
    for (int j = 0; j < DB; ++j) {
      const int r = r0 + 8 * j;
      const float sv = r < rows ? scale_value(s[j]) : 0.0f;
      float d[NR];
#pragma unroll
      for (int t = 0; t < NR; ++t) d[t] = r < rows ? dy[t][min(r, rows - 1)] : 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v = w[j][i];
        const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 3)};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = (e & 1 ? p[e / 2].y : p[e / 2].x) * sv;
#pragma unroll
          for (int t = 0; t < NR; ++t) acc[t][8 * i + e] = fmaf(x, d[t], acc[t][8 * i + e]);
        }
      }
    }
    if (r0 + 8 * DB < rows) load(r0 + 8 * DB);
  }
#pragma unroll
  for (int t = 0; t < NR; ++t) {
    // (piece e of a lane at 256 e + 4 lane: neighbouring lanes side by side)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *(f32x4*)&part[wave][256 * e + 4 * lane] = f32x4{acc[t][4 * e], acc[t][4 * e + 1], acc[t][4 * e + 2], acc[t][4 * e + 3]};
    __syncthreads();
    for (int i = tid; i < 1024; i += 512) {
      const int l = (i & 255) >> 2;
      const int64_t c = (int64_t)blockIdx.x * 1024 + 16 * l + 4 * (i >> 8) + (i & 3);
      float v = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += part[q][i];
      if (c < k) {
        const int64_t at = ((int64_t)blockIdx.y * NR + t) * ldo + c;
        if (OUT) ((__bf16*)out)[at] = (__bf16)v;
        else ((float*)out)[at] = v;
      }
    }
    __syncthreads();
  }
}

// The parts' sums: 32 times four columns per workgroup, eight threads' shares of the parts each.
template <int OUT>
__global__ __launch_bounds__(256) void mx_dx_parts_kernel(const float* __restrict__ parts, int64_t n, int64_t k, int count,
                                                          void* __restrict__ dX, int64_t lddx) {
  __shared__ __attribute__((aligned(16))) f32x4 sums[8][32];
  const int q = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + q, total = n * k;
  f32x4 v{0.f, 0.f, 0.f, 0.f};
  if (4 * i < total) {
#pragma unroll 8
    for (int p = g; p < count; p += 8) {
      const f32x4 x = *(const f32x4*)(parts + p * total + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
  }
  sums[g][q] = v;
  __syncthreads();
  if (g != 0 || 4 * i >= total) return;
#pragma unroll
  for (int p = 1; p < 8; ++p) {
    const f32x4 x = sums[p][q];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += x[e];
  }
  const int64_t row = 4 * i / k, at = row * lddx + 4 * i - row * k;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (OUT) ((__bf16*)dX)[at + e] = (__bf16)v[e];
    else ((float*)dX)[at + e] = v[e];
  }
}

// Tiles of 32 output channels x 32 FB rows for sizes that make few tiles: the
// four waves of a workgroup share k instead, in pairs of stages of 256 in turn, in
// LDS of their own, so that none waits for another (with the waves at the four
// products of one stage and a barrier for each, 53 rows x 4096 x 14336 took 13.4 us
// beside the quantization, with this 11).
//   Operands as above.  A wave copies a stage's rows itself, one stage ahead.  A
//   pair's 16 scale bytes per row are loaded into the row's two lanes, 8 each, and
//   exchanged between the wave's halves.  (Loaded word by word in their place they
//   took the address unit as long as the codes.)
// The rest of k behind the last pair goes to the first waves, byte by byte where
// scales are concerned.  The waves' sums are added in wave order through LDS.
constexpr int TW = 4;
template <int FB>
struct MxThin {
  static constexpr int kRows = 32 + 32 * FB, kBuf = kRows * 128, kLoads = kRows / 8;
  static constexpr int kLd = 36, kRing = TW * 2 * kBuf, kSums = TW * 32 * FB * kLd * 4;
  static constexpr int kLds = kRing > kSums ? kRing : kSums;
};

template <int FB>
__device__ __forceinline__ void thin_stage(const char* __restrict__ b, const int (&rd)[4], const uint32_t (&s)[1 + FB],
                                           f32x16 (&acc)[1][FB]) {
  u32x4 w[4][1], x[4][FB];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i][0] = *(const u32x4*)(b + rd[i]);
#pragma unroll
    for (int j = 0; j < FB; ++j) x[i][j] = *(const u32x4*)(b + 4096 * (1 + j) + rd[i]);
  }
  uint32_t sw[1] = {s[0]}, sx[FB];
#pragma unroll
  for (int j = 0; j < FB; ++j) sx[j] = s[1 + j];
  __builtin_amdgcn_sched_barrier(0);   // (all reads go out before the first product)
  mx_product<0, 1, FB>(w[0], x[0], sw, sx, acc);
  mx_product<1, 1, FB>(w[1], x[1], sw, sx, acc);
  mx_product<2, 1, FB>(w[2], x[2], sw, sx, acc);
  mx_product<3, 1, FB>(w[3], x[3], sw, sx, acc);
}

template <int FB, int OUT_BF16>
__global__ __launch_bounds__(64 * TW) void mx_thin_kernel(const uint8_t* __restrict__ xcodes, const uint8_t* __restrict__ xscales,
                                                          int64_t n, int64_t k, const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, int64_t m, void* __restrict__ Y,
                                                          int64_t ldy) {
  using TL = MxThin<FB>;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  int64_t o0, t0;
  if (!tile_of(m, n, 32, 32 * FB, o0, t0)) return;
  const int64_t kh = k / 2, kb = k / 32;
  const int64_t om = min((int64_t)32, m - o0), tn = min((int64_t)32 * FB, n - t0);
  codes += o0 * kh;
  scales += o0 * kb;
  xcodes += t0 * kh;
  xscales += t0 * kb;
  const uint32_t wbound = (uint32_t)(om * kh), xbound = (uint32_t)(tn * kh);

  // Copy q: rows 8 q + lane / 8 of the stage's channels (q < 4), then of its rows;
  // piece (lane % 8) ^ (row / 2) % 8, which depends on q % 2.
  constexpr uint32_t kPast = 0x20000000u;   // past every bound (below 2^28: checked on the host), also with k's offsets added; two of them too
  int piece[2];
  uint32_t off[TL::kLoads];
#pragma unroll
  for (int p = 0; p < 2; ++p) piece[p] = (lane & 7) ^ (4 * p + (lane >> 4));
#pragma unroll
  for (int q = 0; q < TL::kLoads; ++q) {
    const int row = 8 * (q < 4 ? q : q - 4) + (lane >> 3);
    off[q] = row < (q < 4 ? om : tn) ? (uint32_t)(row * kh) + 16 * piece[q & 1] : kPast;
  }
  char* const ring = smem + wave * 2 * TL::kBuf;
  auto copy = [&](int slot, uint32_t add, int64_t left) __attribute__((always_inline)) {   // left: bytes of a row from there on
#if __HIP_DEVICE_COMPILE__
    const __amdgpu_buffer_rsrc_t wrs = __builtin_amdgcn_make_buffer_rsrc((void*)codes, (short)0, wbound, 0x00020000);
    const __amdgpu_buffer_rsrc_t xrs = __builtin_amdgcn_make_buffer_rsrc((void*)xcodes, (short)0, xbound, 0x00020000);
#pragma unroll
    for (int q = 0; q < TL::kLoads; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(q < 4 ? wrs : xrs, (__attribute__((address_space(3))) void*)(ring + slot * TL::kBuf + q * 1024),
                                               16, left >= 128 || 16 * piece[q & 1] < left ? off[q] + add : kPast, 0, 0, 0);
#endif
  };
  uint32_t soff[1 + FB];   // scales of channel r, of rows r, 32 + r, .. (past the last it)
  soff[0] = (uint32_t)(min(r, (int)om - 1) * kb);
#pragma unroll
  for (int j = 0; j < FB; ++j) soff[1 + j] = (uint32_t)(min(32 * j + r, (int)tn - 1) * kb);

  int rd[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) rd[s] = r * 128 + (((4 * h + s) ^ ((r >> 1) & 7)) * 16);
  f32x16 acc[1][FB];
#pragma unroll
  for (int j = 0; j < FB; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][j][e] = 0.0f;

  const int pairs = (int)(k / 512), mine = pairs > wave ? (pairs - wave + TW - 1) / TW : 0;   // the wave's i-th is wave + TW i
  if (mine > 0) {
    u32x2 raw[1 + FB];
    auto load_scales = [&](int i) __attribute__((always_inline)) {   // (behind the last pair the last one's)
      const int at = 16 * (wave + TW * min(i, mine - 1)) + 8 * h;
#pragma unroll
      for (int j = 0; j <= FB; ++j) raw[j] = *(const u32x2_any*)((j ? xscales : scales) + (soff[j] + at));
    };
    auto copy_stage = [&](int i, int p) __attribute__((always_inline)) {
      copy(p, i < mine ? (uint32_t)(wave + TW * i) * 256 + 128 * p : kPast, 128);
    };
    load_scales(0);
    copy_stage(0, 0);
    __builtin_amdgcn_sched_barrier(0);
    for (int i = 0; i < mine; ++i) {
      copy_stage(i, 1);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(TL::kLoads));   // the first stage and the pair's scales are there
      __builtin_amdgcn_sched_barrier(0);
      // Lane (r, h) holds the words of stage h: h = 0's of its row, then h = 1's.
      uint32_t s0[1 + FB], s1[1 + FB];
#pragma unroll
      for (int j = 0; j <= FB; ++j) {
        const auto v = __builtin_amdgcn_permlane32_swap(raw[j][0], raw[j][1], false, false);
        s0[j] = v[0];
        s1[j] = v[1];
      }
      thin_stage<FB>(ring, rd, s0, acc);
      __builtin_amdgcn_sched_barrier(0);
      load_scales(i + 1);
      copy_stage(i + 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(TL::kLoads + 1 + FB));   // the second stage
      __builtin_amdgcn_sched_barrier(0);
      thin_stage<FB>(ring + TL::kBuf, rd, s1, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const int st = 2 * pairs + wave;   // of the rest, at most two stages
  if ((int64_t)st * 256 < k) {
    copy(0, (uint32_t)st * 128, kh - (int64_t)st * 128);
    uint32_t s[1 + FB];
    const int64_t b0 = (int64_t)st * 8 + 4 * h;
#pragma unroll
    for (int j = 0; j <= FB; ++j) {
      s[j] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b0 + b < kb) s[j] |= (uint32_t)(j ? xscales : scales)[soff[j] + (uint32_t)b0 + b] << (8 * b);
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_sched_barrier(0);
    thin_stage<FB>(ring, rd, s, acc);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
  asm volatile("s_barrier" ::: "memory");

  // Accumulator: lane l, register e -> channel 8 (e / 4) + 4 h + e % 4, row r.
  float* sum = (float*)smem;   // [wave][row][channel]
#pragma unroll
  for (int j = 0; j < FB; ++j)
#pragma unroll
    for (int e4 = 0; e4 < 4; ++e4)
      *(f32x4*)(sum + (wave * 32 * FB + 32 * j + r) * TL::kLd + 8 * e4 + 4 * h) =
          f32x4{acc[0][j][4 * e4], acc[0][j][4 * e4 + 1], acc[0][j][4 * e4 + 2], acc[0][j][4 * e4 + 3]};
  __syncthreads();
  for (int e = tid; e < 1024 * FB; e += 64 * TW) {
    const int row = e >> 5, ch = e & 31;
    if (row >= tn || ch >= om) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < TW; ++w) v += sum[(w * 32 * FB + row) * TL::kLd + ch];
    const int64_t at = (t0 + row) * ldy + o0 + ch;
    if (OUT_BF16) ((__bf16*)Y)[at] = (__bf16)v;
    else ((float*)Y)[at] = v;
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

// Whether the few-row kernel takes a product: it saves the launch that quantizes
// the rows (about 4 us), but every 16 channels quantize them again, and its columns
// serve 4 rows each.  us, few-row kernel / quantization and tiles, by rows and m x k:
//   bf16   4 rows: 4096 x 4096 4.3 / 8.0, 28672 x 4096 15.2 / 17.2, 8192 x 28672 32 / 37;  8 rows: 4096 x 14336 10.6 / 11.6,
//          16384 x 4096 15.3 / 12.6;  16 rows: 4096 x 4096 7.0 / 8.4, 8192 x 4096 11.9 / 10.1
//   MXFP4  4 rows: 4096 x 14336 7.4 / 8.0, 28672 x 4096 12.9 / 12.9;  8 rows: 4096 x 14336 7.9 / 8.2, 28672 x 4096 13.5 / 12.8;
//          16 rows: 4096 x 4096 4.3 / 5.1, 8192 x 4096 7.6 / 6.9
//   fp32   4 rows: 4096 x 4096 5.6 / 7.6, 8192 x 4096 9.6 / 9.4;  8 rows: 4096 x 4096 7.8 / 7.7
bool few_rows(int x_codes, int x_bf16, int64_t n, int64_t k, int64_t m) {
  const int64_t size = m * k;
  if (!x_codes && !x_bf16) return n <= 4 && size <= 1 << 24;
  if (n <= 4) return !x_codes || size < 1 << 26;
  return n <= 8 ? size < 1 << 26 : n <= 16 && size <= 1 << 24;
}

size_t mxfp4_gemm_workspace(int x_codes, int x_bf16, int64_t n, int64_t k, int64_t m) {
  return x_codes || few_rows(x_codes, x_bf16, n, k, m) ? 0 : (size_t)n * (k / 2) + (size_t)n * (k / 32);
}

hipError_t mxfp4_gemm_launch(const void* X, int x_codes, int x_bf16, const uint8_t* xscales, int64_t n, int64_t k, int64_t ldx,
                             const uint8_t* codes, const uint8_t* scales, int64_t m, void* Y, int out_bf16, int64_t ldy,
                             void* ws, hipStream_t s) {
#define NVQ_FEW_(XT, NG, OUT)                                                                                                   \
  hipLaunchKernelGGL((mx_few_kernel<XT, NG, OUT>), dim3((unsigned)((m + 15) / 16)), dim3(64 * FW), 0, s, (const XT*)X, xscales, \
                     n, k, ldx, codes, scales, m, Y, ldy)
#define NVQ_FEW(XT, NG)                    \
  do {                                     \
    if (out_bf16) NVQ_FEW_(XT, NG, 1);     \
    else NVQ_FEW_(XT, NG, 0);              \
    return hipGetLastError();              \
  } while (0)
#define NVQ_FEW_BY(XT)            \
  do {                            \
    if (n <= 4) NVQ_FEW(XT, 1);   \
    if (n <= 8) NVQ_FEW(XT, 2);   \
    NVQ_FEW(XT, 4);               \
  } while (0)
  if (few_rows(x_codes, x_bf16, n, k, m)) {
    if (x_codes) NVQ_FEW_BY(uint8_t);
    if (x_bf16) NVQ_FEW_BY(uint16_t);
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
#define NVQ_GRID(TM, TN, THREADS)                                                          \
  const int64_t blocks = (((m + (TM)-1) / (TM)) * ((n + (TN)-1) / (TN)) + 7) / 8 * 8;     \
  if (blocks > kMaxThreads / (THREADS)) return kTooManyTiles;
#define NVQ_TILE_(OUT, ...)                                                                                                    \
  hipLaunchKernelGGL((mx_tile_kernel<__VA_ARGS__, false, OUT>), dim3((unsigned)blocks), dim3(TL::kThreads), 0, s, (const uint8_t*)X, \
                     k / 2, xscales, n, k / 2, codes, k / 2, scales, m, Y, ldy)
#define NVQ_TILE(...)                            \
  do {                                           \
    using TL = MxTile<__VA_ARGS__>;              \
    NVQ_GRID(TL::kM, TL::kN, TL::kThreads)       \
    if (out_bf16) NVQ_TILE_(1, __VA_ARGS__);     \
    else NVQ_TILE_(0, __VA_ARGS__);              \
    return hipGetLastError();                    \
  } while (0)
#define NVQ_THIN_(FB, OUT)                                                                                                   \
  hipLaunchKernelGGL((mx_thin_kernel<FB, OUT>), dim3((unsigned)blocks), dim3(64 * TW), 0, s, (const uint8_t*)X, xscales, n, k, codes, \
                     scales, m, Y, ldy)
#define NVQ_THIN(FB)                     \
  do {                                   \
    NVQ_GRID(32, 32 * FB, 64 * TW)       \
    if (out_bf16) NVQ_THIN_(FB, 1);      \
    else NVQ_THIN_(FB, 0);               \
    return hipGetLastError();            \
  } while (0)
  // The largest tile that the rows fill more than half of and that gives three
  // quarters of the device's 256 CUs a tile.  us with 32 x 32 / 32 x 64 / 64 x 64 /
  // 128 x 64 / 128 x 128 / 256 x 256 (channels x rows), quantization included: 64 rows x
  // 4096 x 4096 9.1 / 11.1 / 11.7 / 13.5 / 18.3 / -; 128 rows 11.9 / 11.1 / 11.9 / 14.0 /
  // 18.4 / -; 256 rows 18.8 / 15.1 / 12.8 / 14.8 / 18.9 / -; 512 rows - / 24 / 20 / 16.4 /
  // 20.1 / -; 1024 rows - / - / 35 / 28 / 22.8 / 24; 64 rows x 28672 x 4096 28 / 24 / 21 / 18 /
  // 24 / -; 512 rows - / - / 110 / 82 / 58 / 49; 8192 rows - / - / - / 1075 / 656 / 572.
  auto tiles = [&](int64_t tm, int64_t tn) { return ((m + tm - 1) / tm) * ((n + tn - 1) / tn); };
  constexpr int64_t kEnough = 192;
  if (n > 128 && tiles(256, 256) >= kEnough) NVQ_TILE(2, 4, 4, 2, 2, 2);
  if (n > 64 && tiles(128, 128) >= kEnough) NVQ_TILE(2, 2, 2, 2, 2, 4);
  if (tiles(128, 64) >= kEnough) NVQ_TILE(2, 2, 2, 1, 4, 4);
  if (tiles(64, 64) >= kEnough) NVQ_TILE(2, 2, 1, 1, 6, 4);
  if (n > 32 && tiles(32, 64) >= kEnough) NVQ_THIN(2);
  NVQ_THIN(1);
#undef NVQ_THIN
#undef NVQ_THIN_
#undef NVQ_TILE
#undef NVQ_TILE_
#undef NVQ_GRID
#undef NVQ_FEW_BY
#undef NVQ_FEW
#undef NVQ_FEW_
}

// One or two rows of the gradient: parts of m of at least 64 and at most kDxPart, for
// 256 workgroups where m allows it.  (us with 256 / 512 / 1024, one row x 28672 x 4096
// 21.0 / 23.6 / 24.2, 4096 x 14336 15.0 / 15.7 / 15.6.)
namespace {
int64_t dx_few_part(int64_t m, int64_t k) {
  const int64_t parts = std::max<int64_t>(1, 256 / ((k + 1023) / 1024));
  return std::min<int64_t>(kDxPart, std::max<int64_t>(64, ((m + parts - 1) / parts + 63) / 64 * 64));
}
}  // namespace
bool mxfp4_gemm_dx_few(int64_t n) { return n <= 2; }
size_t mxfp4_gemm_dx_few_workspace(int64_t n, int64_t m, int64_t k) {
  const int64_t mper = dx_few_part(m, k), parts = (m + mper - 1) / mper;
  return parts > 1 ? (size_t)(parts * n * k * 4) : 0;
}
hipError_t mxfp4_gemm_dx_few_launch(const uint16_t* dY, int64_t n, int64_t m, int64_t lddy, const uint8_t* codes, const uint8_t* scales,
                                    int64_t k, void* dX, int out_bf16, int64_t lddx, void* ws, hipStream_t s) {
  const int64_t mper = dx_few_part(m, k), parts = (m + mper - 1) / mper;
  const bool one = parts == 1;
  const dim3 grid((unsigned)((k + 1023) / 1024), (unsigned)parts);   // (at most 3907 each)
#define NVQ_DX_(NR, OUT)                                                                                                         \
  hipLaunchKernelGGL((mx_dx_few_kernel<NR, OUT>), grid, dim3(512), 0, s, dY, m, lddy, codes, scales, k, mper, one ? dX : ws, \
                     one ? lddx : k)
#define NVQ_DX(NR)                           \
  do {                                       \
    if (one && out_bf16) NVQ_DX_(NR, 1);     \
    else NVQ_DX_(NR, 0);                     \
  } while (0)
  if (n == 1) NVQ_DX(1);
  else NVQ_DX(2);
#undef NVQ_DX
#undef NVQ_DX_
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || one) return e;
  const dim3 sums((unsigned)((n * k / 4 + 31) / 32));
  if (out_bf16) hipLaunchKernelGGL((mx_dx_parts_kernel<1>), sums, dim3(256), 0, s, (const float*)ws, n, k, (int)parts, dX, lddx);
  else hipLaunchKernelGGL((mx_dx_parts_kernel<0>), sums, dim3(256), 0, s, (const float*)ws, n, k, (int)parts, dX, lddx);
  return hipGetLastError();
}

// The gradient of many rows: the weights are expanded and transposed once, into
// the workspace, and the product runs on bf16 tiles without any expansion.
// The device's 256 CUs hold one 256 x 256 tile each; the rows that this form takes
// are all full ones where the last round of tiles is at least four fifths full, else
// those of the full rounds before it, of which there must be two.  us for m = k =
// 4096 with this / with tiles that expand for themselves: 4096 rows 129 / 140, 8195
// rows 251 / 315, 16384 rows 459 / 536; below a round 2048 rows 105 / 92.
int64_t mxfp4_gemm_dx_expanded_rows(int64_t n, int64_t m, int64_t k) {
  if (m % 8 != 0) return 0;   // (a row of W^T is copied in pieces of 16 bytes)
  const int64_t across = (k + 255) / 256, full = n / 256 * across, rounds = full / 256, left = full % 256;
  if (full >= 256 ? left == 0 || 5 * left >= 4 * 256 : 5 * left >= 4 * 256) return n / 256 * 256;
  return rounds >= 2 ? 256 * rounds / across * 256 : 0;
}

hipError_t mxfp4_gemm_dx_expanded_launch(const uint16_t* dY, int64_t n, int64_t m, int64_t lddy, const uint8_t* codes,
                                         const uint8_t* scales, int64_t k, void* dX, int out_bf16, int64_t lddx, void* ws,
                                         hipStream_t s) {
  const dim3 grid((unsigned)((m + 63) / 64), (unsigned)((k + 63) / 64));
  hipLaunchKernelGGL(mx_transpose_kernel, grid, dim3(256), 0, s, codes, scales, m, k, (uint16_t*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  using TL = MxTile<2, 4, 4, 2, 2, 2, true>;
  const int64_t blocks = (((k + TL::kM - 1) / TL::kM) * ((n + TL::kN - 1) / TL::kN) + 7) / 8 * 8;
  if (blocks > kMaxThreads / TL::kThreads) return kTooManyTiles;
#define NVQ_DX(OUT)                                                                                                            \
  hipLaunchKernelGGL((mx_tile_kernel<2, 4, 4, 2, 2, 2, true, OUT>), dim3((unsigned)blocks), dim3(TL::kThreads), 0, s, (const uint8_t*)dY,   \
                     2 * lddy, nullptr, n, 2 * m, (const uint8_t*)ws, 2 * m, nullptr, k, dX, lddx)
  if (out_bf16) NVQ_DX(1);
  else NVQ_DX(0);
#undef NVQ_DX
  return hipGetLastError();
}

}  // namespace nvq
