// Products of routed token rows with the experts' NVFP4 weights.
//   forward:  Y[r]  = g_e X[tok_idx[r]] Q_e^T   for grp_off[e] <= r < grp_off[e + 1]
//   backward: dX[r] = g_e dY[r] Q_e
// Q = e2m1 * e4m3 is exact in bf16 (at most 6 significant bits), products run
// on the bf16 matrix cores with fp32 accumulation and g is applied once, as
// in nvfp4_gemm.  The group offsets stay on the device: the grid covers the
// most row tiles that any offsets can give, and each workgroup finds its
// expert from them.
#include <algorithm>
#include <cstdlib>

#include "common.h"
#include "dequant.h"
#include "kernels.h"

namespace nvq {

namespace {

// Row range [*b, *e) of expert x, clamped into [0, rows], so that no offsets lead out of the buffers.
__device__ __forceinline__ void group_range(const int64_t* off, int64_t x, int64_t rows, int64_t* b, int64_t* e) {
  *b = min(max(off[x], (int64_t)0), rows);
  *e = min(max(off[x + 1], *b), rows);
}

struct RowTile {
  int64_t expert, r0, r1;   // rows [r0, r1), r1 at most r0 + the tile height and within the expert's rows
  int64_t col;              // column tile
};

// Row tiles of height bt over all experts in order, times ncol column tiles
// each (column tiles of a row tile next to each other): the one of this
// workgroup, false if there is none.  The tiles are dealt to the 8 XCDs
// (blockIdx.x mod 8) in contiguous runs, so that the tiles that share an
// expert's weights or a row tile's activations share an L2.  Called by a whole
// workgroup of NT threads.
template <int NT>
__device__ __forceinline__ bool find_tile(const int64_t* off, int64_t G, int64_t rows, int bt, int64_t ncol,
                                          RowTile* out) {
  __shared__ int64_t wsum[NT / 64];
  __shared__ RowTile found;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t b = 0, e = 0, first = 0, cnt = 0;
  // Tiles of experts x0 + thread, and the sum over all of this turn's.
  auto turn = [&](int64_t x0) {
    const int64_t x = x0 + threadIdx.x;
    b = e = 0;
    if (x < G) group_range(off, x, rows, &b, &e);
    cnt = (e - b + bt - 1) / bt;
    int64_t incl = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int64_t all = 0;
    first = incl - cnt;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      first += w < wave ? wsum[w] : 0;
      all += wsum[w];
    }
    return all;
  };
  int64_t total = 0;
  for (int64_t x0 = 0; x0 < G; x0 += NT) total += turn(x0);
  const int64_t n = total * ncol, per = (n + 7) / 8;
  const int64_t i = blockIdx.x >> 3, id = (blockIdx.x & 7) * per + i;
  if (i >= per || id >= n) return false;   // the same in every thread
  const int64_t tile = id / ncol;
  int64_t before = 0;
  for (int64_t x0 = 0; x0 < G; x0 += NT) {
    const int64_t all = G > NT ? turn(x0) : total;   // (one turn: its values are still there)
    if (tile >= before + first && tile < before + first + cnt) {
      found.expert = x0 + threadIdx.x;
      found.r0 = b + (tile - before - first) * bt;
      found.r1 = min(e, found.r0 + bt);
    }
    before += all;
  }
  __syncthreads();
  *out = found;
  out->col = id - tile * ncol;
  return true;
}

typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
__device__ __forceinline__ constexpr int waitcnt_vm_lgkm0(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// The forward product: 32 RF rows x 32 CF NW output channels per workgroup of
// NW waves, each wave all the rows times its own 32 CF channels, so that a
// weight is expanded once, by the wave that multiplies it, into the fragment
// it is needed in.
//   v_mfma_f32_32x32x16_bf16, A = 32 channels, B = 32 rows: lane (c = l % 32,
//   h = l / 32) holds 8 consecutive k of channel c and of row c.
//   k goes in steps of 64 = four products; product j takes k = 32 h + 8 j ..
//   + 7 of the step for both operands (the order of k in the sum is free), so
//   that a lane's codes of a step are 16 consecutive bytes under two scales.
//   Activations: rows of 128 bytes per step, copied to LDS directly two steps
//   ahead into a ring of three buffers, 16-byte pieces swizzled by
//   (row / 2) % 8: the 16 rows that are read at once then touch all 64 banks.
//   Codes: 128 k at a time (a chunk, two steps), 64 bytes per channel, copied
//   to LDS of the wave's own two chunks ahead, pieces swizzled by
//   (channel / 4) % 4 for the same reason.  (Loaded to registers instead, 32
//   bytes per channel and load, they took the address unit twice the cycles.)
//   Scales: 8 bytes per channel and chunk to registers, one chunk ahead.
template <int NW, int RF, int CF>
struct Tile {
  static constexpr int kRows = 32 * RF, kCols = 32 * CF * NW;
  static constexpr int kXBuf = kRows * 128, kCBuf = CF * 32 * 64;   // bytes of one buffer (of a wave's codes)
  static constexpr int kXLoads = 4 * RF / NW, kCLoads = 2 * CF;     // copies per step, per chunk
  static constexpr int kLds = 3 * kXBuf + 3 * NW * kCBuf;
  static_assert(4 * RF % NW == 0, "whole copies per wave");
};

// A lane's scales of a chunk, for CF groups of 32 channels; word [t] has step
// t's four blocks.  LAST: the end of k, `left` blocks, zeros behind them (the
// codes read there are some of the next channel's, finite, times zeros).
template <int CF, bool LAST>
__device__ __forceinline__ void load_scales(const uint8_t* scales, const uint32_t (&srow)[CF], int64_t left,
                                            u32x2 (&s)[CF]) {
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    if (!LAST) {
      s[f] = *(const u32x2_any*)(scales + srow[f]);
    } else {
      s[f] = u32x2{0u, 0u};
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (b < left) s[f][b >> 2] |= (uint32_t)scales[srow[f] + b] << (8 * (b & 3));
    }
  }
}

// NL copies of 1024 bytes to LDS (16 per lane), from `src` + off[q]; offsets at
// or past the bound bring zeros.
template <int NL, int STRIDE>
__device__ __forceinline__ void copy_lds(char* __restrict__ dst, const void* src, uint32_t bound, const uint32_t (&off)[NL],
                                         bool in) {
#if __HIP_DEVICE_COMPILE__
  __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, (short)0, bound, 0x00020000);
#pragma unroll
  for (int q = 0; q < NL; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + q * STRIDE), 16,
                                             in ? off[q] : 0xFFFFFFF0u, 0, 0, 0);
#endif
}

// What a wave's steps share.
template <int NW, int RF, int CF>
struct Wave {
  uint32_t xoff[Tile<NW, RF, CF>::kXLoads];   // its copies' byte offsets from X
  uint32_t coff[Tile<NW, RF, CF>::kCLoads];   // and from its codes
  int xrd[4], crd[2];                         // LDS offsets of product j's row fragment, of step t's codes
  int h;
};

// Step T of a chunk: its four products on xb, the activations of two steps on
// into xd and (T = 0) the codes of two chunks on into cd; cb and cn are this
// chunk's codes and the next's.  The buffers are distinct, which the restrict
// qualifiers state, so that reads need not wait for the copies in flight.
template <int NW, int RF, int CF, int T, bool WIDE>
__device__ __forceinline__ void product_step(const char* __restrict__ xb, const char* __restrict__ xn,
                                             char* __restrict__ xd, const char* __restrict__ cb,
                                             const char* __restrict__ cn, char* __restrict__ cd, const uint16_t* xsrc,
                                             uint32_t xbound, bool in, const uint8_t* csrc, uint32_t cbound,
                                             const Wave<NW, RF, CF>& w, const u32x2 (&sc)[CF], const u32x2 (&sn)[CF],
                                             u32x4 (&cw)[CF], bf16x8 (&xa)[RF], u32x4 (&qa)[2][CF],
                                             f32x16 (&acc)[RF][CF]) {
  using TL = Tile<NW, RF, CF>;
  constexpr int NX = TL::kXLoads, NC = TL::kCLoads;
  u32x4 cnext[CF];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = j & 1;
    if (j == 2) {
      // The next step's codes.  Behind those of the next chunk were issued three
      // steps' activations, one chunk's codes and one chunk's scales.
      if (T == 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * NX + NC + (WIDE ? CF : 0)));
#pragma unroll
      for (int f = 0; f < CF; ++f) cnext[f] = *(const u32x4*)((T == 0 ? cb : cn) + f * 2048 + w.crd[T ^ 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (j == 3) {
      // The next step's activations: behind them were issued this step's, one
      // chunk's codes and (in a chunk's first step) the next chunk's scales.
      // Every wave has read all of this step's buffer by now.
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(NX + NC + (T == 0 && WIDE ? CF : 0)));
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    // A row fragment is read for the next product right behind the products
    // that use it; codes are expanded for the next product between them.
#pragma unroll
    for (int i = 0; i < RF; ++i) {
#pragma unroll
      for (int f = 0; f < CF; ++f)
        acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, qa[p][f]), xa[i], acc[i][f], 0, 0, 0);
      xa[i] = j < 3 ? *(const bf16x8*)(xb + i * 4096 + w.xrd[(j + 1) & 3]) : *(const bf16x8*)(xn + i * 4096 + w.xrd[0]);
#pragma unroll
      for (int e = i * 4 * CF / RF; e < (i + 1) * 4 * CF / RF; ++e) {
        const int f = e / 4, piece = e % 4;
        // product j + 1 of this step, or product 0 of the next
        const uint32_t word = j < 3 ? cw[f][(j + 1) & 3] : cnext[f][0];
        const uint32_t s2 = (j < 3 ? sc[f][T] : T == 0 ? sc[f][1] : sn[f][0]) >> (16 * w.h);
        const float s = j == 0 || j == 3 ? e4m3_byte<0>(s2) : e4m3_byte<1>(s2);
        qa[p ^ 1][f][piece] = dq_byte(word, s, piece);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (j == 0 && i == 0) {
        copy_lds<NX, NW * 1024>(xd, xsrc, xbound, w.xoff, in);
        if (T == 0) copy_lds<NC, 1024>(cd, csrc, cbound, w.coff, true);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < CF; ++f) cw[f] = cnext[f];
}

// Rows without a token (their number is outside [0, n)) read token 0's and
// are stored as zeros.
template <int NW, int RF, int CF, int OUT_BF16>
__device__ __forceinline__ void tile_product(char* smem, const RowTile& tl, const uint16_t* __restrict__ X, int64_t n,
                                             int64_t k, int64_t ldx, const int32_t* __restrict__ tok_idx,
                                             const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                             float g, int64_t m, void* __restrict__ Y, int64_t ldy, bool vec_out) {
  using TL = Tile<NW, RF, CF>;
  constexpr int NX = TL::kXLoads, NC = TL::kCLoads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int64_t kb = k / 16;
  const int64_t o0 = tl.col * TL::kCols + wave * 32 * CF;
  Wave<NW, RF, CF> w;
  w.h = h;

  // Copy q of a step brings rows 8 (NW q + wave) + lane / 8.
  const int xk = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 8;   // the lane's k in the step: its piece ^ (row / 2) % 8
#pragma unroll
  for (int q = 0; q < NX; ++q) {
    const int64_t r = tl.r0 + 8 * (NW * q + wave) + (lane >> 3);
    const int64_t t = r < tl.r1 ? (tok_idx ? tok_idx[r] : r) : 0;
    w.xoff[q] = (uint32_t)((t >= 0 && t < n ? t : 0) * ldx + xk) * 2;
  }
  // Bytes of X from step st on (below 2^32 - 256: checked on the host).
  auto bound = [&](int64_t st) { return (uint32_t)max((int64_t)0, ((n - 1) * ldx + k - st * 64) * 2); };
  auto inside = [&](int64_t st) { return st * 64 + xk < k; };

  // Codes: copy q of a chunk brings channels 16 q + lane / 4.  Channels past m
  // and bytes past the expert's last are zeros.
  const int64_t first = min(o0, m);   // the wave's first channel; the lane's ones as offsets from it
  codes += first * (k / 2);
  scales += min(first, m - 1) * kb;
#pragma unroll
  for (int q = 0; q < NC; ++q) w.coff[q] = (uint32_t)((16 * q + (lane >> 2)) * (k / 2)) + 16 * ((lane & 3) ^ (lane >> 4));
  auto cbound = [&](int64_t ch) { return (uint32_t)min(max((int64_t)0, (m - first) * (k / 2) - ch * 64), (int64_t)0xFFFFFF00); };
  uint32_t srow[CF];
#pragma unroll
  for (int f = 0; f < CF; ++f) srow[f] = (uint32_t)((min(o0 + 32 * f + c, m - 1) - min(first, m - 1)) * kb);
#pragma unroll
  for (int j = 0; j < 4; ++j) w.xrd[j] = c * 128 + (((4 * h + j) ^ ((c >> 1) & 7)) * 16);
#pragma unroll
  for (int t = 0; t < 2; ++t) w.crd[t] = c * 64 + (((2 * t + h) ^ ((c >> 2) & 3)) * 16);

  f32x16 acc[RF][CF];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int f = 0; f < CF; ++f)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][f][r] = 0.0f;

  char *x0 = smem, *x1 = smem + TL::kXBuf, *x2 = smem + 2 * TL::kXBuf;   // steps st, st + 1, st + 2
  char* cl = smem + 3 * TL::kXBuf + wave * 3 * TL::kCBuf;
  char *c0 = cl, *c1 = cl + TL::kCBuf, *c2 = cl + 2 * TL::kCBuf;         // chunks ch, ch + 1, ch + 2
  const int xw = wave * 1024;
  u32x2 sc[CF], sn[CF];
  u32x4 cw[CF], qa[2][CF];
  bf16x8 xa[RF];
  const int whole = (int)(k / 128), nchunks = (int)((k + 127) / 128);
  if (whole) load_scales<CF, false>(scales, srow, 8, sc);
  else load_scales<CF, true>(scales, srow, kb, sc);
  copy_lds<NC, 1024>(c0, codes, cbound(0), w.coff, true);
  copy_lds<NX, NW * 1024>(x0 + xw, X, bound(0), w.xoff, inside(0));
  __builtin_amdgcn_sched_barrier(0);
  copy_lds<NC, 1024>(c1, codes + 64, cbound(1), w.coff, true);
  copy_lds<NX, NW * 1024>(x1 + xw, X + 64, bound(1), w.xoff, inside(1));
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(NX + NC));   // step 0's and chunk 0's have landed
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int i = 0; i < RF; ++i) xa[i] = *(const bf16x8*)(x0 + i * 4096 + w.xrd[0]);
#pragma unroll
  for (int f = 0; f < CF; ++f) cw[f] = *(const u32x4*)(c0 + f * 2048 + w.crd[0]);
#pragma unroll
  for (int f = 0; f < CF; ++f)
#pragma unroll
    for (int p = 0; p < 4; ++p) qa[0][f][p] = dq_byte(cw[f][0], e4m3_byte<0>(sc[f][0] >> (16 * h)), p);

  // Two steps per chunk, with no branch between them (a join would make the
  // compiler copy the accumulators): where k ends in a chunk's first half, the
  // second multiplies zeros.
  auto chunk = [&]<bool WIDE>(int ch) {
    const int64_t st = 2 * ch;
    load_scales<CF, !WIDE>(scales + (ch + 1) * 8, srow, kb - 8 * (ch + 1), sn);
    __builtin_amdgcn_sched_barrier(0);
    product_step<NW, RF, CF, 0, WIDE>(x0, x1, x2 + xw, c0, c1, c2, X + (st + 2) * 64, bound(st + 2), WIDE || inside(st + 2),
                                      codes + (ch + 2) * 64, cbound(ch + 2), w, sc, sn, cw, xa, qa, acc);
    product_step<NW, RF, CF, 1, WIDE>(x1, x2, x0 + xw, c0, c1, c2, X + (st + 3) * 64, bound(st + 3), WIDE || inside(st + 3),
                                      codes, 0, w, sc, sn, cw, xa, qa, acc);
#pragma unroll
    for (int f = 0; f < CF; ++f) sc[f] = sn[f];
    char *x = x0, *cc = c0;
    x0 = x2;
    x2 = x1;
    x1 = x;
    c0 = c1;
    c1 = c2;
    c2 = cc;
  };
  int ch = 0;
  for (; ch < whole - 1; ++ch) chunk.template operator()<true>(ch);
  for (; ch < nchunks; ++ch) chunk.template operator()<false>(ch);
  // The copies issued for steps past the end still write LDS (zeros): none may
  // be in flight once the workgroup's LDS is released.
  __builtin_amdgcn_s_waitcnt(0);

  // Accumulator: lane l, register r -> channel 8 (r / 4) + 4 h + r % 4, row c.
#pragma unroll
  for (int i = 0; i < RF; ++i) {
    const int64_t row = tl.r0 + 32 * i + c;
    if (row >= tl.r1) continue;
    const bool token = !tok_idx || (tok_idx[row] >= 0 && tok_idx[row] < n);
#pragma unroll
    for (int f = 0; f < CF; ++f)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int64_t o = o0 + 32 * f + 8 * r4 + 4 * h;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = token ? acc[i][f][4 * r4 + r] * g : 0.0f;
        if (vec_out && o + 4 <= m) {
          if (OUT_BF16) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *(bf16x4*)((__bf16*)Y + row * ldy + o) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
          } else {
            *(f32x4*)((float*)Y + row * ldy + o) = f32x4{v[0], v[1], v[2], v[3]};
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (o + r < m) {
              if (OUT_BF16) ((__bf16*)Y)[row * ldy + o + r] = (__bf16)v[r];
              else ((float*)Y)[row * ldy + o + r] = v[r];
            }
        }
      }
  }
}

template <int NW, int RF, int CF, int OUT_BF16>
__global__ __launch_bounds__(64 * NW, 2) void grouped_gemm_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t k,
                                                                  int64_t ldx, const int32_t* __restrict__ tok_idx,
                                                                  int64_t rows, const int64_t* __restrict__ off,
                                                                  int64_t G, const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const float* __restrict__ gs, int64_t m,
                                                                  void* __restrict__ Y, int64_t ldy, int vec_out) {
  using TL = Tile<NW, RF, CF>;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  RowTile tl;
  if (!find_tile<64 * NW>(off, G, rows, TL::kRows, (m + TL::kCols - 1) / TL::kCols, &tl)) return;
  tile_product<NW, RF, CF, OUT_BF16>(smem, tl, X, n, k, ldx, tok_idx, codes + tl.expert * m * (k / 2),
                                     scales + tl.expert * m * (k / 16), gs[tl.expert], m, Y, ldy, vec_out != 0);
}

constexpr int ET = 128, EK = 64, ELD = EK + 8, EBUF = 2 * ET * ELD;

// The gradient of the rows: 128 rows x 128 input channels per workgroup, the
// sum over m in steps of 64.  A weight tile of 64 m x 128 k is expanded and
// stored transposed, [k][m], so that both operands are read as above.
template <int OUT_BF16>
__global__ __launch_bounds__(256) void grouped_dx_kernel(const uint16_t* __restrict__ dY, int64_t rows, int64_t m,
                                                         int64_t lddy, const int64_t* __restrict__ off, int64_t G,
                                                         const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales,
                                                         const float* __restrict__ gs, int64_t k,
                                                         void* __restrict__ dX, int64_t lddx) {
  __shared__ __attribute__((aligned(16))) uint16_t smem[EBUF];
  RowTile tl;
  if (!find_tile<256>(off, G, rows, ET, (k + ET - 1) / ET, &tl)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave >> 1, wc = wave & 1;
  const int64_t o0 = tl.col * ET;
  const int64_t kb = k / 16;
  codes += tl.expert * m * (k / 2);
  scales += tl.expert * m * kb;
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  uint16_t* Ds = smem;
  uint16_t* Qs = smem + ET * ELD;
  const int arow = wr * 64 + (lane & 31), brow = wc * 64 + (lane & 31), koff = 8 * (lane >> 5);
  for (int64_t m0 = 0; m0 < m; m0 += EK) {
    // dY: 128 rows x 64 m, element by element (rows of dY have any alignment)
    for (int q = 0; q < 32; ++q) {
      const int e = q * 256 + tid, r = e >> 6, c = e & 63;
      const bool ok = tl.r0 + r < tl.r1 && m0 + c < m;
      Ds[r * ELD + c] = ok ? dY[(tl.r0 + r) * lddy + m0 + c] : (uint16_t)0;
    }
    // weights: 64 m x 8 blocks, 2 blocks per thread
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int e = q * 256 + tid, r = e >> 3, b = e & 7;
      const int64_t blk = o0 / 16 + b;
      const bool ok = m0 + r < m && blk < kb;
      u32x2 cv{0u, 0u};
      float sb = 0.0f;
      if (ok) {
        cv = *(const u32x2*)(codes + (m0 + r) * (k / 2) + blk * 8);
        sb = e4m3_byte<0>(scales[(m0 + r) * kb + blk]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t p = dq_byte(cv[j >> 2], sb, j & 3);
        Qs[(16 * b + 2 * j) * ELD + r] = (uint16_t)p;
        Qs[(16 * b + 2 * j + 1) * ELD + r] = (uint16_t)(p >> 16);
      }
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < EK; ks += 16) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        a[t] = *(const bf16x8*)(Ds + (arow + 32 * t) * ELD + ks + koff);
        b[t] = *(const bf16x8*)(Qs + (brow + 32 * t) * ELD + ks + koff);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
  const float g = gs[tl.expert];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t orow = tl.r0 + wr * 64 + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        const int64_t col = o0 + wc * 64 + j * 32 + (lane & 31);
        if (orow < tl.r1 && col < k) {
          const float v = acc[i][j][r] * g;
          if (OUT_BF16) ((__bf16*)dX)[orow * lddx + col] = (__bf16)v;
          else ((float*)dX)[orow * lddx + col] = v;
        }
      }
}

// Workgroups for every row tile of height bt that rows over G experts can
// make (an expert with rows adds at most one part tile), times ncol; a
// multiple of 8, as find_tile deals them to the XCDs.
int64_t most_tiles(int64_t rows, int64_t G, int bt, int64_t ncol) {
  return ((rows / bt + std::min(rows, G)) * ncol + 7) / 8 * 8;
}

}  // namespace

hipError_t nvfp4_gemm_grouped_launch(const uint16_t* X, int64_t n, int64_t k, int64_t ldx, const int32_t* tok_idx,
                                     int64_t rows, const int64_t* grp_off, int64_t G, const uint8_t* codes,
                                     const uint8_t* scales, const float* g, int64_t m, void* Y, int out_bf16,
                                     int64_t ldy, hipStream_t s) {
  const int vec = ldy % 4 == 0 && (uintptr_t)Y % (out_bf16 ? 8 : 16) == 0;
#define NVQ_GROUPED(NW, RF, CF)                                                                                      \
  do {                                                                                                               \
    using TL = Tile<NW, RF, CF>;                                                                                     \
    const int64_t blocks = most_tiles(rows, G, TL::kRows, (m + TL::kCols - 1) / TL::kCols);                          \
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;                                                            \
    if (out_bf16)                                                                                                    \
      hipLaunchKernelGGL((grouped_gemm_kernel<NW, RF, CF, 1>), dim3((unsigned)blocks), dim3(64 * NW), 0, s, X, n, k, \
                         ldx, tok_idx, rows, grp_off, G, codes, scales, g, m, Y, ldy, vec);                          \
    else                                                                                                             \
      hipLaunchKernelGGL((grouped_gemm_kernel<NW, RF, CF, 0>), dim3((unsigned)blocks), dim3(64 * NW), 0, s, X, n, k, \
                         ldx, tok_idx, rows, grp_off, G, codes, scales, g, m, Y, ldy, vec);                          \
  } while (0)
  const int64_t avg = rows / std::min(rows, G);
  const char* force = getenv("NVQ_RF");
  const int f = force ? atoi(force) : avg >= 96 ? 4 : avg >= 16 ? 2 : 1;
  if (f == 4) NVQ_GROUPED(8, 4, 2);
  else if (f == 2) NVQ_GROUPED(8, 2, 2);
  else if (f == 5) NVQ_GROUPED(4, 4, 1);
  else if (f == 3) NVQ_GROUPED(4, 2, 1);
  else if (f == 6) NVQ_GROUPED(4, 1, 2);
  else NVQ_GROUPED(4, 1, 1);
#undef NVQ_GROUPED
  return hipGetLastError();
}

hipError_t nvfp4_gemm_grouped_dx_launch(const uint16_t* dY, int64_t rows, int64_t m, int64_t lddy,
                                        const int64_t* grp_off, int64_t G, const uint8_t* codes, const uint8_t* scales,
                                        const float* g, int64_t k, void* dX, int out_bf16, int64_t lddx,
                                        hipStream_t s) {
  const int64_t blocks = most_tiles(rows, G, ET, (k + ET - 1) / ET);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (out_bf16)
    hipLaunchKernelGGL(grouped_dx_kernel<1>, grid, dim3(256), 0, s, dY, rows, m, lddy, grp_off, G, codes, scales, g, k,
                       dX, lddx);
  else
    hipLaunchKernelGGL(grouped_dx_kernel<0>, grid, dim3(256), 0, s, dY, rows, m, lddy, grp_off, G, codes, scales, g, k,
                       dX, lddx);
  return hipGetLastError();
}

}  // namespace nvq
