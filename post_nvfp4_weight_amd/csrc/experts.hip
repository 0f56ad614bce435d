// Products of routed token rows with the experts' NVFP4 weights.
//   forward:  Y[r]  = g_e X[tok_idx[r]] Q_e^T   for grp_off[e] <= r < grp_off[e + 1]
//   backward: dX[r] = g_e dY[r] Q_e
// Q = e2m1 * e4m3 is exact in bf16 (at most 6 significant bits), products run
// on the bf16 matrix cores with fp32 accumulation and g is applied once, as
// in nvfp4_gemm.  The group offsets stay on the device: the grid covers the
// most row tiles that any offsets can give, and each workgroup finds its
// expert from them.
#include <algorithm>

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
};

// The tile-th row tile of height bt over all experts in order; false past the
// last one.  Called by a whole workgroup of NT threads.
template <int NT>
__device__ __forceinline__ bool find_tile(const int64_t* off, int64_t G, int64_t rows, int bt, int64_t tile,
                                          RowTile* out) {
  __shared__ int64_t wsum[NT / 64];
  __shared__ RowTile found;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t before = 0;   // tiles of the experts before this turn's
  for (int64_t x0 = 0; x0 < G; x0 += NT) {
    const int64_t x = x0 + threadIdx.x;
    int64_t b = 0, e = 0;
    if (x < G) group_range(off, x, rows, &b, &e);
    const int64_t cnt = (e - b + bt - 1) / bt;
    int64_t incl = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t y = __shfl_up(incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int64_t base = before, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      base += w < wave ? wsum[w] : 0;
      all += wsum[w];
    }
    const int64_t first = base + incl - cnt;
    if (tile >= first && tile < first + cnt) {
      found.expert = x;
      found.r0 = b + (tile - first) * bt;
      found.r1 = min(e, found.r0 + bt);
    }
    before += all;
    __syncthreads();
    if (tile < before) {   // the same in every thread
      *out = found;
      return true;
    }
  }
  return false;
}

// The forward product: 128 rows x 128 output channels per workgroup, four
// waves of 64 x 64, k in steps of 64; both operands in LDS as [row][k], rows
// padded to 72 elements, double-buffered.
constexpr int ET = 128, EK = 64, ELD = EK + 8, EBUF = 2 * ET * ELD;

template <int OUT_BF16>
__global__ __launch_bounds__(256) void grouped_gemm_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t k,
                                                           int64_t ldx, const int32_t* __restrict__ tok_idx,
                                                           int64_t rows, const int64_t* __restrict__ off, int64_t G,
                                                           const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales,
                                                           const float* __restrict__ gs, int64_t m,
                                                           void* __restrict__ Y, int64_t ldy) {
  __shared__ __attribute__((aligned(16))) uint16_t smem[2 * EBUF];
  RowTile tl;
  if (!find_tile<256>(off, G, rows, ET, blockIdx.x, &tl)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave >> 1, wc = wave & 1;
  const int64_t o0 = (int64_t)blockIdx.y * ET;
  const int64_t kb = k / 16;
  codes += tl.expert * m * (k / 2);
  scales += tl.expert * m * kb;

  // Per step: 128 rows x 64 k of X = 4 x 16 B per thread; 128 weight rows x 4
  // blocks = 2 blocks per thread.
  const uint16_t* xrow[4];
  bool xok[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t r = tl.r0 + ((q * 256 + tid) >> 3);
    int64_t t = r < tl.r1 ? (tok_idx ? tok_idx[r] : r) : -1;
    xok[q] = t >= 0 && t < n;
    xrow[q] = X + (xok[q] ? t : 0) * ldx;
  }
  const int wrow = tid >> 1, wh = tid & 1;
  const int64_t row = min(o0 + wrow, m - 1);
  auto load = [&](int64_t k0, u32x4 (&xv)[4], u32x2 (&cv)[2], uint32_t (&sv)[2]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) xv[q] = *(const u32x4*)(xrow[q] + min(k0 + ((q * 256 + tid) & 7) * 8, k - 8));
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t blk = min(k0 / 16 + 2 * wh + b, kb - 1);
      cv[b] = *(const u32x2*)(codes + row * (k / 2) + blk * 8);
      sv[b] = scales[row * kb + blk];
    }
  };
  auto store = [&](uint16_t* buf, int64_t k0, const u32x4 (&xv)[4], const u32x2 (&cv)[2], const uint32_t (&sv)[2]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = q * 256 + tid, r = e >> 3, c8 = (e & 7) * 8;
      *(u32x4*)(buf + r * ELD + c8) = xok[q] && k0 + c8 < k ? xv[q] : u32x4{0u, 0u, 0u, 0u};
    }
    uint16_t* qb = buf + ET * ELD;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t keep = o0 + wrow < m && k0 + 32 * wh + 16 * b < k ? ~0u : 0u;
      const float sb = e4m3_byte<0>(sv[b]);
      u32x4 lo, hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = dq_byte(cv[b][0], sb, j) & keep;
        hi[j] = dq_byte(cv[b][1], sb, j) & keep;
      }
      *(u32x4*)(qb + wrow * ELD + 32 * wh + 16 * b) = lo;
      *(u32x4*)(qb + wrow * ELD + 32 * wh + 16 * b + 8) = hi;
    }
  };

  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int64_t nsteps = (k + EK - 1) / EK;
  u32x4 xv[4];
  u32x2 cv[2];
  uint32_t sv[2];
  load(0, xv, cv, sv);
  store(smem, 0, xv, cv, sv);
  __syncthreads();
  const int arow = wr * 64 + (lane & 31), brow = wc * 64 + (lane & 31), koff = 8 * (lane >> 5);
  for (int64_t st = 0; st < nsteps; ++st) {
    const int cur = (int)(st & 1);
    if (st + 1 < nsteps) load((st + 1) * EK, xv, cv, sv);
    const uint16_t* Xs = smem + cur * EBUF;
    const uint16_t* Qs = Xs + ET * ELD;
#pragma unroll
    for (int ks = 0; ks < EK; ks += 16) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        a[t] = *(const bf16x8*)(Xs + (arow + 32 * t) * ELD + ks + koff);
        b[t] = *(const bf16x8*)(Qs + (brow + 32 * t) * ELD + ks + koff);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    if (st + 1 < nsteps) store(smem + (cur ^ 1) * EBUF, (st + 1) * EK, xv, cv, sv);
    __syncthreads();
  }

  // Accumulator layout: lane l, register r -> row 8 (r/4) + 4 (l/32) + r%4, column l%32.
  const float g = gs[tl.expert];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t orow = tl.r0 + wr * 64 + i * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        const int64_t col = o0 + wc * 64 + j * 32 + (lane & 31);
        if (orow < tl.r1 && col < m) {
          const float v = acc[i][j][r] * g;
          if (OUT_BF16) ((__bf16*)Y)[orow * ldy + col] = (__bf16)v;
          else ((float*)Y)[orow * ldy + col] = v;
        }
      }
}

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
  if (!find_tile<256>(off, G, rows, ET, blockIdx.x, &tl)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave >> 1, wc = wave & 1;
  const int64_t o0 = (int64_t)blockIdx.y * ET;
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

// The most row tiles of height bt that rows over G experts can make: every
// expert that has rows adds at most one part tile.
int64_t most_tiles(int64_t rows, int64_t G, int bt) { return rows / bt + std::min(rows, G); }

}  // namespace

hipError_t nvfp4_gemm_grouped_launch(const uint16_t* X, int64_t n, int64_t k, int64_t ldx, const int32_t* tok_idx,
                                     int64_t rows, const int64_t* grp_off, int64_t G, const uint8_t* codes,
                                     const uint8_t* scales, const float* g, int64_t m, void* Y, int out_bf16,
                                     int64_t ldy, hipStream_t s) {
  const dim3 grid((unsigned)most_tiles(rows, G, ET), (unsigned)((m + ET - 1) / ET));
  if (out_bf16)
    hipLaunchKernelGGL(grouped_gemm_kernel<1>, grid, dim3(256), 0, s, X, n, k, ldx, tok_idx, rows, grp_off, G, codes,
                       scales, g, m, Y, ldy);
  else
    hipLaunchKernelGGL(grouped_gemm_kernel<0>, grid, dim3(256), 0, s, X, n, k, ldx, tok_idx, rows, grp_off, G, codes,
                       scales, g, m, Y, ldy);
  return hipGetLastError();
}

hipError_t nvfp4_gemm_grouped_dx_launch(const uint16_t* dY, int64_t rows, int64_t m, int64_t lddy,
                                        const int64_t* grp_off, int64_t G, const uint8_t* codes, const uint8_t* scales,
                                        const float* g, int64_t k, void* dX, int out_bf16, int64_t lddx,
                                        hipStream_t s) {
  const dim3 grid((unsigned)most_tiles(rows, G, ET), (unsigned)((k + ET - 1) / ET));
  if (out_bf16)
    hipLaunchKernelGGL(grouped_dx_kernel<1>, grid, dim3(256), 0, s, dY, rows, m, lddy, grp_off, G, codes, scales, g, k,
                       dX, lddx);
  else
    hipLaunchKernelGGL(grouped_dx_kernel<0>, grid, dim3(256), 0, s, dY, rows, m, lddy, grp_off, G, codes, scales, g, k,
                       dX, lddx);
  return hipGetLastError();
}

}  // namespace nvq
