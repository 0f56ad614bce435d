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

struct RowTile {
  int64_t expert, r0, r1;   // rows [r0, r1), r1 at most r0 + the tile height and within the expert's rows
  int64_t col;              // column tile
};

// Row tiles of height BT over all experts in order, times ncol column tiles
// each (column tiles of a row tile next to each other): the one of this
// workgroup, false if there is none.  The tiles are dealt to the 8 XCDs
// (blockIdx.x mod 8) in contiguous runs, so that the tiles that share an
// expert's weights or a row tile's activations share an L2.  Each wave sums the
// tile counts of all experts by itself, 4 experts per lane and turn: no
// barrier, and about 1 us less than sums across the workgroup took, which a
// one-token product spends several times over.  Offsets are clamped into
// [0, rows], so that none lead out of the buffers.
template <int BT>
__device__ __forceinline__ bool find_tile(const int64_t* __restrict__ off, int64_t G, int64_t rows, uint32_t ncol,
                                          RowTile* out) {
  constexpr int EPL = 4;
  const int lane = threadIdx.x & 63;
  int b[EPL], e[EPL], mine = 0, incl = 0;
  auto turn = [&](int64_t x0) {   // tiles of experts x0 + EPL lane ..; returns the sum over the wave
    int64_t v[EPL + 1];
#pragma unroll
    for (int i = 0; i <= EPL; ++i) v[i] = off[min(x0 + EPL * lane + i, G)];
    mine = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      b[i] = (int)min(max(v[i], (int64_t)0), rows);
      e[i] = (int)min(max(v[i + 1], (int64_t)b[i]), rows);
      mine += (int)(((uint32_t)(e[i] - b[i]) + BT - 1) / BT);
    }
    incl = wave_inclusive(mine);
    return (uint32_t)__builtin_amdgcn_readlane(incl, 63);
  };
  uint32_t total = 0;
  for (int64_t x0 = 0; x0 < G; x0 += 64 * EPL) total += turn(x0);
  const uint64_t n = (uint64_t)total * ncol, per = (n + 7) / 8;
  const uint32_t i = blockIdx.x >> 3;
  const uint64_t id = (blockIdx.x & 7) * per + i;
  if (i >= per || id >= n) return false;
  const uint32_t tile = (uint32_t)id / ncol;   // (the grid has fewer than 2^31 workgroups)
  uint32_t before = 0;
  for (int64_t x0 = 0; x0 < G; x0 += 64 * EPL) {
    const uint32_t all = G > 64 * EPL ? turn(x0) : total;   // (one turn: its values are still there)
    if (tile < before + all) {
      const uint32_t first = before + incl - mine;   // of the lane's experts
      const uint64_t who = __ballot(tile >= first && tile < first + mine);
      if (!who) return false;   // (only decreasing offsets that make the sums overflow)
      const int src = __ffsll((unsigned long long)who) - 1;
      int at = (int)(tile - first), x = 0, r0 = 0, r1 = 0;
      bool found = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int cnt = (int)(((uint32_t)(e[j] - b[j]) + BT - 1) / BT);
        const bool here = !found && at < cnt;
        x = here ? j : x;
        r0 = here ? b[j] + at * BT : r0;
        r1 = here ? min(e[j], b[j] + at * BT + BT) : r1;
        found |= here;
        at -= cnt;
      }
      out->expert = x0 + EPL * src + __builtin_amdgcn_readlane(x, src);
      out->r0 = __builtin_amdgcn_readlane(r0, src);
      out->r1 = __builtin_amdgcn_readlane(r1, src);
      out->col = (uint32_t)id - tile * ncol;
      return true;
    }
    before += all;
  }
  return false;
}

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

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
//   to LDS of the wave's own, a ring of CR chunks, pieces swizzled by
//   (channel / 4) % 4 for the same reason.  (Loaded to registers instead, 32
//   bytes per channel and load, they took the address unit twice the cycles.)
//   Scales: 8 bytes per channel and chunk to registers, one chunk ahead (on the
//   large tile two chunks at a time).
// What bounds it, by the rows per expert.  Many: the matrix cores, and with them
// the power: 16384 tokens x 8 of 256 experts 2048 x 4096 take 1.94 to 2.07 ms (1.1
// PFLOP/s), the cores busy two thirds of the cycles at 1.3 to 1.6 GHz, the
// expansion (2.5 vector operations a code) between the products; the library's
// dense product of as many flops takes 1.42 to 1.75 ms at 85 %.  Few: reading the
// codes: 64 tokens x 8 (122 to 156 experts in use, 140 on average: 663 MB) take
// 0.165 ms, 4.0 TB/s, the vector units busy half of it with the expansion.  Tried
// and slower there: smaller and wider tiles (64 x 64, 32 x 128, 32 x 256: 184 to
// 230 us against 185), other starting places in k for other tiles (208).  Tried
// and slower for many rows: 256 x 256 tiles on 8 waves and 256 rows on 4 (2.5 ms),
// 8 waves on 128 x 512 (equal), products in groups before their expansion (2.09
// ms), each product followed by its own (2.06 ms against 2.04 in the same run).
template <int NW, int RF, int CF, int CR>
struct Tile {
  static constexpr int kRows = 32 * RF, kCols = 32 * CF * NW;
  static constexpr int kXBuf = kRows * 128, kCBuf = CF * 32 * 64;   // bytes of one buffer (of a wave's codes)
  static constexpr int kXLoads = 4 * RF / NW, kCLoads = 2 * CF;     // copies per step, per chunk
  static constexpr int kLds = 3 * kXBuf + CR * NW * kCBuf;
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

// Copies q0 .. q1 - 1 of NL, each 1024 bytes to LDS (16 per lane), from `src` +
// off[q]; offsets at or past the bound bring zeros.
template <int NL, int STRIDE>
__device__ __forceinline__ void copy_lds(char* __restrict__ dst, const void* src, uint32_t bound, const uint32_t (&off)[NL],
                                         bool in, int q0 = 0, int q1 = NL) {
#if __HIP_DEVICE_COMPILE__
  __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, (short)0, bound, 0x00020000);
#pragma unroll
  for (int q = 0; q < NL; ++q)
    if (q >= q0 && q < q1)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + q * STRIDE), 16,
                                               in ? off[q] : 0xFFFFFFF0u, 0, 0, 0);
#endif
}

// What is copied for activations past the last input channel where X is FAR.
__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

// The same for rows of X, offsets in 16-byte pieces.  FAR: X has 2^32 bytes or
// more, which a buffer cannot span; the copies then go by 64-bit addresses.
template <int NL, int STRIDE, bool FAR>
__device__ __forceinline__ void copy_x(char* __restrict__ dst, const uint16_t* src, uint32_t bound, const uint32_t (&off)[NL],
                                       bool in, int q0 = 0, int q1 = NL) {
#if __HIP_DEVICE_COMPILE__
  if (FAR) {
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      if (q < q0 || q >= q1) continue;
      const void* p = in ? (const void*)((const char*)src + (uint64_t)off[q] * 16) : (const void*)&kZeros;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                       (__attribute__((address_space(3))) void*)(dst + q * STRIDE), 16, 0, 0);
    }
  } else {
    __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)src, (short)0, bound, 0x00020000);
#pragma unroll
    for (int q = 0; q < NL; ++q)
      if (q >= q0 && q < q1)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + q * STRIDE), 16,
                                                 in ? off[q] * 16 : 0xFFFFFFF0u, 0, 0, 0);
  }
#endif
}

// What a wave's steps share.
template <int NW, int RF, int CF, int CR>
struct Wave {
  uint32_t xoff[Tile<NW, RF, CF, CR>::kXLoads];   // its copies' offsets from X (16-byte pieces)
  uint32_t coff[Tile<NW, RF, CF, CR>::kCLoads];   // and from its codes (bytes)
  int xrd[4], crd[2];                         // LDS offsets of product j's row fragment, of step t's codes
  int h;
};

// Step T of a chunk: its four products on xb, the activations of two steps on
// into xd and (T = 0) the codes of CR - 1 chunks on into cd; cb and cn are
// this chunk's codes and the next's.  The buffers are distinct, which the restrict
// qualifiers state, so that reads need not wait for the copies in flight.
template <int NW, int RF, int CF, int CR, int T, bool SCALES, bool FAR>
__device__ __forceinline__ void product_step(const char* __restrict__ xb, const char* __restrict__ xn,
                                             char* __restrict__ xd, const char* __restrict__ cb,
                                             const char* __restrict__ cn, char* __restrict__ cd, const uint16_t* xsrc,
                                             uint32_t xbound, bool in, const uint8_t* csrc, uint32_t cbound,
                                             const Wave<NW, RF, CF, CR>& w, const u32x2 (&sc)[CF], const u32x2 (&sn)[CF],
                                             u32x4 (&cw)[CF], bf16x8 (&xa)[RF], u32x4 (&qa)[2][CF],
                                             f32x16 (&acc)[RF][CF]) {
  using TL = Tile<NW, RF, CF, CR>;
  constexpr int NX = TL::kXLoads, NC = TL::kCLoads;
  u32x4 cnext[CF];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = j & 1;
    if (j == 2) {
      // The next step's codes.  Behind those of the next chunk were issued, with
      // a ring of three, three steps' activations, one chunk's codes and one
      // chunk's scales; with a ring of two, this step's activations.
      if (T == 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(CR == 3 ? 3 * NX + NC + (SCALES ? CF : 0) : NX));
#pragma unroll
      for (int f = 0; f < CF; ++f)
        cnext[f] = *(const u32x4*)((T == 0 ? cb : CR == 3 ? cn : cd) + f * 2048 + w.crd[T ^ 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (j == 3) {
      // The next step's activations: behind them were issued this step's, one
      // chunk's codes and (in a chunk's first step) the next chunk's scales.
      // Every wave has read all of this step's buffer by now.
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(NX + NC + (T == 0 && SCALES ? CF : 0)));
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
      // The copies one by one between the products: issued together, they held
      // the wave at the full address queue (16384 tokens 2072 us instead of 1993).
      if (j == 0) copy_x<NX, NW * 1024, FAR>(xd, xsrc, xbound, w.xoff, in, i * NX / RF, (i + 1) * NX / RF);
      if (j == 1 && T == 0) copy_lds<NC, 1024>(cd, csrc, cbound, w.coff, true, i * NC / RF, (i + 1) * NC / RF);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int f = 0; f < CF; ++f) cw[f] = cnext[f];
}

// A wave's accumulators times g to rows [tl.r0, tl.r1) of out, channels from
// o0 on (below width); rows without a token as zeros.
// Accumulator: lane l, register r -> channel 8 (r / 4) + 4 h + r % 4, row c.
// 32 rows at a time go through LDS of the wave's own (what the workgroup held
// there is not needed behind the barrier), so that a row's channels leave in
// 16-byte pieces side by side: stored from the registers, 8 bytes per row,
// they took the 16384-token product 0.15 to 0.28 ms of 2.1.
template <int NW, int RF, int CF, int OUT_BF16, int LDS>
__device__ __forceinline__ void store_tile(char* smem, const f32x16 (&acc)[RF][CF], const RowTile& tl, float g,
                                           const int32_t* __restrict__ tok_idx, int64_t n, int64_t o0, int64_t width,
                                           void* __restrict__ out, int64_t ldo, bool vec_out) {
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
  asm volatile("s_barrier" ::: "memory");
  constexpr int ES = OUT_BF16 ? 2 : 4, ROW = 32 * CF * ES + 16, PR = 32 * CF * ES / 16;   // 16-byte pieces per row
  static_assert(NW * 32 * ROW <= LDS, "output staging");
  char* st = smem + wave * 32 * ROW;
#pragma unroll
  for (int i = 0; i < RF; ++i) {
    const int64_t row0 = tl.r0 + 32 * i, trow = row0 + c;
    const bool token = !tok_idx || trow >= tl.r1 || (tok_idx[trow] >= 0 && tok_idx[trow] < n);
#pragma unroll
    for (int f = 0; f < CF; ++f)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = token ? acc[i][f][4 * r4 + r] * g : 0.0f;
        char* p = st + c * ROW + (32 * f + 8 * r4 + 4 * h) * ES;
        if (OUT_BF16) {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          *(bf16x4*)p = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        } else {
          *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int q = 0; q < 32 * PR / 64; ++q) {
      const int e = q * 64 + lane, r = e / PR, piece = e % PR;
      const u32x4 v = *(const u32x4*)(st + r * ROW + piece * 16);
      const int64_t row = row0 + r, o = o0 + piece * (16 / ES);
      if (row >= tl.r1) continue;
      if (vec_out && o + 16 / ES <= width) {
        *(u32x4*)((char*)out + (row * ldo + o) * ES) = v;
      } else {
#pragma unroll
        for (int x = 0; x < 16 / ES; ++x)
          if (o + x < width) {
            if (OUT_BF16) ((uint16_t*)out)[row * ldo + o + x] = (uint16_t)(v[x >> 1] >> (16 * (x & 1)));
            else ((uint32_t*)out)[row * ldo + o + x] = v[x];
          }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Rows without a token (their number is outside [0, n)) read token 0's and
// are stored as zeros; rows behind the tile's last are zeros that nothing is
// fetched for (FAR: token 0's).
template <int NW, int RF, int CF, int CR, int OUT_BF16, bool FAR>
__device__ __forceinline__ void tile_product(char* smem, const RowTile& tl, const uint16_t* __restrict__ X, int64_t n,
                                             int64_t k, int64_t ldx, const int32_t* __restrict__ tok_idx,
                                             const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                             float g, int64_t m, void* __restrict__ Y, int64_t ldy, bool vec_out) {
  using TL = Tile<NW, RF, CF, CR>;
  constexpr int NX = TL::kXLoads, NC = TL::kCLoads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int64_t kb = k / 16;
  const int64_t o0 = tl.col * TL::kCols + wave * 32 * CF;
  Wave<NW, RF, CF, CR> w;
  w.h = h;

  // Copy q of a step brings rows 8 (NW q + wave) + lane / 8.
  const int xk = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 8;   // the lane's k in the step: its piece ^ (row / 2) % 8
#pragma unroll
  for (int q = 0; q < NX; ++q) {
    const int64_t r = tl.r0 + 8 * (NW * q + wave) + (lane >> 3);
    const int64_t t = r < tl.r1 ? (tok_idx ? tok_idx[r] : r) : 0;
    w.xoff[q] = (uint32_t)(((t >= 0 && t < n ? t : 0) * ldx + xk) / 8);
    if (!FAR && r >= tl.r1) w.xoff[q] = 0x0FFFFFFF;   // past the bound: zeros, nothing fetched
  }
  // Bytes of X from step st on (not FAR: below 2^32 - 256).
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
  char* cl = smem + 3 * TL::kXBuf + wave * CR * TL::kCBuf;
  char *c0 = cl, *c1 = cl + TL::kCBuf, *c2 = cl + (CR - 1) * TL::kCBuf;   // chunks ch, ch + 1, ch + CR - 1
  const int xw = wave * 1024;
  u32x2 sc[CF], sn[CF];
  u32x4 cw[CF], qa[2][CF];
  bf16x8 xa[RF];
  const int whole = (int)(k / 128), nchunks = (int)((k + 127) / 128);
  if (whole) load_scales<CF, false>(scales, srow, 8, sc);
  else load_scales<CF, true>(scales, srow, kb, sc);
  copy_lds<NC, 1024>(c0, codes, cbound(0), w.coff, true);
  copy_x<NX, NW * 1024, FAR>(x0 + xw, X, bound(0), w.xoff, inside(0));
  __builtin_amdgcn_sched_barrier(0);
  if (CR == 3) copy_lds<NC, 1024>(c1, codes + 64, cbound(1), w.coff, true);
  copy_x<NX, NW * 1024, FAR>(x1 + xw, X + 64, bound(1), w.xoff, inside(1));
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(CR == 3 ? NX + NC : NX));   // step 0's and chunk 0's have landed
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
  // second multiplies zeros.  SCALES: the caller has just issued CF scale loads.
  auto steps = [&]<bool INSIDE, bool SCALES>(int ch, const u32x2(&s0)[CF], const u32x2(&s1)[CF]) {
    const int64_t st = 2 * ch;
    product_step<NW, RF, CF, CR, 0, SCALES, FAR>(x0, x1, x2 + xw, c0, c1, c2, X + (st + 2) * 64, bound(st + 2), INSIDE || inside(st + 2),
                                      codes + (ch + CR - 1) * 64, cbound(ch + CR - 1), w, s0, s1, cw, xa, qa, acc);
    product_step<NW, RF, CF, CR, 1, SCALES, FAR>(x1, x2, x0 + xw, c0, c1, c2, X + (st + 3) * 64, bound(st + 3), INSIDE || inside(st + 3),
                                      codes, 0, w, s0, s1, cw, xa, qa, acc);
    char *x = x0, *cc = c0;
    x0 = x2;
    x2 = x1;
    x1 = x;
    c0 = c1;
    c1 = CR == 3 ? c2 : cc;
    c2 = cc;
  };
  auto chunk = [&]<bool WIDE>(int ch) {
    load_scales<CF, !WIDE>(scales + (ch + 1) * 8, srow, kb - 8 * (ch + 1), sn);
    __builtin_amdgcn_sched_barrier(0);
    steps.template operator()<WIDE, WIDE>(ch, sc, sn);
#pragma unroll
    for (int f = 0; f < CF; ++f) sc[f] = sn[f];
  };
  int ch = 0;
  // On the large tile pairs of chunks with another whole pair behind them, whose
  // scales come in one load per channel (16384 tokens 2006 us instead of 2036; the
  // 64 x 128 tile lost by the second loop: 36 us instead of 32 at 17 steps).
  if (CR == 2 && ch + 4 <= whole) {
    u32x2 sb[CF], ta[CF], tb[CF];
#pragma unroll
    for (int f = 0; f < CF; ++f) sb[f] = *(const u32x2_any*)(scales + srow[f] + 8);
    for (; ch + 4 <= whole; ch += 2) {
#pragma unroll
      for (int f = 0; f < CF; ++f) {
        const u32x4 v = *(const u32x4_any*)(scales + (ch + 2) * 8 + srow[f]);
        ta[f] = u32x2{v[0], v[1]};
        tb[f] = u32x2{v[2], v[3]};
      }
      __builtin_amdgcn_sched_barrier(0);
      steps.template operator()<true, true>(ch, sc, sb);
      steps.template operator()<true, false>(ch + 1, sb, ta);
#pragma unroll
      for (int f = 0; f < CF; ++f) {
        sc[f] = ta[f];
        sb[f] = tb[f];
      }
    }
  }
  for (; ch < whole - 1; ++ch) chunk.template operator()<true>(ch);
  for (; ch < nchunks; ++ch) chunk.template operator()<false>(ch);
  // (store_tile first waits for the copies issued for steps past the end, which
  // still write LDS.)
  store_tile<NW, RF, CF, OUT_BF16, TL::kLds>(smem, acc, tl, g, tok_idx, n, o0, m, Y, ldy, vec_out);
}

// Calls f with the number of 32-row blocks that hold rows of the tile, at most RF: a
// tile at an expert's end does not multiply the blocks it has no rows for.
template <int RF, typename F>
__device__ __forceinline__ void for_row_blocks(const RowTile& tl, F f) {
  if constexpr (RF > 1) {
    if (tl.r1 - tl.r0 <= 32 * (RF - 1)) {
      for_row_blocks<RF - 1>(tl, f);
      return;
    }
  }
  f.template operator()<RF>();
}

template <int NW, int RF, int CF, int CR, int OUT_BF16, bool FAR>
__global__ __launch_bounds__(64 * NW, 2) void grouped_gemm_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t k,
                                                                  int64_t ldx, const int32_t* __restrict__ tok_idx,
                                                                  int64_t rows, const int64_t* __restrict__ off,
                                                                  int64_t G, const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const float* __restrict__ gs, int64_t m,
                                                                  void* __restrict__ Y, int64_t ldy, int vec_out) {
  using TL = Tile<NW, RF, CF, CR>;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  RowTile tl;
  if (!find_tile<TL::kRows>(off, G, rows, (uint32_t)((m + TL::kCols - 1) / TL::kCols), &tl)) return;
  for_row_blocks<RF>(tl, [&]<int R>() {
    tile_product<NW, R, CF, CR, OUT_BF16, FAR>(smem, tl, X, n, k, ldx, tok_idx, codes + tl.expert * m * (k / 2),
                                          scales + tl.expert * m * (k / 16), gs[tl.expert], m, Y, ldy, vec_out != 0);
  });
}

// ---- few rows ---------------------------------------------------------------------
// A token's experts are so few tiles of the kernel above that most of the
// device would idle.  Here a workgroup of 8 waves takes 16 rows and 32 output
// channels, the waves share k in turn, in pairs of 128 k (whole 128-byte lines
// of codes), and nothing is staged: all of a pair's loads are issued ahead, the
// next pairs' while it is multiplied.
//   v_mfma_f32_16x16x32_bf16, A = 16 channels, B = 16 rows: lane (c = l % 16,
//   q = l / 16) takes the 32 consecutive k from 32 q of each 128, 8 per product
//   (16 bytes of codes and 2 scales per channel), of channel c and row c.
// Lanes without a row read the tile's last row's activations and are not
// stored.  The waves' partial sums are added in wave order through LDS.
// Bound by one pass of loads over a cold weight: 8 rows on 256 experts 2048 x
// 4096 read 38 MB in 13.7 us (2.8 TB/s).  Waves that each take their own channels
// over all of k instead: 251 us against 197 at 64 tokens.
constexpr int FW = 8, FROWS = 16, FCG = 2, FCOLS = 16 * FCG, FD = 2;
typedef float f32x4c __attribute__((ext_vector_type(4)));

struct FewPair {
  u32x4 w[2][FCG];
  uint32_t s[2][FCG];
};
struct FewX {
  u32x4 v[4];
};

template <int OUT_BF16>
__global__ __launch_bounds__(64 * FW, 4) void grouped_few_kernel(const uint16_t* __restrict__ X, int64_t n, int64_t k,
                                                                 int64_t ldx, const int32_t* __restrict__ tok_idx,
                                                                 int64_t rows, const int64_t* __restrict__ off,
                                                                 int64_t G, const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 const float* __restrict__ gs, int64_t m,
                                                                 void* __restrict__ Y, int64_t ldy) {
  __shared__ __attribute__((aligned(16))) float part[FW][FROWS][FCOLS + 4];
  RowTile tl;
  if (!find_tile<FROWS>(off, G, rows, (uint32_t)((m + FCOLS - 1) / FCOLS), &tl)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int64_t kb = k / 16, o0 = tl.col * FCOLS;
  codes += (tl.expert * m + o0) * (k / 2);
  scales += (tl.expert * m + o0) * kb;
  uint32_t crow[FCG], srow[FCG];   // the lane's channels from the tile's first (past m: the last one)
#pragma unroll
  for (int f = 0; f < FCG; ++f) {
    const int64_t o = min((int64_t)(16 * f + c), m - 1 - o0);
    crow[f] = (uint32_t)(o * (k / 2)) + 16 * q;
    srow[f] = (uint32_t)(o * kb) + 2 * q;
  }
  const int whole = (int)(k / 256);   // pairs of 128 k that k has
  auto load_pair = [&](int p, FewPair& x) {
    const uint8_t *cp = codes + (int64_t)p * 128, *sp = scales + (int64_t)p * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int f = 0; f < FCG; ++f) {
        x.w[u][f] = *(const u32x4_any*)(cp + 64 * u + crow[f]);
        x.s[u][f] = *(const u16_any*)(sp + 8 * u + srow[f]);
      }
  };
  const int mine = whole > wave ? (whole - wave + FW - 1) / FW : 0;   // the wave's i-th is wave + FW i
  FewPair buf[FD];
#pragma unroll
  for (int d = 0; d < FD; ++d)
    if (d < mine) load_pair(wave + FW * d, buf[d]);
  const int64_t row = min(tl.r0 + c, tl.r1 - 1);
  const int64_t t = tok_idx ? tok_idx[row] : row;
  const bool token = t >= 0 && t < n;
  const uint16_t* xrow = X + (token ? t : 0) * ldx + 32 * q;
  auto load_x = [&](int64_t k0, FewX& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x.v[j] = *(const u32x4*)(xrow + k0 + 8 * j);
  };
  f32x4c acc[FCG];
#pragma unroll
  for (int f = 0; f < FCG; ++f) acc[f] = f32x4c{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const u32x4 (&w)[FCG], const uint32_t (&s2)[FCG], const FewX& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < FCG; ++f) {
        const float s = j < 2 ? e4m3_byte<0>(s2[f]) : e4m3_byte<1>(s2[f]);
        const u32x4 qv{dq_byte<0>(w[f][j], s), dq_byte<1>(w[f][j], s), dq_byte<2>(w[f][j], s), dq_byte<3>(w[f][j], s)};
        acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, qv), __builtin_bit_cast(bf16x8, x.v[j]),
                                                         acc[f], 0, 0, 0);
      }
  };
  FewX xa, xb;
  auto k_of = [&](int i) { return 256 * (int64_t)(wave + FW * i); };
  // Multiplies pair i (its first half's activations are in xa), then loads pair i + FD in its place.
  auto stage = [&](int i, FewPair& p, bool more, bool ahead) {
    load_x(k_of(i) + 128, xb);
    __builtin_amdgcn_sched_barrier(0);
    multiply(p.w[0], p.s[0], xa);
    if (more) load_x(k_of(i + 1), xa);
    __builtin_amdgcn_sched_barrier(0);
    multiply(p.w[1], p.s[1], xb);
    if (ahead) load_pair(wave + FW * (i + FD), p);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (mine > 0) {
    load_x(k_of(0), xa);
    int i = 0;
    for (; i + 2 * FD <= mine; i += FD)
#pragma unroll
      for (int d = 0; d < FD; ++d) stage(i + d, buf[d], true, true);
    // fewer than 2 FD pairs left
#pragma unroll
    for (int d = 0; d < 2 * FD - 1; ++d)
      if (i + d < mine) stage(i + d, buf[d % FD], i + d + 1 < mine, i + d + FD < mine);
  }
  // The rest of k, less than a pair: blocks past k as zero codes under zero scales.
  FewPair cur;
  if (wave == whole % FW && (int64_t)whole * 256 < k) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k0 = (int64_t)whole * 256 + 128 * u, b0 = k0 / 16 + 2 * q;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xa.v[j] = k0 + 32 * q + 8 * j < k ? *(const u32x4*)(xrow + k0 + 8 * j) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int f = 0; f < FCG; ++f) {
        u32x2 lo{0u, 0u}, hi{0u, 0u};
        uint32_t s = 0;
        if (b0 < kb) {
          lo = *(const u32x2_any*)(codes + k0 / 2 + crow[f]);
          s = scales[k0 / 16 + srow[f]];
        }
        if (b0 + 1 < kb) {
          hi = *(const u32x2_any*)(codes + k0 / 2 + 8 + crow[f]);
          s |= (uint32_t)scales[k0 / 16 + 1 + srow[f]] << 8;
        }
        cur.w[u][f] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        cur.s[u][f] = s;
      }
      multiply(cur.w[u], cur.s[u], xa);
    }
  }
  // Accumulator register r of lane l: channel 4 q + r, row c.
#pragma unroll
  for (int f = 0; f < FCG; ++f) *(f32x4c*)&part[wave][c][16 * f + 4 * q] = acc[f];
  if (wave == 0 && q == 0) part[0][c][FCOLS] = token ? 1.0f : 0.0f;   // (in the padding)
  __syncthreads();
  const int r = tid / FCOLS, o = tid % FCOLS;
  static_assert(FROWS * FCOLS == 64 * FW, "one output per thread");
  if (tl.r0 + r >= tl.r1 || o0 + o >= m) return;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < FW; ++w) v += part[w][r][o];
  v = part[0][r][FCOLS] != 0.0f ? v * gs[tl.expert] : 0.0f;
  const int64_t at = (tl.r0 + r) * ldy + o0 + o;
  if (OUT_BF16) ((__bf16*)Y)[at] = (__bf16)v;
  else ((float*)Y)[at] = v;
}

// ---- the gradient of the rows ---------------------------------------------------
// dX[r] = g dY[r] Q: 32 RF rows x 32 CF NW input channels per workgroup, as
// above with the sum over m, in steps of 64.  A lane needs 8 codes of one input
// channel under 8 output channels, which lie in 8 rows of the matrix: the
// step's 64 m x 128 bytes of codes go to LDS as they are (16-byte pieces
// swizzled by (m / 2) % 8) and are read with ds_read_b64_tr_b4, which gives lane i of 16 the
// 16 nibbles of column i out of 16 rows of 16 (the width of a scale block).
// So of a step, product j = 2 u + v takes m = 32 u + 16 h + 8 v .. + 7, and a
// lane's 8 codes come under 8 different scales, which are staged transposed,
// [block][m].  dY's rows are copied like the activations when m and their
// stride are multiples of 8 (DMA), else through registers, zeros past m.
// Bound as the forward product: 4099 tokens x 6 of 64 experts 2048 x 2048 take
// 234 us (0.9 PFLOP/s), the matrix cores busy 45 %, the vector units (two scales
// per code pair) about as long.  8 waves on 256 x 256: 289 us against 276.
// The two weight formats differ in their scales alone.  F::kBlock: codes per
// scale.  A scale is staged as it is multiplied by: an E4M3 byte, or the bf16
// of an E8M0 byte (2^-127 is a bf16 below the normal range, NaN stays NaN).
// MXFP4's two bytes are converted where they are loaded, so that a step waits for
// each and, as loads return in order, for the copies ahead of it: 333 x 1004 x 1056
// takes 14 us for its four steps, 64 rows x 4096 x 4096 16.7 for four.
struct Nvfp4 {
  static constexpr int kBlock = 16, kBytes = 1;
  // Of the scales of 16 m, those of m = 8 v + 2 piece and the next.
  static __device__ __forceinline__ f32x2c pair(const u32x4 (&s)[1], int v, int piece) {
    const int w = (int)s[0][2 * v + (piece >> 1)];
    const f32x2c p = (piece & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true) : __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    return p;
  }
};
struct Mxfp4 {
  static constexpr int kBlock = 32, kBytes = 2;
  static __device__ __forceinline__ f32x2c pair(const u32x4 (&s)[2], int v, int piece) {
    const uint32_t w = s[v][piece];
    return f32x2c{__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
  }
  static __device__ __forceinline__ uint32_t bf16_of(uint32_t byte) { return byte == 0 ? 0x0040u : byte == 255 ? 0x7FC0u : byte << 7; }
};

template <int NW, int RF, int CF, typename F>
struct GradTile {
  static constexpr int kRows = 32 * RF, kCols = 32 * CF * NW, kStride = kCols / 2;   // bytes of codes per m
  static constexpr int kYBuf = kRows * 128, kCBuf = 64 * kStride, kSBuf = 64 * kCols / F::kBlock * F::kBytes;
  static constexpr int kYLoads = 4 * RF / NW, kCLoads = kCBuf / 1024 / NW;
  static constexpr int kLds = 3 * (kYBuf + kCBuf + kSBuf);
  static_assert(kStride == 128 && NW == 4, "the swizzle and the copies' shapes");
};

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ u32x2 read_tr4(const char* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i32x2*)p));
}
// Codes m, m + 1 (byte `piece` of word) under their scales.
__device__ __forceinline__ uint32_t dq_pair(uint32_t word, f32x2c s, int piece) {
  f32x2c v;
  switch (piece) {
    case 0: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 0); break;
    case 1: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 1); break;
    case 2: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 2); break;
    default: v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 3); break;
  }
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2c{v.x * s.x, v.y * s.y}, bf16x2c));
}

// The codes and scales of product pair u of a step, for CF groups of 32 channels.
template <int CF, typename F>
struct GradCodes {
  u32x2 w[CF];
  u32x4 s[CF][F::kBytes];
};
template <int CF, typename F>
__device__ __forceinline__ void read_grad_codes(const char* cb, const char* sb, int u, const int (&crd)[CF],
                                                const int (&srd)[CF], GradCodes<CF, F>& q) {
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    q.w[f] = read_tr4(cb + u * 4096 + crd[f]);
#pragma unroll
    for (int b = 0; b < F::kBytes; ++b) q.s[f][b] = *(const u32x4*)(sb + u * 32 * F::kBytes + srd[f] + 16 * b);
  }
}

// A thread's scales of a step to LDS, [block][m].
template <typename F>
__device__ __forceinline__ void store_scale(char* sw, uint32_t v) {
  if constexpr (F::kBytes == 1) {
#pragma unroll
    for (int b = 0; b < 4; ++b) sw[b * 64] = (char)(v >> (8 * b));
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) *(uint16_t*)(sw + b * 128) = (uint16_t)(v >> (16 * b));
  }
}

// A thread's part of one step's dY through registers (not DMA): RF pieces.
template <int RF>
struct GradRows {
  u32x4 v[RF];
};

// One step: its four products, the copies of two steps on, and to LDS what
// registers hold of the next step.  yb, cb, sb: this step's buffers, n: the
// next step's, d: two steps on; all distinct.
template <int NW, int RF, int CF, bool DMA, typename F>
__device__ __forceinline__ void gradient_step(const char* __restrict__ yb, const char* __restrict__ cb,
                                              const char* __restrict__ sb, const char* __restrict__ yn,
                                              const char* __restrict__ cn, const char* __restrict__ sn,
                                              char* __restrict__ yw, char* __restrict__ sw, char* __restrict__ yd,
                                              char* __restrict__ cd, const uint16_t* ysrc, uint32_t ybound,
                                              const uint8_t* csrc, uint32_t cbound,
                                              const uint32_t (&yoff)[GradTile<NW, RF, CF, F>::kYLoads],
                                              const uint32_t (&coff)[GradTile<NW, RF, CF, F>::kCLoads], bool in,
                                              const int (&yrd)[4], const int (&crd)[CF], const int (&srd)[CF],
                                              GradCodes<CF, F>& q, bf16x8 (&ya)[RF], u32x4 (&qa)[2][CF],
                                              f32x16 (&acc)[RF][CF], uint32_t& sreg, GradRows<RF>& yreg, auto load_next) {
  using TL = GradTile<NW, RF, CF, F>;
  constexpr int NY = DMA ? TL::kYLoads : 0, NC = TL::kCLoads;
  GradCodes<CF, F> q1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = j & 1;
    if (j == 0) {
      // What registers hold of the next step to LDS, then the loads of the step behind it.
      store_scale<F>(sw, sreg);
      if (!DMA)
#pragma unroll
        for (int r = 0; r < RF; ++r) *(u32x4*)(yw + r * NW * 1024) = yreg.v[r];
      read_grad_codes<CF, F>(cb, sb, 1, crd, srd, q1);
      __builtin_amdgcn_sched_barrier(0);
      load_next();
      __builtin_amdgcn_sched_barrier(0);
    }
    if (j == 3) {
      // The next step's copies: behind them were issued this step's.  The register loads
      // between them do not count: the compiler may put them under a branch, which a wave
      // without a row inside m skips.
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(NY + NC));
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      read_grad_codes<CF, F>(cn, sn, 0, crd, srd, q);
    }
#pragma unroll
    for (int i = 0; i < RF; ++i) {
#pragma unroll
      for (int f = 0; f < CF; ++f)
        acc[i][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, qa[p][f]), ya[i], acc[i][f], 0, 0, 0);
      ya[i] = j < 3 ? *(const bf16x8*)(yb + i * 4096 + yrd[(j + 1) & 3]) : *(const bf16x8*)(yn + i * 4096 + yrd[0]);
#pragma unroll
      for (int e = i * 4 * CF / RF; e < (i + 1) * 4 * CF / RF; ++e) {
        const int f = e / 4, piece = e % 4, v = (j + 1) & 1;
        // product j + 1: pair 0 or 1 of this step, or pair 0 of the next
        const GradCodes<CF, F>& c = j == 1 || j == 2 ? q1 : q;
        qa[p ^ 1][f][piece] = dq_pair(c.w[f][v], F::pair(c.s[f], v, piece), piece);
      }
      if (DMA && j == 0) copy_lds<TL::kYLoads, NW * 1024>(yd, ysrc, ybound, yoff, in, i * NY / RF, (i + 1) * NY / RF);
      if (j == 1) copy_lds<NC, NW * 1024>(cd, csrc, cbound, coff, true, i * NC / RF, (i + 1) * NC / RF);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <int NW, int RF, int CF, bool DMA, int OUT_BF16, typename F>
__device__ __forceinline__ void tile_gradient(char* smem, const RowTile& tl, const uint16_t* __restrict__ dY, int64_t m,
                                              int64_t lddy, const uint8_t* __restrict__ codes,
                                              const uint8_t* __restrict__ scales, float g, int64_t k,
                                              void* __restrict__ dX, int64_t lddx, bool vec_out) {
  using TL = GradTile<NW, RF, CF, F>;
  constexpr int NC = TL::kCLoads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 31, h = lane >> 5;
  const int64_t kb = k / F::kBlock;
  const int64_t t0 = tl.col * TL::kCols, o0 = t0 + wave * 32 * CF;   // the tile's and the wave's first channel

  // Copy q of a step: rows 8 (NW q + wave) + lane / 8 of dY (of the step's m for codes), 16-byte piece `piece`.
  const int piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4)), mk = 8 * piece;
  const int64_t rows = tl.r1 - tl.r0;
  dY += tl.r0 * lddy;
  uint32_t yoff[TL::kYLoads], coff[NC];
#pragma unroll
  for (int q = 0; q < TL::kYLoads; ++q)
    yoff[q] = 8 * (NW * q + wave) + (lane >> 3) < rows ? (uint32_t)((8 * (NW * q + wave) + (lane >> 3)) * lddy + mk) * 2
                                                       : 0xFFFFFFF0u;   // past the bound: zeros, nothing fetched
#pragma unroll
  for (int q = 0; q < NC; ++q) coff[q] = (uint32_t)((8 * (NW * q + wave) + (lane >> 3)) * (k / 2)) + 16 * piece;
  // Bytes from step st on, of the tile's rows (below 2^32: checked on the host) and of the expert's codes.
  auto ybound = [&](int64_t st) { return (uint32_t)max((int64_t)0, ((rows - 1) * lddy + m - 64 * st) * 2); };
  auto inside = [&](int64_t st) { return st * 64 + mk < m; };
  auto cbound = [&](int64_t st) {
    return (uint32_t)min(max((int64_t)0, (m - 64 * st) * (k / 2) - t0 / 2), (int64_t)0xFFFFFF00);
  };
  auto csrc = [&](int64_t st) { return codes + 64 * st * (k / 2) + t0 / 2; };
  // Scales: the thread brings 4 bytes to LDS, of SQ blocks of row tid / 4 of the step; zeros past m.
  constexpr int SQ = 4 / F::kBytes;
  const int sm = tid >> 2, sq = (tid & 3) * SQ;
  auto load_scale = [&](int64_t st) {
    const int64_t mm = st * 64 + sm, b0 = t0 / F::kBlock + sq;
    uint32_t v = 0;
    if (F::kBytes == 1 && kb % 4 == 0) {   // whole words inside the row
      const bool ok = mm < m && b0 < kb;
      v = *(const u32_any*)(scales + (ok ? mm * kb + b0 : 0));
      v = ok ? v : 0;
    } else {
#pragma unroll
      for (int b = 0; b < SQ; ++b) {
        const bool ok = mm < m && b0 + b < kb;
        const uint32_t x = scales[ok ? mm * kb + b0 + b : 0];
        if constexpr (F::kBytes == 1) v |= (ok ? x : 0) << (8 * b);
        else v |= (ok ? Mxfp4::bf16_of(x) : 0) << (16 * b);
      }
    }
    return v;
  };
  auto load_rows = [&](int64_t st, GradRows<RF>& y) {
#pragma unroll
    for (int q = 0; q < RF; ++q) {
      const int64_t r = 8 * (NW * q + wave) + (lane >> 3), mm = st * 64 + mk;
      const uint16_t* p = dY + min(r, rows - 1) * lddy + mm;
      y.v[q] = u32x4{0u, 0u, 0u, 0u};
      if (mm + 8 <= m) {
        y.v[q] = *(const u32x4_a2*)p;
      } else {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (mm + x < m) y.v[q][x >> 1] |= (uint32_t)p[x] << (16 * (x & 1));
      }
    }
  };

  int yrd[4], crd[CF], srd[CF];
#pragma unroll
  for (int j = 0; j < 4; ++j) yrd[j] = c * 128 + (((4 * (j >> 1) + 2 * h + (j & 1)) ^ ((c >> 1) & 7)) * 16);
#pragma unroll
  for (int f = 0; f < CF; ++f) {
    crd[f] = (16 * h + (lane & 15)) * 128 + ((wave * CF + f) ^ ((lane & 15) >> 1)) * 16 + 8 * (c >> 4);
    srd[f] = ((((wave * CF + f) * 32 + c) / F::kBlock) * 64 + 16 * h) * F::kBytes;
  }

  f32x16 acc[RF][CF];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int f = 0; f < CF; ++f)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][f][r] = 0.0f;

  // Steps st, st + 1, st + 2 in turn.
  char *y0 = smem, *y1 = y0 + TL::kYBuf, *y2 = y1 + TL::kYBuf;
  char *c0 = smem + 3 * TL::kYBuf, *c1 = c0 + TL::kCBuf, *c2 = c1 + TL::kCBuf;
  char *s0 = smem + 3 * (TL::kYBuf + TL::kCBuf), *s1 = s0 + TL::kSBuf, *s2 = s1 + TL::kSBuf;
  const int wo = wave * 1024, yo = wo + lane * 16, so = (sq * 64 + sm) * F::kBytes;
  const int nsteps = (int)((m + 63) / 64);
  GradRows<RF> yreg;
  uint32_t sreg = load_scale(0);
  if (!DMA) load_rows(0, yreg);
  store_scale<F>(s0 + so, sreg);
  if (!DMA)
#pragma unroll
    for (int q = 0; q < RF; ++q) *(u32x4*)(y0 + yo + q * NW * 1024) = yreg.v[q];
  sreg = load_scale(1);
  if (!DMA) load_rows(1, yreg);
  __builtin_amdgcn_sched_barrier(0);
  if (DMA) copy_lds<TL::kYLoads, NW * 1024>(y0 + wo, dY, ybound(0), yoff, inside(0));
  copy_lds<NC, NW * 1024>(c0 + wo, csrc(0), cbound(0), coff, true);
  __builtin_amdgcn_sched_barrier(0);
  if (DMA) copy_lds<TL::kYLoads, NW * 1024>(y1 + wo, dY + 64, ybound(1), yoff, inside(1));
  copy_lds<NC, NW * 1024>(c1 + wo, csrc(1), cbound(1), coff, true);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((DMA ? TL::kYLoads : 0) + NC));   // step 0's have landed
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  GradCodes<CF, F> q;
  u32x4 qa[2][CF];
  bf16x8 ya[RF];
  read_grad_codes<CF, F>(c0, s0, 0, crd, srd, q);
#pragma unroll
  for (int i = 0; i < RF; ++i) ya[i] = *(const bf16x8*)(y0 + i * 4096 + yrd[0]);
#pragma unroll
  for (int f = 0; f < CF; ++f)
#pragma unroll
    for (int p = 0; p < 4; ++p) qa[0][f][p] = dq_pair(q.w[f][0], F::pair(q.s[f], 0, p), p);

  for (int st = 0; st < nsteps; ++st) {
    gradient_step<NW, RF, CF, DMA, F>(y0, c0, s0, y1, c1, s1, y1 + yo, s1 + so, y2 + wo, c2 + wo, dY + 64 * (int64_t)(st + 2),
                                   ybound(st + 2), csrc(st + 2), cbound(st + 2), yoff, coff, inside(st + 2), yrd, crd, srd, q,
                                   ya, qa, acc, sreg, yreg, [&]() {
                                     sreg = load_scale(st + 2);
                                     if (!DMA) load_rows(st + 2, yreg);
                                   });
    char *y = y0, *cc = c0, *ss = s0;
    y0 = y1;
    y1 = y2;
    y2 = y;
    c0 = c1;
    c1 = c2;
    c2 = cc;
    s0 = s1;
    s1 = s2;
    s2 = ss;
  }
  store_tile<NW, RF, CF, OUT_BF16, TL::kLds>(smem, acc, tl, g, nullptr, 0, o0, k, dX, lddx, vec_out);
}

template <int NW, int RF, int CF, bool DMA, int OUT_BF16>
__global__ __launch_bounds__(64 * NW, 2) void grouped_dx_kernel(const uint16_t* __restrict__ dY, int64_t rows, int64_t m,
                                                                int64_t lddy, const int64_t* __restrict__ off, int64_t G,
                                                                const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales,
                                                                const float* __restrict__ gs, int64_t k,
                                                                void* __restrict__ dX, int64_t lddx, int vec_out) {
  using TL = GradTile<NW, RF, CF, Nvfp4>;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  RowTile tl;
  if (!find_tile<TL::kRows>(off, G, rows, (uint32_t)((k + TL::kCols - 1) / TL::kCols), &tl)) return;
  for_row_blocks<RF>(tl, [&]<int R>() {
    tile_gradient<NW, R, CF, DMA, OUT_BF16, Nvfp4>(smem, tl, dY, m, lddy, codes + tl.expert * m * (k / 2),
                                            scales + tl.expert * m * (k / 16), gs[tl.expert], k, dX, lddx, vec_out != 0);
  });
}

// The gradient of one MXFP4 matrix's product: row tiles without a search, in
// contiguous runs per XCD as above.  Where tiles are few, m is cut into `splits`
// parts of mper (a multiple of 64), each with a tile of its own, whose fp32 sums go
// to dX + part * rows * k (dX is then the workspace, mx_dx_sum_kernel adds them).
template <int NW, int RF, int CF, bool DMA, int OUT_BF16>
__global__ __launch_bounds__(64 * NW, 2) void mx_dx_kernel(const uint16_t* __restrict__ dY, int64_t rows, int64_t m,
                                                           int64_t lddy, const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t k,
                                                           void* __restrict__ dX, int64_t lddx, int vec_out, int64_t mper,
                                                           uint32_t splits) {
  using TL = GradTile<NW, RF, CF, Mxfp4>;
  __shared__ __attribute__((aligned(1024))) char smem[TL::kLds];
  const uint32_t ncol = (uint32_t)((k + TL::kCols - 1) / TL::kCols);
  const uint64_t all = (uint64_t)((rows + TL::kRows - 1) / TL::kRows) * ncol * splits, per = (all + 7) / 8;
  uint64_t id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || id >= all) return;
  const int64_t part = (uint32_t)id % splits, m0 = part * mper;
  id /= splits;
  const uint32_t tile = (uint32_t)id / ncol;   // (fewer than 2^31 workgroups)
  RowTile tl;
  tl.expert = 0;
  tl.col = (uint32_t)id - tile * ncol;
  tl.r0 = (int64_t)tile * TL::kRows;
  tl.r1 = min(rows, tl.r0 + TL::kRows);
  for_row_blocks<RF>(tl, [&]<int R>() {
    tile_gradient<NW, R, CF, DMA, OUT_BF16, Mxfp4>(smem, tl, dY + m0, min(mper, m - m0), lddy, codes + m0 * (k / 2),
                                                   scales + m0 * (k / 32), 1.0f, k,
                                                   (char*)dX + part * rows * k * (OUT_BF16 ? 2 : 4), lddx, vec_out != 0);
  });
}

// dX = the parts' sums, in their order; four columns per thread (k is a multiple of 32).
template <int OUT_BF16>
__global__ __launch_bounds__(256) void mx_dx_sum_kernel(const float* __restrict__ parts, int64_t rows, int64_t k, uint32_t splits,
                                                        void* __restrict__ dX, int64_t lddx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = k / 4;
  if (i >= rows * quads) return;
  const int64_t row = i / quads, col = 4 * (i - row * quads);
  f32x4 v = *(const f32x4*)(parts + 4 * i);
#pragma unroll 8
  for (uint32_t s = 1; s < splits; ++s) {
    const f32x4 p = *(const f32x4*)(parts + s * rows * k + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += p[e];
  }
  const int64_t at = row * lddx + col;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (OUT_BF16) ((__bf16*)dX)[at + e] = (__bf16)v[e];
    else ((float*)dX)[at + e] = v[e];
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
  const int vec = ldy % (out_bf16 ? 8 : 4) == 0 && (uintptr_t)Y % 16 == 0;
#define NVQ_LAUNCH(KERNEL, ROWS, COLS, THREADS, ...)                                                                 \
  do {                                                                                                               \
    const int64_t blocks = most_tiles(rows, G, ROWS, (m + (COLS)-1) / (COLS));                                       \
    if (blocks > kMaxThreads / (THREADS)) return kTooManyTiles;                                                      \
    hipLaunchKernelGGL((KERNEL), dim3((unsigned)blocks), dim3(THREADS), 0, s, X, n, k, ldx, tok_idx, rows, grp_off, G, \
                       codes, scales, g, m, Y, ldy __VA_OPT__(, ) __VA_ARGS__);                                      \
    return hipGetLastError();                                                                                        \
  } while (0)
#define NVQ_TILE(RF, CF, CR, FAR)                                                                               \
  do {                                                                                                          \
    using TL = Tile<4, RF, CF, CR>;                                                                             \
    if (out_bf16) NVQ_LAUNCH((grouped_gemm_kernel<4, RF, CF, CR, 1, FAR>), TL::kRows, TL::kCols, 256, vec);     \
    NVQ_LAUNCH((grouped_gemm_kernel<4, RF, CF, CR, 0, FAR>), TL::kRows, TL::kCols, 256, vec);                   \
  } while (0)
  const int64_t used = std::min(rows, G);   // the most experts that can have rows
  if (((n - 1) * ldx + k) * 2 >= 0xFFFFFF00) NVQ_TILE(4, 2, 2, true);
  // Times in us, few rows / 64 x 128 tiles / 128 x 256 tiles, measured for
  // layers of 8 to 256 experts, 1000 to 4096 outputs and 1024 to 4096 inputs.
  // Few rows: up to about one round of its workgroups on the device (512); 8 rows
  // on 256 experts 2048 x 4096 15 / 24 / 34, 16 rows 27 / 24 / 35; 12 rows on
  // 64 experts 2048 x 2048 13 / 14 / 20, 18 rows 16 / 15 / 20.
  if (most_tiles(rows, G, FROWS, (m + FCOLS - 1) / FCOLS) <= 768) {
    if (out_bf16) NVQ_LAUNCH(grouped_few_kernel<1>, FROWS, FCOLS, 64 * FW);
    NVQ_LAUNCH(grouped_few_kernel<0>, FROWS, FCOLS, 64 * FW);
  }
  // Large tiles: enough of them for the device, and experts that fill them; 64
  // experts 2048 x 2048 with 1536 rows - / 54 / 68, 4200 rows - / 82 / 78,
  // 24594 rows - / 280 / 214; 16 experts 4096 x 1024 with 1024 rows - / 22 / 29,
  // 2800 rows - / 42 / 34; 8 experts 1024 x 2048 with 3074 rows - / 25 / 32.
  if (rows >= 32 * used && most_tiles(rows, G, 128, (m + 255) / 256) >= 448) NVQ_TILE(4, 2, 2, false);
  NVQ_TILE(2, 1, 3, false);
#undef NVQ_TILE
#undef NVQ_LAUNCH
}

hipError_t nvfp4_gemm_grouped_dx_launch(const uint16_t* dY, int64_t rows, int64_t m, int64_t lddy,
                                        const int64_t* grp_off, int64_t G, const uint8_t* codes, const uint8_t* scales,
                                        const float* g, int64_t k, void* dX, int out_bf16, int64_t lddx,
                                        hipStream_t s) {
  const int vec = lddx % (out_bf16 ? 8 : 4) == 0 && (uintptr_t)dX % 16 == 0;
  const bool dma = m % 8 == 0 && lddy % 8 == 0 && (uintptr_t)dY % 16 == 0 && lddy < (1 << 23);
#define NVQ_DX(RF, DMA)                                                                                             \
  do {                                                                                                              \
    using TL = GradTile<4, RF, 2, Nvfp4>;                                                                                  \
    const int64_t blocks = most_tiles(rows, G, TL::kRows, (k + TL::kCols - 1) / TL::kCols);                         \
    if (blocks > kMaxThreads / 256) return kTooManyTiles;                                                           \
    if (out_bf16)                                                                                                   \
      hipLaunchKernelGGL((grouped_dx_kernel<4, RF, 2, DMA, 1>), dim3((unsigned)blocks), dim3(256), 0, s, dY, rows, m, \
                         lddy, grp_off, G, codes, scales, g, k, dX, lddx, vec);                                     \
    else                                                                                                            \
      hipLaunchKernelGGL((grouped_dx_kernel<4, RF, 2, DMA, 0>), dim3((unsigned)blocks), dim3(256), 0, s, dY, rows, m, \
                         lddy, grp_off, G, codes, scales, g, k, dX, lddx, vec);                                     \
  } while (0)
  // Rows per expert: 128-row tiles from 24 on, else 64.  us with 64 / 128, 8 rows a
  // token on 256 experts 2048 x 4096: 256 tokens (8 rows per expert) 324 / 387, 1024
  // tokens 500 / 499, 4096 tokens 942 / 788.
  const int64_t avg = rows / std::min(rows, G);
  if (avg >= 24) {
    if (dma) NVQ_DX(4, true);
    else NVQ_DX(4, false);
  } else {
    if (dma) NVQ_DX(2, true);
    else NVQ_DX(2, false);
  }
#undef NVQ_DX
  return hipGetLastError();
}

// Tiles of 128 or 64 rows x 256 columns, and parts of m: as many as give the
// device's 512 places a tile each, of at least four steps of 64, whose sums are at
// most 64 MiB.  (Without parts 64 rows x 28672 x 4096 took 518 us, with them 43.)
// (Parts of at least 128 / 256 / 512: 333 x 1004 x 1056 18.4 / 17.1 / 19.6 us, 16 x 4096 x 4096
// 17.7 / 15.1 / 17.6, 256 rows 30.8 / 31.0 / 28.4.)
// 128 rows where there are more than 512, or where more than 64 have parts of at
// least 1024 to share the expansion over.  us with 64 / 128 rows: 513 x 4096 x 4096 49 /
// 41, 2048 rows 105 / 93, 512 rows 42 / 47 (parts of 512), 256 rows 29 / 32, 512 x 14336 x
// 4096 108 / 88 (parts of 1792), 512 x 28672 x 4096 209 / 150, 333 x 1004 x 1056 17 / 24.
namespace {
struct DxSplit {
  int64_t height, mper, splits;
};
DxSplit dx_split(int64_t rows, int64_t m, int64_t k) {
  DxSplit d{128, 0, 0};
  for (;;) {
    const int64_t tiles = ((rows + d.height - 1) / d.height) * ((k + 255) / 256);
    const int64_t want = std::max<int64_t>(1, std::min({512 / tiles, (m + 255) / 256, (int64_t)(64 << 20) / (rows * k * 4)}));
    d.mper = ((m + want - 1) / want + 63) / 64 * 64;
    d.splits = (m + d.mper - 1) / d.mper;
    if (d.height == 64 || rows > 512 || (rows > 64 && d.mper >= 1024)) return d;
    d.height = 64;
  }
}
}  // namespace

size_t mxfp4_gemm_dx_split_workspace(int64_t rows, int64_t m, int64_t k) {
  const DxSplit d = dx_split(rows, m, k);
  return d.splits > 1 ? (size_t)d.splits * rows * k * 4 : 0;
}

hipError_t mxfp4_gemm_dx_launch(const uint16_t* dY, int64_t rows, int64_t m, int64_t lddy, const uint8_t* codes,
                                const uint8_t* scales, int64_t k, void* dX, int out_bf16, int64_t lddx, void* ws, hipStream_t s) {
  const DxSplit d = dx_split(rows, m, k);
  const bool split = d.splits > 1;
  void* to = split ? ws : dX;
  const int64_t ldo = split ? k : lddx;
  const int to_bf16 = split ? 0 : out_bf16;
  const int vec = ldo % (to_bf16 ? 8 : 4) == 0 && (uintptr_t)to % 16 == 0;
  const bool dma = m % 8 == 0 && lddy % 8 == 0 && (uintptr_t)dY % 16 == 0 && lddy < (1 << 23);
  const int64_t blocks = (((rows + d.height - 1) / d.height) * ((k + 255) / 256) * d.splits + 7) / 8 * 8;
  if (blocks > kMaxThreads / 256) return kTooManyTiles;
#define NVQ_DX_(RF, DMA, OUT)                                                                                               \
  hipLaunchKernelGGL((mx_dx_kernel<4, RF, 2, DMA, OUT>), dim3((unsigned)blocks), dim3(256), 0, s, dY, rows, m, lddy, codes, \
                     scales, k, to, ldo, vec, d.mper, (uint32_t)d.splits)
#define NVQ_DX(RF, DMA)                       \
  do {                                        \
    if (to_bf16) NVQ_DX_(RF, DMA, 1);         \
    else NVQ_DX_(RF, DMA, 0);                 \
  } while (0)
  if (d.height == 128) {
    if (dma) NVQ_DX(4, true);
    else NVQ_DX(4, false);
  } else {
    if (dma) NVQ_DX(2, true);
    else NVQ_DX(2, false);
  }
#undef NVQ_DX
#undef NVQ_DX_
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !split) return e;
  const dim3 grid((unsigned)((rows * (k / 4) + 255) / 256));
  if (out_bf16) hipLaunchKernelGGL((mx_dx_sum_kernel<1>), grid, dim3(256), 0, s, (const float*)ws, rows, k, (uint32_t)d.splits, dX, lddx);
  else hipLaunchKernelGGL((mx_dx_sum_kernel<0>), grid, dim3(256), 0, s, (const float*)ws, rows, k, (uint32_t)d.splits, dX, lddx);
  return hipGetLastError();
}

}  // namespace nvq
