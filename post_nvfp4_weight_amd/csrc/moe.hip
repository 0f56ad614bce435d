// The mixture-of-experts layer around its experts: the router's top-k choice,
// tokens sorted by expert, and the weighted sum of each token's experts, with
// the gradients of the first and the last.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace nvq {

namespace {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(uint16_t* p, float v) {
  const __bf16 b = (__bf16)v;   // nearest even, NaN kept
  *p = __builtin_bit_cast(uint16_t, b);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// ---- router -------------------------------------------------------------------
// One wave per token; lane l holds the EPL consecutive logits from l * EPL, so
// the lowest index among equal logits is in the lowest lane.  Each of the K
// rounds takes the wave's largest remaining logit, then the lowest lane and
// the lowest element of it that holds that value.  A -inf logit is never
// chosen; a row with a NaN or +inf is rejected.  Weights are a softmax with
// the row's largest logit subtracted, sums in fp32.
template <typename L, int EPL>
__global__ __launch_bounds__(256) void topk_kernel(const L* __restrict__ logits, int64_t T, int E, int64_t ld, int K,
                                                   int renorm, int32_t* __restrict__ ids,
                                                   float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const float ninf = -__builtin_inff();
  const L* row = logits + t * ld;
  float v[EPL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    v[i] = e < E ? load_f(row + e) : ninf;
    bad |= !(v[i] < __builtin_inff());
  }
  if (__ballot(bad)) {
    if (lane < K) {
      ids[t * K + lane] = -1;
      weights[t * K + lane] = __builtin_nanf("");
    }
    return;
  }
  float own = ninf;   // largest of the lane's remaining logits
#pragma unroll
  for (int i = 0; i < EPL; ++i) own = fmaxf(own, v[i]);
  float top = 0.0f, total = 0.0f, myval = ninf;
  int myid = -1;
  for (int s = 0; s < K; ++s) {
    const float best = wave_max(own);
    if (s == 0) {
      top = best == ninf ? 0.0f : best;
      if (!renorm) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) total += expf(v[i] - top);
        total = wave_sum(total);
      }
    }
    if (best == ninf) break;
    const int src = __ffsll((unsigned long long)__ballot(own == best)) - 1;
    int at = 0;
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i) at = v[i] == best ? i : at;
    const int id = __shfl(lane * EPL + at, src);
    if (lane == src) {
      own = ninf;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        v[i] = i == at ? ninf : v[i];
        own = fmaxf(own, v[i]);
      }
    }
    if (lane == s) {
      myval = best;
      myid = id;
    }
  }
  const float ex = expf(myval - top);   // 0 for a slot that no expert filled
  if (renorm) total = wave_sum(ex);
  if (lane < K) {
    ids[t * K + lane] = myid;
    weights[t * K + lane] = myid >= 0 ? ex / total : 0.0f;
  }
}

// Gradient of the router: with c = sum_s dw_s w_s, d logit_j is
// p_j (sum of dw_s over the slots with id j - c), p_j the softmax over all
// experts, or with renorm the same over the chosen experts only (w_s in the
// place of p_j).  One wave per token, lanes as in topk_kernel.
template <typename L, int EPL>
__global__ __launch_bounds__(256) void topk_backward_kernel(const L* __restrict__ logits, int64_t T, int E, int64_t ld,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ weights,
                                                            const float* __restrict__ dweights, int K, int renorm,
                                                            L* __restrict__ dlogits, int64_t ldd) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const int myid = lane < K ? ids[t * K + lane] : -1;
  const float myw = lane < K ? weights[t * K + lane] : 0.0f;
  const float mydw = lane < K ? dweights[t * K + lane] : 0.0f;
  // a rejected row (ids -1) has NaN weights, and so a NaN gradient; an empty one has none
  const bool taken = myid >= 0 && myid < E;
  const float c = wave_sum(lane < K && (taken || !(myw == 0.0f)) ? mydw * myw : 0.0f);
  float p[EPL], d[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) d[i] = 0.0f;
  if (renorm) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = c != c ? c : 0.0f;
  } else {
    float top = -__builtin_inff(), total = 0.0f;
    const L* row = logits + t * ld;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      p[i] = e < E ? load_f(row + e) : -__builtin_inff();
      top = fmaxf(top, p[i]);
    }
    top = wave_max(top);
    top = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += p[i] = expf(p[i] - top);
    total = wave_sum(total);
    const float r = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= r;
  }
  for (int s = 0; s < K; ++s) {
    const int id = __shfl(myid, s);
    const float w = __shfl(myw, s), dw = __shfl(mydw, s);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (id == lane * EPL + i) {
        if (renorm) d[i] += w * (dw - c);
        else d[i] += dw;
      }
  }
  L* out = dlogits + t * ldd;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (e < E) store_f(out + e, renorm ? d[i] + p[i] : p[i] * (d[i] - c));
  }
}

// ---- tokens sorted by expert -----------------------------------------------------
// A stable counting sort.  Assignment i (token i / K, slot i % K) goes to row
// base(expert) + the number of earlier assignments of that expert.  Blocks
// take consecutive chunks of SORT_CHUNK assignments, the waves of a block
// consecutive parts of its chunk; ranks inside 64 assignments come from ballots
// over the bits of the expert number, so nothing depends on timing.
constexpr int SORT_T = 1024, SORT_W = SORT_T / 64, SORT_CHUNK = 4096;

// LDS counts cnt[w][e] of wave w's part [b, e) of the assignments.
__device__ __forceinline__ void sort_count(const int32_t* ids, int64_t beg, int64_t end, int E, int* cnt) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < SORT_W * E; i += SORT_T) cnt[i] = 0;
  __syncthreads();
  for (int64_t i = beg + lane; i < end; i += 64) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)E) atomicAdd(cnt + wave * E + id, 1);   // integer counts: no order
  }
  __syncthreads();
}

// Exclusive sum of v over the SORT_T threads of the block; *total the whole sum.
__device__ __forceinline__ int block_exclusive(int v, int* part, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) part[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < SORT_W; ++w) {
    before += w < wave ? part[w] : 0;
    all += part[w];
  }
  *total = all;
  return before + x - v;
}

// cnt[w][e] holds the row of wave w's next assignment of expert e.
__device__ __forceinline__ void sort_place(const int32_t* ids, int64_t beg, int64_t end, int K, int E, int* cnt,
                                           int32_t* tok_idx, int32_t* pos) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  int* base = cnt + wave * E;
  for (int64_t i0 = beg; i0 < end; i0 += 64) {
    const int64_t i = i0 + lane;
    int id = i < end ? ids[i] : -1;
    const bool ok = (unsigned)id < (unsigned)E;
    if (!ok) id = 0;
    unsigned long long same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long m = __ballot((id >> b) & 1);
      same &= ((id >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    int row = -1;
    if (ok) row = base[id] + rank;
    // Every lane has read its base before one lane per expert moves it on, and
    // reads it anew in the next turn (LDS operations of a wave run in order).
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (ok && rank == 0) base[id] += __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i < end) {
      pos[i] = row;
      if (ok) tok_idx[row] = (int32_t)(i / K);
    }
  }
}

__device__ __forceinline__ void wave_part(int64_t beg, int64_t end, int64_t* b, int64_t* e) {
  const int64_t n = end - beg;
  const int64_t per = ((n + SORT_W - 1) / SORT_W + 63) / 64 * 64;
  const int wave = threadIdx.x >> 6;
  *b = std::min<int64_t>(end, beg + wave * per);
  *e = std::min<int64_t>(end, *b + per);
}

// Few assignments: one workgroup does it all.
__global__ __launch_bounds__(SORT_T) void sort_small_kernel(const int32_t* __restrict__ ids, int64_t n, int K, int E,
                                                            int32_t* __restrict__ tok_idx, int64_t* __restrict__ grp_off,
                                                            int32_t* __restrict__ pos) {
  extern __shared__ int cnt[];   // SORT_W * E
  __shared__ int part[SORT_W];
  int64_t b, e;
  wave_part(0, n, &b, &e);
  sort_count(ids, b, e, E, cnt);
  const int x = threadIdx.x;
  int mine = 0, total;
  if (x < E)
    for (int w = 0; w < SORT_W; ++w) mine += cnt[w * E + x];
  int run = block_exclusive(mine, part, &total);
  if (x < E) {
    grp_off[x] = run;
    for (int w = 0; w < SORT_W; ++w) {
      const int c = cnt[w * E + x];
      cnt[w * E + x] = run;
      run += c;
    }
  }
  if (x == 0) grp_off[E] = total;
  __syncthreads();
  sort_place(ids, b, e, K, E, cnt, tok_idx, pos);
  for (int64_t i = total + x; i < n; i += SORT_T) tok_idx[i] = -1;
}

// Many: counts of each chunk [nb][E] ...
__global__ __launch_bounds__(SORT_T) void sort_hist_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                           int32_t* __restrict__ hist) {
  extern __shared__ int cnt[];   // E
  for (int i = threadIdx.x; i < E; i += SORT_T) cnt[i] = 0;
  __syncthreads();
  const int64_t beg = (int64_t)blockIdx.x * SORT_CHUNK, end = std::min<int64_t>(n, beg + SORT_CHUNK);
  for (int64_t i = beg + threadIdx.x; i < end; i += SORT_T) {
    const int id = ids[i];
    if ((unsigned)id < (unsigned)E) atomicAdd(cnt + id, 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += SORT_T) hist[(int64_t)blockIdx.x * E + i] = cnt[i];
}

// ... their exclusive sums over the chunks in place, and each expert's total
// (64 experts per workgroup, each wave a range of chunks) ...
__global__ __launch_bounds__(SORT_T) void sort_scan_kernel(int32_t* __restrict__ hist, int nb, int E,
                                                           int32_t* __restrict__ total) {
  __shared__ int sum[SORT_W][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (nb + SORT_W - 1) / SORT_W;
  const int b0 = std::min(nb, wave * per), b1 = std::min(nb, b0 + per);
  int s = 0;
  if (e < E)
    for (int b = b0; b < b1; ++b) s += hist[(int64_t)b * E + e];
  sum[wave][lane] = s;
  __syncthreads();
  int run = 0, all = 0;
  for (int w = 0; w < SORT_W; ++w) {
    run += w < wave ? sum[w][lane] : 0;
    all += sum[w][lane];
  }
  if (e >= E) return;
  for (int b = b0; b < b1; ++b) {
    const int c = hist[(int64_t)b * E + e];
    hist[(int64_t)b * E + e] = run;
    run += c;
  }
  if (wave == 0) total[e] = all;
}

// ... and the rows.
__global__ __launch_bounds__(SORT_T) void sort_place_kernel(const int32_t* __restrict__ ids, int64_t n, int K, int E,
                                                            const int32_t* __restrict__ hist,
                                                            const int32_t* __restrict__ total,
                                                            int32_t* __restrict__ tok_idx,
                                                            int64_t* __restrict__ grp_off, int32_t* __restrict__ pos) {
  extern __shared__ int cnt[];   // SORT_W * E
  __shared__ int part[SORT_W];
  const int64_t beg = (int64_t)blockIdx.x * SORT_CHUNK, end = std::min<int64_t>(n, beg + SORT_CHUNK);
  int64_t b, e;
  wave_part(beg, end, &b, &e);
  sort_count(ids, b, e, E, cnt);
  const int x = threadIdx.x;
  int all;
  const int off = block_exclusive(x < E ? total[x] : 0, part, &all);
  if (x < E) {
    int run = off + hist[(int64_t)blockIdx.x * E + x];
    for (int w = 0; w < SORT_W; ++w) {
      const int c = cnt[w * E + x];
      cnt[w * E + x] = run;
      run += c;
    }
    if (blockIdx.x == 0) grp_off[x] = off;
  }
  if (blockIdx.x == 0 && x == 0) grp_off[E] = all;
  __syncthreads();
  sort_place(ids, b, e, K, E, cnt, tok_idx, pos);
  for (int64_t i = beg + x; i < end; i += SORT_T)
    if (i >= all) tok_idx[i] = -1;
}

// ---- a token's experts summed ------------------------------------------------------
template <typename Y, typename O>
__global__ __launch_bounds__(256) void combine_kernel(const Y* __restrict__ y, int64_t rows, int64_t d, int64_t ldy,
                                                      const int32_t* __restrict__ pos, const float* __restrict__ w,
                                                      int64_t T, int K, O* __restrict__ out, int64_t ldo) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x)
    for (int64_t c = threadIdx.x; c < d; c += 256) {
      float s = 0.0f;
      for (int j = 0; j < K; ++j) {
        const int64_t r = pos[t * K + j];
        const float v = (uint64_t)r < (uint64_t)rows ? load_f(y + r * ldy + c) : 0.0f;
        s = fmaf(w ? w[t * K + j] : 1.0f, v, s);
      }
      store_f(out + t * ldo + c, s);
    }
}

template <typename G, typename Y>
__global__ __launch_bounds__(256) void combine_backward_kernel(const G* __restrict__ dout, int64_t T, int64_t d,
                                                               int64_t ldd, const Y* __restrict__ y, int64_t rows,
                                                               int64_t ldy, const int32_t* __restrict__ pos,
                                                               const float* __restrict__ w, int K, Y* __restrict__ dy,
                                                               int64_t lddy, float* __restrict__ dw) {
  __shared__ float part[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t i = blockIdx.x; i < T * K; i += gridDim.x) {
    const int64_t t = i / K, r = pos[i];
    const bool ok = (uint64_t)r < (uint64_t)rows;
    const float wt = w ? w[i] : 1.0f;
    float s = 0.0f;
    if (ok)
      for (int64_t c = threadIdx.x; c < d; c += 256) {
        const float g = load_f(dout + t * ldd + c);
        if (dw) s = fmaf(g, load_f(y + r * ldy + c), s);
        if (dy) store_f(dy + r * lddy + c, wt * g);
      }
    if (dw) {
      s = wave_sum(s);
      if (lane == 0) part[wave] = s;
      __syncthreads();
      if (threadIdx.x == 0) dw[i] = part[0] + part[1] + part[2] + part[3];
      __syncthreads();
    }
  }
}

template <typename L>
hipError_t topk_run(const L* logits, int64_t T, int E, int64_t ld, int K, int renorm, int32_t* ids, float* weights,
                    hipStream_t s) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  const int epl = (E + 63) / 64;
  if (epl <= 1) hipLaunchKernelGGL((topk_kernel<L, 1>), grid, block, 0, s, logits, T, E, ld, K, renorm, ids, weights);
  else if (epl <= 2) hipLaunchKernelGGL((topk_kernel<L, 2>), grid, block, 0, s, logits, T, E, ld, K, renorm, ids, weights);
  else if (epl <= 4) hipLaunchKernelGGL((topk_kernel<L, 4>), grid, block, 0, s, logits, T, E, ld, K, renorm, ids, weights);
  else if (epl <= 8) hipLaunchKernelGGL((topk_kernel<L, 8>), grid, block, 0, s, logits, T, E, ld, K, renorm, ids, weights);
  else hipLaunchKernelGGL((topk_kernel<L, 16>), grid, block, 0, s, logits, T, E, ld, K, renorm, ids, weights);
  return hipGetLastError();
}

template <typename L>
hipError_t topk_backward_run(const L* logits, int64_t T, int E, int64_t ld, const int32_t* ids, const float* w,
                             const float* dw, int K, int renorm, L* dl, int64_t ldd, hipStream_t s) {
  const dim3 grid((unsigned)((T + 3) / 4)), block(256);
  const int epl = (E + 63) / 64;
  if (epl <= 1) hipLaunchKernelGGL((topk_backward_kernel<L, 1>), grid, block, 0, s, logits, T, E, ld, ids, w, dw, K, renorm, dl, ldd);
  else if (epl <= 2) hipLaunchKernelGGL((topk_backward_kernel<L, 2>), grid, block, 0, s, logits, T, E, ld, ids, w, dw, K, renorm, dl, ldd);
  else if (epl <= 4) hipLaunchKernelGGL((topk_backward_kernel<L, 4>), grid, block, 0, s, logits, T, E, ld, ids, w, dw, K, renorm, dl, ldd);
  else if (epl <= 8) hipLaunchKernelGGL((topk_backward_kernel<L, 8>), grid, block, 0, s, logits, T, E, ld, ids, w, dw, K, renorm, dl, ldd);
  else hipLaunchKernelGGL((topk_backward_kernel<L, 16>), grid, block, 0, s, logits, T, E, ld, ids, w, dw, K, renorm, dl, ldd);
  return hipGetLastError();
}

int64_t sort_blocks(int64_t n) { return (n + SORT_CHUNK - 1) / SORT_CHUNK; }
constexpr int64_t kSortSmall = 16384;   // assignments up to which one workgroup sorts

}  // namespace

hipError_t moe_topk_launch(const void* logits, int bf16, int64_t T, int64_t E, int64_t ld, int K, int renorm,
                           int32_t* ids, float* weights, hipStream_t s) {
  return bf16 ? topk_run((const uint16_t*)logits, T, (int)E, ld, K, renorm, ids, weights, s)
              : topk_run((const float*)logits, T, (int)E, ld, K, renorm, ids, weights, s);
}

hipError_t moe_topk_backward_launch(const void* logits, int bf16, int64_t T, int64_t E, int64_t ld, const int32_t* ids,
                                    const float* weights, const float* dweights, int K, int renorm, void* dlogits,
                                    int64_t ldd, hipStream_t s) {
  return bf16 ? topk_backward_run((const uint16_t*)logits, T, (int)E, ld, ids, weights, dweights, K, renorm,
                                  (uint16_t*)dlogits, ldd, s)
              : topk_backward_run((const float*)logits, T, (int)E, ld, ids, weights, dweights, K, renorm,
                                  (float*)dlogits, ldd, s);
}

size_t moe_sort_workspace(int64_t n, int64_t E) {
  return n <= kSortSmall ? 0 : (size_t)(sort_blocks(n) + 1) * E * sizeof(int32_t);
}

hipError_t moe_sort_launch(const int32_t* ids, int64_t n, int K, int64_t E, int32_t* tok_idx, int64_t* grp_off,
                           int32_t* pos, void* ws, hipStream_t s) {
  const size_t lds = (size_t)SORT_W * E * sizeof(int);
  if (n <= kSortSmall) {
    hipLaunchKernelGGL(sort_small_kernel, dim3(1), dim3(SORT_T), lds, s, ids, n, K, (int)E, tok_idx, grp_off, pos);
    return hipGetLastError();
  }
  const int nb = (int)sort_blocks(n);
  int32_t* hist = (int32_t*)ws;
  int32_t* total = hist + (int64_t)nb * E;
  hipLaunchKernelGGL(sort_hist_kernel, dim3(nb), dim3(SORT_T), E * sizeof(int), s, ids, n, (int)E, hist);
  hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)((E + 63) / 64)), dim3(SORT_T), 0, s, hist, nb, (int)E, total);
  hipLaunchKernelGGL(sort_place_kernel, dim3(nb), dim3(SORT_T), lds, s, ids, n, K, (int)E, hist, total, tok_idx, grp_off,
                     pos);
  return hipGetLastError();
}

hipError_t moe_combine_launch(const void* Y, int y_bf16, int64_t rows, int64_t d, int64_t ldy, const int32_t* pos,
                              const float* weights, int64_t T, int K, void* out, int out_bf16, int64_t ldo,
                              hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(T, 1 << 20)), block(256);
#define NVQ_COMBINE(YT, OT)                                                                                    \
  hipLaunchKernelGGL((combine_kernel<YT, OT>), grid, block, 0, s, (const YT*)Y, rows, d, ldy, pos, weights, T, K, \
                     (OT*)out, ldo)
  if (y_bf16) {
    if (out_bf16) NVQ_COMBINE(uint16_t, uint16_t);
    else NVQ_COMBINE(uint16_t, float);
  } else {
    if (out_bf16) NVQ_COMBINE(float, uint16_t);
    else NVQ_COMBINE(float, float);
  }
#undef NVQ_COMBINE
  return hipGetLastError();
}

hipError_t moe_combine_backward_launch(const void* dout, int dout_bf16, int64_t T, int64_t d, int64_t ldd, const void* Y,
                                       int y_bf16, int64_t rows, int64_t ldy, const int32_t* pos, const float* weights,
                                       int K, void* dY, int64_t lddy, float* dw, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(T * K, 1 << 20)), block(256);
#define NVQ_COMBINE_BWD(GT, YT)                                                                                  \
  hipLaunchKernelGGL((combine_backward_kernel<GT, YT>), grid, block, 0, s, (const GT*)dout, T, d, ldd, (const YT*)Y, \
                     rows, ldy, pos, weights, K, (YT*)dY, lddy, dw)
  if (dout_bf16) {
    if (y_bf16) NVQ_COMBINE_BWD(uint16_t, uint16_t);
    else NVQ_COMBINE_BWD(uint16_t, float);
  } else {
    if (y_bf16) NVQ_COMBINE_BWD(float, uint16_t);
    else NVQ_COMBINE_BWD(float, float);
  }
#undef NVQ_COMBINE_BWD
  return hipGetLastError();
}

}  // namespace nvq
