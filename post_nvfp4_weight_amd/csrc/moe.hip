// The mixture-of-experts layer around its experts: the router's top-k choice,
// tokens sorted by expert, and the weighted sum of each token's experts, with
// the gradients of the first and the last.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "router.h"

namespace nvq {

namespace {

template <typename L, int LPT, int EPL, int SORTED>
__global__ __launch_bounds__(256) void topk_kernel(const L* __restrict__ logits, int64_t T, int E, int64_t ld, int K,
                                                   int renorm, int32_t* __restrict__ ids,
                                                   float* __restrict__ weights) {
  const int lane = threadIdx.x % LPT;
  const int64_t t = (int64_t)blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  const int64_t row = t < T ? t : T - 1;   // lanes without a token repeat the last one and write nothing
  int32_t id;
  float w;
  route_token<L, LPT, EPL, SORTED>(logits + row * ld, E, K, renorm, lane, id, w);
  if (lane < K && t < T) {
    ids[t * K + lane] = id;
    weights[t * K + lane] = w;
  }
}

// Gradient of the router: with c = sum_s dw_s w_s, d logit_j is
// p_j (sum of dw of the slots with id j - c), p_j the softmax over all experts,
// or with renorm the sum of w_s (dw_s - c) of the slots with id j.  LPT lanes
// per token as in topk_kernel; the slots' terms reach their experts' lanes
// through a row of LDS (one addition per slot, lanes of one instruction in order).
template <typename L, int LPT, int EPL>
__global__ __launch_bounds__(256) void topk_backward_kernel(const L* __restrict__ logits, int64_t T, int E, int64_t ld,
                                                            const int32_t* __restrict__ ids,
                                                            const float* __restrict__ weights,
                                                            const float* __restrict__ dweights, int K, int renorm,
                                                            L* __restrict__ dlogits, int64_t ldd) {
  using R = RowLayout<L, LPT, EPL>;
  __shared__ __attribute__((aligned(16))) float term[256 / LPT][LPT * EPL];
  const int lane = threadIdx.x % LPT;
  const int64_t t = (int64_t)blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  if (t >= T) return;   // whole groups; nothing below crosses them
  float* mine = term[threadIdx.x / LPT];
  const int myid = lane < K ? ids[t * K + lane] : -1;
  const float myw = lane < K ? weights[t * K + lane] : 0.0f;
  const float mydw = lane < K ? dweights[t * K + lane] : 0.0f;
  // a rejected row (ids -1) has NaN weights, and so a NaN gradient; an empty slot has none
  const bool taken = myid >= 0 && myid < E;
  const float c = group_sum<LPT>(taken || myw != 0.0f ? mydw * myw : 0.0f);
#pragma unroll
  for (int i = 0; i < EPL; ++i) mine[i * LPT + lane] = 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // a group is part of one wave, whose LDS operations run in order
  if (taken) atomicAdd(mine + myid, renorm ? myw * (mydw - c) : mydw);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float p[EPL], total = 0.0f, top = 0.0f;
  if (!renorm) {
    load_row<L, LPT, EPL>(logits + t * ld, E, lane, p);
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) own = max(own, order_key(p[i]));   // (a NaN comes out as NaN, or meets one in c)
    top = key_value(group_max<LPT>(own));
    top = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < EPL; ++i) total += p[i] = expf(p[i] - top);
    total = group_sum<LPT>(total);
    total = total == 0.0f ? 1.0f : total;
  }
  L* out = dlogits + t * ldd;
#pragma unroll
  for (int v = 0; v < EPL / R::VW; ++v) {
    const int e0 = R::index(lane, v * R::VW);
    float r[R::VW];
#pragma unroll
    for (int i = 0; i < R::VW; ++i) {
      const float d = mine[e0 + i];
      r[i] = renorm ? (c != c ? c : d) : p[v * R::VW + i] / total * (d - c);
    }
    if (e0 + R::VW <= E) {
      typedef L Vec __attribute__((ext_vector_type(R::VW), aligned(sizeof(L))));
      Vec x;
#pragma unroll
      for (int i = 0; i < R::VW; ++i) {
        L y;
        store_f(&y, r[i]);
        x[i] = y;
      }
      *(Vec*)(out + e0) = x;
    } else {
#pragma unroll
      for (int i = 0; i < R::VW; ++i)
        if (e0 + i < E) store_f(out + e0 + i, r[i]);
    }
  }
}

// ---- tokens sorted by expert -----------------------------------------------------
// A stable counting sort.  Assignment i (token i / K, slot i % K) goes to row
// base(expert) + the number of earlier assignments of that expert.  Blocks
// take consecutive chunks of assignments, the waves of a block consecutive
// parts of its chunk, 64 at a time; ranks inside 64 come from ballots over the
// bits of the expert number, so nothing depends on timing.
// Few assignments: one workgroup and launch.  Many: counts per chunk, their
// sums, and the rows, three launches.  A chunk's rows are first sorted in LDS
// and leave in runs per expert: written one by one, 4 bytes each, they took
// the last launch 15.5 us instead of 12.5 (2^21 assignments, 256 experts).
// Bound at that size by the ballots' instructions: 20 us over all, of which the
// 25 MB would take 5; up to 2^16 by the launches' own 11 us.
constexpr int SORT_T = 1024, SORT_W = SORT_T / 64;

// i / K for 0 <= i < 2^31 as a multiplication: with s = ceil(log2 K) and
// mul = ceil(2^(31 + s) / K), i mul / 2^(31 + s) exceeds i / K by less than
// i / 2^(31 + s) < 1 / K, which never reaches the next whole number.
struct DivK {
  uint32_t mul, shift;
};
DivK div_by(uint32_t k) {
  DivK d{0, 0};
  while (((uint64_t)1 << d.shift) < k) ++d.shift;
  d.mul = (uint32_t)((((uint64_t)1 << (31 + d.shift)) + k - 1) / k);
  return d;
}
__device__ __forceinline__ int32_t div_k(int64_t i, DivK d) { return (int32_t)(__umulhi(2 * (uint32_t)i, d.mul) >> d.shift); }

// Inclusive sum over the wave's lanes (row shifts, then the rows' last lanes to the rows behind).
__device__ __forceinline__ int wave_inclusive(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Exclusive sums of N values per expert over the threads x < E (thread = expert),
// in place, and the whole sums in total; the waves past E only join the barrier.
template <int N>
__device__ __forceinline__ void expert_sums(int E, int (&v)[N], int (&total)[N], int (*part)[SORT_W]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = (E + 63) / 64;
  int incl[N];
  if (wave < nw) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      incl[i] = wave_inclusive(v[i]);
      if (lane == 63) part[i][wave] = incl[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) total[i] = 0;
  int before[N] = {};
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = part[i][w];
      before[i] += w < wave ? p : 0;
      total[i] += p;
    }
  if (wave < nw) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = before[i] + incl[i] - v[i];
  }
}

// Loads the wave's part of a chunk that starts at beg and ends before end (n of
// the call at most): assignment 64 u + lane of the part in id[u], -1 for none;
// and counts it per expert into cnt[wave][e] (LDS).
template <int PER>
__device__ __forceinline__ void sort_count(const int32_t* __restrict__ ids, int64_t beg, int64_t end, int E, int* cnt,
                                           int (&id)[PER]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t i = beg + (wave * PER + u) * 64 + lane;
    const int x = i < end ? ids[i] : -1;
    id[u] = (unsigned)x < (unsigned)E ? x : -1;
  }
  for (int i = threadIdx.x; i < SORT_W * E; i += SORT_T) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if (id[u] >= 0) atomicAdd(cnt + wave * E + id[u], 1);   // integer counts: no order
  __syncthreads();
}

// Of the thread's expert: the counts of the waves, their sum in the return value ...
__device__ __forceinline__ int wave_counts(int E, const int* cnt, int (&c)[SORT_W]) {
  int sum = 0;
  if ((int)threadIdx.x < E)
#pragma unroll
    for (int w = 0; w < SORT_W; ++w) sum += c[w] = cnt[w * E + threadIdx.x];
  return sum;
}
// ... and the waves' first places, from the expert's first one on.
__device__ __forceinline__ void wave_bases(int E, int* cnt, const int (&c)[SORT_W], int first) {
  if ((int)threadIdx.x < E)
#pragma unroll
    for (int w = 0; w < SORT_W; ++w) {
      cnt[w * E + threadIdx.x] = first;
      first += c[w];
    }
}

// place(u, at): the place among the counted ones of each assignment (id[u] >= 0), by wave, in order.
template <int PER, typename F>
__device__ __forceinline__ void sort_rank(const int (&id)[PER], int E, int* cnt, F place) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int bits = 1;
  while ((1 << bits) < E) ++bits;
  int* base = cnt + wave * E;
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const bool ok = id[u] >= 0;
    const int x = ok ? id[u] : 0;
    const uint64_t some = __ballot(ok);
    uint32_t lo = (uint32_t)some, hi = (uint32_t)(some >> 32);   // the lanes with the lane's expert
    for (int b = 0; b < bits; ++b) {
      const int t = (int)((uint32_t)x << (31 - b)) >> 31;        // all ones where the bit is set
      const uint64_t m = __ballot(t != 0);
      lo &= ~((uint32_t)m ^ (uint32_t)t);
      hi &= ~((uint32_t)(m >> 32) ^ (uint32_t)t);
    }
    const int rank = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));   // of them, below the lane
    const int at = ok ? base[x] + rank : -1;
    // Every lane has read its base before one lane per expert moves it on, and
    // reads it anew in the next turn (LDS operations of a wave run in order).
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (ok && rank == 0) base[x] = at + __popc(lo) + __popc(hi);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    place(u, at);
  }
}

// Few assignments: one workgroup does it all.
template <int PER>
__global__ __launch_bounds__(SORT_T) void sort_small_kernel(const int32_t* __restrict__ ids, int64_t n, DivK K, int E,
                                                            int32_t* __restrict__ tok_idx, int64_t* __restrict__ grp_off,
                                                            int32_t* __restrict__ pos) {
  extern __shared__ int cnt[];   // SORT_W * E
  __shared__ int part[1][SORT_W];
  int id[PER], c[SORT_W], sum[1], all[1];
  sort_count<PER>(ids, 0, n, E, cnt, id);
  sum[0] = wave_counts(E, cnt, c);
  expert_sums<1>(E, sum, all, part);
  wave_bases(E, cnt, c, sum[0]);
  const int total = all[0];
  if ((int)threadIdx.x < E) grp_off[threadIdx.x] = sum[0];
  if (threadIdx.x == 0) grp_off[E] = total;
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  sort_rank<PER>(id, E, cnt, [&](int u, int at) {
    const int64_t i = (wave * PER + u) * 64 + lane;
    if (i < n) pos[i] = at;
    if (at >= 0) tok_idx[at] = div_k(i, K);
  });
  for (int64_t i = total + (int)threadIdx.x; i < n; i += SORT_T) tok_idx[i] = -1;
}

// Many: counts of each chunk [nb][E] ...
template <int PER>
__global__ __launch_bounds__(SORT_T) void sort_hist_kernel(const int32_t* __restrict__ ids, int64_t n, int E,
                                                           int32_t* __restrict__ hist) {
  extern __shared__ int cnt[];   // E
  const int64_t beg = (int64_t)blockIdx.x * (SORT_T * PER) + threadIdx.x;
  int id[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) id[u] = beg + u * SORT_T < n ? ids[beg + u * SORT_T] : -1;
  for (int i = threadIdx.x; i < E; i += SORT_T) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if ((unsigned)id[u] < (unsigned)E) atomicAdd(cnt + id[u], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += SORT_T) hist[(int64_t)blockIdx.x * E + i] = cnt[i];
}

// ... their exclusive sums over the chunks in place, and each expert's total
// (64 experts per workgroup, each wave a range of chunks, SCAN_U counts in
// flight at once) ...
constexpr int SCAN_U = 16;
__global__ __launch_bounds__(SORT_T) void sort_scan_kernel(int32_t* __restrict__ hist, int nb, int E,
                                                           int32_t* __restrict__ total) {
  __shared__ int sum[SORT_W][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (nb + SORT_W - 1) / SORT_W;
  const int b0 = min(nb, wave * per), b1 = min(nb, b0 + per);
  int c[SCAN_U], s = 0;
  auto load = [&](int b) {
#pragma unroll
    for (int u = 0; u < SCAN_U; ++u) c[u] = e < E && b + u < b1 ? hist[(int64_t)(b + u) * E + e] : 0;
  };
  for (int b = b0; b < b1; b += SCAN_U) {
    load(b);
#pragma unroll
    for (int u = 0; u < SCAN_U; ++u) s += c[u];
  }
  sum[wave][lane] = s;
  __syncthreads();
  int run = 0, all = 0;
  for (int w = 0; w < SORT_W; ++w) {
    run += w < wave ? sum[w][lane] : 0;
    all += sum[w][lane];
  }
  if (e >= E) return;
  for (int b = b0; b < b1; b += SCAN_U) {
    if (per > SCAN_U) load(b);   // else c still holds them
#pragma unroll
    for (int u = 0; u < SCAN_U; ++u)
      if (b + u < b1) {
        hist[(int64_t)(b + u) * E + e] = run;
        run += c[u];
      }
  }
  if (wave == 0) total[e] = all;
}

// ... and the rows: the chunk's places in LDS first, then each place's row is
// its expert's shift (row of the chunk's first one of the expert - its place) away.
template <int PER>
__global__ __launch_bounds__(SORT_T) void sort_place_kernel(const int32_t* __restrict__ ids, int64_t n, DivK K, int E,
                                                            const int32_t* __restrict__ hist,
                                                            const int32_t* __restrict__ total,
                                                            int32_t* __restrict__ tok_idx,
                                                            int64_t* __restrict__ grp_off, int32_t* __restrict__ pos) {
  extern __shared__ int cnt[];   // SORT_W * E, then E shifts
  __shared__ int part[2][SORT_W];
  __shared__ int32_t tok[SORT_T * PER];
  __shared__ uint16_t expert[SORT_T * PER];
  int* shift = cnt + SORT_W * E;
  const int64_t beg = (int64_t)blockIdx.x * (SORT_T * PER), end = std::min<int64_t>(n, beg + SORT_T * PER);
  const int x = threadIdx.x, wave = x >> 6, lane = x & 63;
  int id[PER], c[SORT_W], sum[2], all[2];
  sum[0] = x < E ? total[x] : 0;
  const int before = x < E ? hist[(int64_t)blockIdx.x * E + x] : 0;
  sort_count<PER>(ids, beg, end, E, cnt, id);
  sum[1] = wave_counts(E, cnt, c);
  expert_sums<2>(E, sum, all, part);   // the experts' first rows, and their first places in the chunk
  wave_bases(E, cnt, c, sum[1]);
  if (x < E) {
    shift[x] = sum[0] + before - sum[1];
    if (blockIdx.x == 0) grp_off[x] = sum[0];
  }
  if (blockIdx.x == 0 && x == 0) grp_off[E] = all[0];
  __syncthreads();
  sort_rank<PER>(id, E, cnt, [&](int u, int at) {
    const int64_t i = beg + (wave * PER + u) * 64 + lane;
    if (i < end) pos[i] = at >= 0 ? at + shift[id[u]] : -1;
    if (at >= 0) {
      tok[at] = div_k(i, K);
      expert[at] = (uint16_t)id[u];
    }
  });
  __syncthreads();
  for (int i = x; i < all[1]; i += SORT_T) tok_idx[i + shift[expert[i]]] = tok[i];
  for (int64_t i = beg + x; i < end; i += SORT_T)
    if (i >= all[0]) tok_idx[i] = -1;
}

// ---- a token's experts summed ------------------------------------------------------
// Elements move in vectors of VW (16 bytes of the wider type), at any element's
// address (the device loads and stores them whole); the columns behind the last
// whole vector one by one.
template <typename E, int VW>
__device__ __forceinline__ void load_vec(const E* p, float (&v)[VW]) {
  typedef E Vec __attribute__((ext_vector_type(VW), aligned(sizeof(E))));
  const Vec x = *(const Vec*)p;
#pragma unroll
  for (int i = 0; i < VW; ++i) {
    const E e = x[i];
    v[i] = load_f(&e);
  }
}
template <typename E, int VW>
__device__ __forceinline__ void store_vec(E* p, const float (&v)[VW]) {
  typedef E Vec __attribute__((ext_vector_type(VW), aligned(sizeof(E))));
  Vec x;
#pragma unroll
  for (int i = 0; i < VW; ++i) {
    E e;
    store_f(&e, v[i]);
    x[i] = e;
  }
  *(Vec*)p = x;
}

// One thread per vector of a token's columns: blockDim = (columns, tokens).
// KC slots' loads are in flight together; sums run in slot order.  Bound by
// reading the rows once: 16384 x 8 rows of 4096 bf16 in 225 us, 5.4 TB/s.
constexpr int KC = 8;
template <typename Y, typename O, int VW>
__global__ __launch_bounds__(256) void combine_kernel(const Y* __restrict__ y, int64_t rows, int64_t d, int64_t ldy,
                                                      const int32_t* __restrict__ pos, const float* __restrict__ w,
                                                      int64_t T, int K, O* __restrict__ out, int64_t ldo,
                                                      int col_blocks) {
  const int64_t v = (int64_t)(blockIdx.x % col_blocks) * blockDim.x + threadIdx.x;
  const int64_t t = (int64_t)(blockIdx.x / col_blocks) * blockDim.y +
                    __builtin_amdgcn_readfirstlane(threadIdx.y);   // the same in a whole wave: blockDim.x is 64 or more
  if (v * VW >= d || t >= T) return;
  auto columns = [&]<int W>(int64_t c) {
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    for (int s0 = 0; s0 < K; s0 += KC) {
      float wt[KC], x[KC][W];
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int64_t i = t * K + s0 + j;
        const int64_t r = s0 + j < K ? pos[i] : -1;
        wt[j] = s0 + j < K ? (w ? w[i] : 1.0f) : 0.0f;
#pragma unroll
        for (int q = 0; q < W; ++q) x[j][q] = 0.0f;
        if ((uint64_t)r < (uint64_t)rows) load_vec<Y, W>(y + r * ldy + c, x[j]);
      }
#pragma unroll
      for (int j = 0; j < KC; ++j)
#pragma unroll
        for (int q = 0; q < W; ++q) sum[q] = fmaf(wt[j], x[j][q], sum[q]);
    }
    store_vec<O, W>(out + t * ldo + c, sum);
  };
  if (v * VW + VW <= d) columns.template operator()<VW>(v * VW);
  else
    for (int64_t c = v * VW; c < d; ++c) columns.template operator()<1>(c);
}

// Its gradients: a workgroup of NW waves per token, dout's row read once for
// KC slots at a time; each lane sums its columns' products, then lanes and
// waves are added in a fixed order.  Bound by the rows' traffic: 5003 x 6 rows
// of 2056 fp32 and their gradients (0.54 GB) in 126 us, 4.2 TB/s.
template <typename G, typename Y, int VW, int NW>
__global__ __launch_bounds__(64 * NW) void combine_backward_kernel(const G* __restrict__ dout, int64_t T, int64_t d,
                                                                   int64_t ldd, const Y* __restrict__ y, int64_t rows,
                                                                   int64_t ldy, const int32_t* __restrict__ pos,
                                                                   const float* __restrict__ w, int K,
                                                                   Y* __restrict__ dy, int64_t lddy,
                                                                   float* __restrict__ dw) {
  __shared__ float part[NW][KC];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  for (int s0 = 0; s0 < K; s0 += KC) {
    int r[KC];
    float wt[KC], dot[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const int64_t i = t * K + s0 + j;
      r[j] = s0 + j < K ? pos[i] : -1;
      if (r[j] >= rows) r[j] = -1;
      wt[j] = s0 + j < K ? (w ? w[i] : 1.0f) : 0.0f;
      dot[j] = 0.0f;
    }
    auto columns = [&]<int W>(int64_t c) {
      float g[W], x[KC][W];
      load_vec<G, W>(dout + t * ldd + c, g);
      if (dw) {
#pragma unroll
        for (int j = 0; j < KC; ++j) {
#pragma unroll
          for (int q = 0; q < W; ++q) x[j][q] = 0.0f;
          if (r[j] >= 0) load_vec<Y, W>(y + (int64_t)r[j] * ldy + c, x[j]);
        }
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (r[j] >= 0) {
#pragma unroll
            for (int q = 0; q < W; ++q) dot[j] = fmaf(g[q], x[j][q], dot[j]);
          }
      }
      if (dy)
#pragma unroll
        for (int j = 0; j < KC; ++j)
          if (r[j] >= 0) {
            float o[W];
#pragma unroll
            for (int q = 0; q < W; ++q) o[q] = wt[j] * g[q];
            store_vec<Y, W>(dy + (int64_t)r[j] * lddy + c, o);
          }
    };
    for (int64_t c = (int64_t)threadIdx.x * VW; c < d; c += 64 * NW * VW) {
      if (c + VW <= d) columns.template operator()<VW>(c);
      else
        for (int64_t e = c; e < d; ++e) columns.template operator()<1>(e);
    }
    if (!dw) continue;
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const float sum = group_sum<64>(dot[j]);
      if (lane == 0) part[wave][j] = sum;
    }
    __syncthreads();
    if (threadIdx.x < KC && s0 + (int)threadIdx.x < K) {
      float sum = 0.0f;
#pragma unroll
      for (int x = 0; x < NW; ++x) sum += part[x][threadIdx.x];
      dw[t * K + s0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// Calls f(LPT, EPL) with the constants for E experts: 16 lanes per token when
// there are tokens enough to fill the device that way, at most 256 experts and
// 16 slots.  us with 64 / 16 lanes: 256 experts bf16, 8 slots, 2048 tokens 3.4 /
// 3.9, 4096 tokens 4.2 / 3.5, 65536 tokens 33 / 16; 64 experts fp32, 6 slots, 1024
// tokens 3.1 / 3.2, 4096 tokens 4.1 / 3.3; the gradient with 128 experts fp32, 4096
// tokens 3.4 / 3.8, 16384 tokens 6.7 / 5.7.
constexpr int64_t kTopkWaves = 4096;   // tokens from which 16 lanes per token are taken
template <typename F>
hipError_t topk_dispatch(int64_t T, int E, int K, F f) {
  const int lanes = T >= kTopkWaves && E <= 256 && K <= 16 ? 16 : 64;
  int epl = 1;
  while (epl * lanes < E) epl *= 2;
#define NVQ_TOPK_CASE(LPT, EPL) \
  if (lanes == LPT && epl == EPL) return f.template operator()<LPT, EPL>()
  NVQ_TOPK_CASE(16, 1);
  NVQ_TOPK_CASE(16, 2);
  NVQ_TOPK_CASE(16, 4);
  NVQ_TOPK_CASE(16, 8);
  NVQ_TOPK_CASE(16, 16);
  NVQ_TOPK_CASE(64, 1);
  NVQ_TOPK_CASE(64, 2);
  NVQ_TOPK_CASE(64, 4);
  NVQ_TOPK_CASE(64, 8);
  NVQ_TOPK_CASE(64, 16);
#undef NVQ_TOPK_CASE
  return hipErrorInvalidValue;
}

// f(t0, nt) for parts of T tokens, as many as a launch of that many threads per token holds: whole workgroups
// (at most 16 tokens each, where a token has few threads), or single tokens where fewer than 64 fit.
template <typename F>
hipError_t in_parts(int64_t T, int64_t threads, F f) {
  const int64_t fit = kMaxThreads / threads, most = fit < 64 ? fit : fit / 64 * 64;
  if (most == 0) return hipErrorInvalidValue;
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    f(t0, std::min(most, T - t0));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename L>
hipError_t topk_run(const L* logits, int64_t T, int E, int64_t ld, int K, int renorm, int32_t* ids, float* weights,
                    hipStream_t s) {
  return topk_dispatch(T, E, K, [&]<int LPT, int EPL>() {
    const int64_t per = 256 / LPT;
    const auto run = [&]<int SORTED>() {
      return in_parts(T, LPT, [&](int64_t t0, int64_t nt) {
        hipLaunchKernelGGL((topk_kernel<L, LPT, EPL, SORTED>), dim3((unsigned)((nt + per - 1) / per)), dim3(256), 0, s,
                           logits + t0 * ld, nt, E, ld, K, renorm, ids + t0 * K, weights + t0 * K);
      });
    };
    if constexpr (sizeof(L) == 2)
      if (K <= 8) return run.template operator()<8>();
    return run.template operator()<0>();
  });
}

template <typename L>
hipError_t topk_backward_run(const L* logits, int64_t T, int E, int64_t ld, const int32_t* ids, const float* w,
                             const float* dw, int K, int renorm, L* dl, int64_t ldd, hipStream_t s) {
  return topk_dispatch(T, E, K, [&]<int LPT, int EPL>() {
    const int64_t per = 256 / LPT;
    return in_parts(T, LPT, [&](int64_t t0, int64_t nt) {
      hipLaunchKernelGGL((topk_backward_kernel<L, LPT, EPL>), dim3((unsigned)((nt + per - 1) / per)), dim3(256), 0, s,
                         logits + t0 * ld, nt, E, ld, ids + t0 * K, w + t0 * K, dw + t0 * K, K, renorm, dl + t0 * ldd, ldd);
    });
  });
}

// Assignments up to which one workgroup sorts (8192 of them, 256 experts: one
// workgroup 10.9 us, three launches 12.3), and up to which chunks are 4096 long,
// which gives each CU one; 8192 behind it (2^20: 14.6 / 17.0 us, 2^21: 22.1 / 19.1).
constexpr int64_t kSortSmall = 8 * SORT_T, kSortLarge = (int64_t)1 << 20;
int sort_per(int64_t n) { return n > kSortLarge ? 8 : 4; }
int64_t sort_blocks(int64_t n) { return (n + SORT_T * sort_per(n) - 1) / (SORT_T * sort_per(n)); }

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
  const DivK div = div_by((uint32_t)K);
#define NVQ_SORT(PER)                                                                                                   \
  hipLaunchKernelGGL(sort_small_kernel<PER>, dim3(1), dim3(SORT_T), lds, s, ids, n, div, (int)E, tok_idx, grp_off, pos)
  if (n <= kSortSmall) {
    if (n <= SORT_T) NVQ_SORT(1);
    else if (n <= 4 * SORT_T) NVQ_SORT(4);
    else NVQ_SORT(8);
    return hipGetLastError();
  }
#undef NVQ_SORT
  const int nb = (int)sort_blocks(n);
  int32_t* hist = (int32_t*)ws;
  int32_t* total = hist + (int64_t)nb * E;
#define NVQ_SORT(PER)                                                                                                  \
  do {                                                                                                                 \
    hipLaunchKernelGGL(sort_hist_kernel<PER>, dim3(nb), dim3(SORT_T), E * sizeof(int), s, ids, n, (int)E, hist);        \
    hipLaunchKernelGGL(sort_scan_kernel, dim3((unsigned)((E + 63) / 64)), dim3(SORT_T), 0, s, hist, nb, (int)E, total); \
    hipLaunchKernelGGL(sort_place_kernel<PER>, dim3(nb), dim3(SORT_T), lds + E * sizeof(int), s, ids, n, div, (int)E,    \
                       hist, total, tok_idx, grp_off, pos);                                                            \
  } while (0)
  if (sort_per(n) == 8) NVQ_SORT(8);
  else NVQ_SORT(4);
#undef NVQ_SORT
  return hipGetLastError();
}

template <typename Y, typename O, int VW>
static hipError_t combine_run(const Y* y, int64_t rows, int64_t d, int64_t ldy, const int32_t* pos, const float* w, int64_t T,
                              int K, O* out, int64_t ldo, hipStream_t s) {
  const int64_t nv = (d + VW - 1) / VW;
  int bx = 64;   // columns of a workgroup; at least a wave, so that a wave's slots are uniform
  while (bx < 256 && bx < nv) bx *= 2;
  const int by = 256 / bx;
  const int64_t cb = (nv + bx - 1) / bx;
  return in_parts(T, cb * bx, [&](int64_t t0, int64_t nt) {
    hipLaunchKernelGGL((combine_kernel<Y, O, VW>), dim3((unsigned)(cb * ((nt + by - 1) / by))), dim3(bx, by), 0, s, y, rows,
                       d, ldy, pos + t0 * K, w ? w + t0 * K : nullptr, nt, K, out + t0 * ldo, ldo, (int)cb);
  });
}

hipError_t moe_combine_launch(const void* Y, int y_bf16, int64_t rows, int64_t d, int64_t ldy, const int32_t* pos,
                              const float* weights, int64_t T, int K, void* out, int out_bf16, int64_t ldo,
                              hipStream_t s) {
#define NVQ_RUN(YT, OT, VW) combine_run<YT, OT, VW>((const YT*)Y, rows, d, ldy, pos, weights, T, K, (OT*)out, ldo, s)
  if (y_bf16 && out_bf16) return NVQ_RUN(uint16_t, uint16_t, 8);
  if (y_bf16) return NVQ_RUN(uint16_t, float, 4);
  if (out_bf16) return NVQ_RUN(float, uint16_t, 4);
  return NVQ_RUN(float, float, 4);
#undef NVQ_RUN
}

template <typename G, typename Y, int VW>
static hipError_t combine_backward_run(const G* dout, int64_t T, int64_t d, int64_t ldd, const Y* y, int64_t rows,
                                       int64_t ldy, const int32_t* pos, const float* w, int K, Y* dy, int64_t lddy,
                                       float* dw, hipStream_t s) {
  auto run = [&]<int NW>() {
    return in_parts(T, 64 * NW, [&](int64_t t0, int64_t nt) {
      hipLaunchKernelGGL((combine_backward_kernel<G, Y, VW, NW>), dim3((unsigned)nt), dim3(64 * NW), 0, s, dout + t0 * ldd,
                         nt, d, ldd, y, rows, ldy, pos + t0 * K, w ? w + t0 * K : nullptr, K, dy, lddy,
                         dw ? dw + t0 * K : nullptr);
    });
  };
  // Waves per token: one for short rows, more for few tokens with long rows.  us
  // with 1 / 2 / 4 / 16 waves, 8 slots bf16: 4096 tokens d = 512 14.8 / 22.6 / 30.4 /
  // 96.9, d = 1024 25.2 / 28.0 / 34.4 / 99.1, d = 4096 143 / 148 / 124 / 186; 512 tokens
  // d = 4096 35.4 / 22.4 / 16.6 / 19.7; 256 tokens 29.6 / 18.2 / 12.3 / 10.4; 8 tokens
  // d = 1024 8.1 / 6.2 / 6.2 / 6.2, d = 2048 12.4 / 8.2 / 6.4 / 6.3.
  const int64_t nv = (d + VW - 1) / VW;
  if (nv <= (T >= 4096 ? 128 : 64)) return run.template operator()<1>();
  if (nv <= 128) return run.template operator()<2>();
  if (T >= 512 || nv <= 256) return run.template operator()<4>();
  return run.template operator()<16>();
}

hipError_t moe_combine_backward_launch(const void* dout, int dout_bf16, int64_t T, int64_t d, int64_t ldd, const void* Y,
                                       int y_bf16, int64_t rows, int64_t ldy, const int32_t* pos, const float* weights,
                                       int K, void* dY, int64_t lddy, float* dw, hipStream_t s) {
#define NVQ_RUN(GT, YT, VW)                                                                                           \
  combine_backward_run<GT, YT, VW>((const GT*)dout, T, d, ldd, (const YT*)Y, rows, ldy, pos, weights, K, (YT*)dY, lddy, \
                                   dw, s)
  if (dout_bf16 && y_bf16) return NVQ_RUN(uint16_t, uint16_t, 8);
  if (dout_bf16) return NVQ_RUN(uint16_t, float, 4);
  if (y_bf16) return NVQ_RUN(float, uint16_t, 4);
  return NVQ_RUN(float, float, 4);
#undef NVQ_RUN
}

}  // namespace nvq
