// A whole mixture-of-experts MLP with NVFP4 experts for a few tokens (at most
// 64), in two kernels:
//   1. routing (moe_topk's choice, or the caller's), then for each expert in use
//      and each of its tokens  act = w silu(G x) (U x),  w the token's weight;
//   2. out[t] = sum over its experts of g_e D act.
// A token's row is a column of the matrix instructions, so an expert's weights are read and
// expanded once for all its tokens, and a sum over experts stays in registers.
// Q = e2m1 * e4m3 is exact in bf16 and g is applied to the sums.  The
// activation between the products is held as two bf16 parts, hi + lo (16 or more
// significant bits as long as it is above 2^-110): as one bf16 it would be the one value
// that the layer rounds to 8 bits before its end, for a product that waits for weights anyway.
// What bounds it: reading the weights of the experts in use once.
#include <algorithm>

#include "common.h"
#include "dequant.h"
#include "kernels.h"
#include "router.h"

namespace nvq {

namespace {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

constexpr int MW = 8;   // waves per workgroup
constexpr uint32_t kNone = 0x80000000u;   // an offset past every buffer (checked on the host), also with k's offsets added

// An expert in use: its rows of the activations start at `row`, in the order of its tokens (bits).
struct Entry {
  int32_t expert, row;
  uint64_t tokens;
};

struct MoeMlp {
  const uint16_t* X;
  const void* logits;
  int32_t* ids;
  float* weights;
  const uint8_t *ucodes, *uscales, *dcodes, *dscales;
  const float *ug, *dg;
  void* out;
  int64_t ldx, ldl, d, h, m, ldo;
  int T, E, K, renorm;
  // workspace
  int32_t* count;     // experts in use
  float* bad;         // per token: 0, or NaN from the weight of a slot without an expert
  Entry* entries;
  uint16_t *hi, *lo;  // activations [rows x h]
};

// 256 k of 16 CG channels: lane (c = l % 16, q = l / 16) takes the 32 k from 32 q of each 128, of channel c.
template <int CG>
struct Pair {
  u32x4 w[2][CG];
  uint32_t s[2][CG];
};
// cp, sp: the channels' first codes and scales (uniform); crow, srow: the lane's offsets, its channel and q included.
template <int CG>
__device__ __forceinline__ void load_pair(const uint8_t* const (&cp)[CG], const uint8_t* const (&sp)[CG], uint32_t crow, uint32_t srow,
                                          int64_t p, int q, int64_t k, Pair<CG>& x) {
  if ((p + 1) * 256 <= k) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int f = 0; f < CG; ++f) {
        x.w[u][f] = *(const u32x4_any*)(cp[f] + p * 128 + 64 * u + crow);
        x.s[u][f] = *(const u16_any*)(sp[f] + p * 16 + 8 * u + srow);
      }
    return;
  }
  // The rest of k: blocks past it as zero codes under zero scales.
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t left = k / 16 - (p * 16 + 8 * u + 2 * q);   // blocks from the lane's first on
#pragma unroll
    for (int f = 0; f < CG; ++f) {
      u32x2 a{0u, 0u}, b{0u, 0u};
      uint32_t s = 0;
      if (left > 0) {
        a = *(const u32x2_any*)(cp[f] + p * 128 + 64 * u + crow);
        s = sp[f][p * 16 + 8 * u + srow];
      }
      if (left > 1) {
        b = *(const u32x2_any*)(cp[f] + p * 128 + 64 * u + crow + 8);
        s |= (uint32_t)sp[f][p * 16 + 8 * u + srow + 1] << 8;
      }
      x.w[u][f] = u32x4{a[0], a[1], b[0], b[1]};
      x.s[u][f] = s;
    }
  }
}
// The eight k from 8 j of the lane's 32, expanded.
__device__ __forceinline__ bf16x8 expand(const u32x4& w, uint32_t s2, int j) {
  const float s = j < 2 ? e4m3_byte<0>(s2) : e4m3_byte<1>(s2);
  const uint32_t v = w[j];
  return __builtin_bit_cast(bf16x8, u32x4{dq_byte<0>(v, s), dq_byte<1>(v, s), dq_byte<2>(v, s), dq_byte<3>(v, s)});
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
#if __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
#else
  return u32x4{0u, 0u, 0u, 0u};
#endif
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
#if __HIP_DEVICE_COMPILE__
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, bytes, 0x00020000);
#else
  return __amdgpu_buffer_rsrc_t();
#endif
}
// The lane's 32 k of half u of pair p from its row's offset, zeros from k on.
__device__ __forceinline__ void load_half(__amdgpu_buffer_rsrc_t rs, uint32_t row, int64_t p, int u, int q, int64_t k, u32x4 (&x)[4]) {
  const int64_t k0 = p * 256 + 128 * u + 32 * q;
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = load16(rs, k0 + 8 * j < k ? row + (uint32_t)(k0 + 8 * j) * 2 : kNone);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ Entry uniform_entry(const Entry& e) {
  Entry r;
  r.expert = __builtin_amdgcn_readfirstlane(e.expert);
  r.row = __builtin_amdgcn_readfirstlane(e.row);
  r.tokens = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)e.tokens) |
             (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(e.tokens >> 32)) << 32;
  return r;
}
// Tokens before t.
__device__ __forceinline__ int before(uint64_t tokens, int t) { return __popcll(tokens & ((1ull << t) - 1)); }

// Kernel 1.  Every workgroup routes all tokens for itself (a launch for it
// alone would cost more), lists the experts in use, then takes items, 16
// channels of gate and of up of one expert, in turn with the other workgroups;
// the eight waves each a part of k, their sums added in wave order through LDS.
// NG: groups of 16 tokens.
size_t up_lds(int64_t T, int64_t E, int64_t K) { return E * 8 + T * K * 8 + std::min(E, T * K) * sizeof(Entry); }

template <typename L, int EPL, int NG>
__global__ __launch_bounds__(64 * MW, NG == 1 ? 4 : 2) void moe_up_kernel(const MoeMlp a) {
  __shared__ __attribute__((aligned(16))) float part[MW][16][36];
  __shared__ int s_count;
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  const int slots = a.T * a.K;
  Entry* list = (Entry*)dyn;
  uint64_t* mask = (uint64_t*)(list + min(a.E, slots));
  int32_t* ids = (int32_t*)(mask + a.E);
  float* ws = (float*)(ids + slots);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;

  for (int e = tid; e < a.E; e += 64 * MW) mask[e] = 0;
  __syncthreads();
  if (a.logits) {
    for (int t = wave; t < a.T; t += MW) {
      int32_t id;
      float w;
      route_token<L, 64, EPL, 0>((const L*)a.logits + t * a.ldl, a.E, a.K, a.renorm, lane, id, w);
      if (lane < a.K) {
        ids[t * a.K + lane] = id;
        ws[t * a.K + lane] = w;
        if (id >= 0) atomicOr((unsigned long long*)&mask[id], 1ull << t);
        if (blockIdx.x == 0) {
          a.ids[t * a.K + lane] = id;
          a.weights[t * a.K + lane] = w;
        }
      }
    }
  } else {
    for (int p = tid; p < slots; p += 64 * MW) {
      const int id = a.ids[p];
      ids[p] = id;
      ws[p] = a.weights[p];
      if (id >= 0 && id < a.E) atomicOr((unsigned long long*)&mask[id], 1ull << (p / a.K));
    }
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0, rows = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const uint64_t tokens = e0 + lane < a.E ? mask[e0 + lane] : 0;
      const uint64_t used = __ballot(tokens != 0);
      const int mine = __popcll(tokens), incl = wave_inclusive(mine);
      if (tokens) list[n + before(used, lane)] = Entry{e0 + lane, rows + incl - mine, tokens};
      n += __popcll(used);
      rows += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) s_count = n;
  }
  __syncthreads();
  const int used = __builtin_amdgcn_readfirstlane(s_count);
  if (blockIdx.x == 0) {
    if (tid == 0) *a.count = used;
    for (int i = tid; i < used; i += 64 * MW) a.entries[i] = list[i];
    if (tid < a.T) {
      float nan = 0.0f;
      for (int s = 0; s < a.K; ++s) {
        const int id = ids[tid * a.K + s];
        if (id < 0 || id >= a.E) nan += ws[tid * a.K + s] * 0.0f;
      }
      a.bad[tid] = nan;
    }
  }

  const int nt = (int)((a.h + 15) / 16), items = used * nt;
  const int64_t kh = a.d / 2, kb = a.d / 16;
  const int npairs = (int)((a.d + 255) / 256), mine = npairs > wave ? (npairs - wave + MW - 1) / MW : 0;
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.X, (uint32_t)(((a.T - 1) * a.ldx + a.d) * 2));
  uint32_t xrow[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) xrow[g] = 16 * g + c < a.T ? (uint32_t)((16 * g + c) * a.ldx * 2) : kNone;

  // What is loaded next: the li-th of the wave's pairs of item `lit`.
  int lit = blockIdx.x, li = 0;
  const uint8_t *cp[2], *sp[2];
  uint32_t crow = 0, srow = 0;
  auto locate = [&]() {
    if (lit >= items) return;
    const int at = lit / nt;
    const int64_t e = __builtin_amdgcn_readfirstlane(list[at].expert), o0 = 16 * (int64_t)(lit - at * nt);
    const uint32_t o = (uint32_t)min((int64_t)c, a.h - 1 - o0);   // (channels past h repeat the last one and are not stored)
    crow = o * (uint32_t)kh + 16 * q;
    srow = o * (uint32_t)kb + 2 * q;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      cp[f] = a.ucodes + (e * 2 * a.h + f * a.h + o0) * kh;
      sp[f] = a.uscales + (e * 2 * a.h + f * a.h + o0) * kb;
    }
  };
  auto load_next = [&](Pair<2>& b) {
    if (lit < items) load_pair<2>(cp, sp, crow, srow, wave + MW * li, q, a.d, b);
    if (++li == mine) {
      li = 0;
      lit += gridDim.x;
      locate();
    }
  };

  f32x4 acc[NG][2];
  auto clear = [&]() {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int f = 0; f < 2; ++f) acc[g][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  int item = blockIdx.x;
  auto finish = [&]() {   // the item's activations
    const int at = item / nt;
    const Entry e = uniform_entry(list[at]);
    const int o0 = 16 * (item - at * nt);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t here = (uint32_t)(e.tokens >> (16 * g)) & 0xFFFF;
      if (!here) continue;   // (the same for all waves)
#pragma unroll
      for (int f = 0; f < 2; ++f) *(f32x4*)&part[wave][c][16 * f + 4 * q] = acc[g][f];
      __syncthreads();
      const int col = tid >> 4, ch = tid & 15;
      if (tid < 256 && (here >> col & 1) && o0 + ch < a.h) {
        float gate = 0.0f, up = 0.0f;
#pragma unroll
        for (int w = 0; w < MW; ++w) {
          gate += part[w][col][ch];
          up += part[w][col][16 + ch];
        }
        const int t = 16 * g + col;
        float w = 0.0f;
        for (int s = 0; s < a.K; ++s) w += ids[t * a.K + s] == e.expert ? ws[t * a.K + s] : 0.0f;
        const float scale = a.ug[e.expert];
        gate *= scale;
        up *= scale;
        const float z = expf(-fabsf(gate)), one = 1.0f / (1.0f + z);
        const float v = gate * (gate >= 0.0f ? one : z * one) * up * w;
        const __bf16 hi = (__bf16)v;
        const float rest = v - (float)hi;
        const __bf16 lo = (__bf16)(fabsf((float)hi) < __builtin_inff() ? rest : 0.0f);   // (an infinity or NaN is in hi alone)
        const int64_t to = (e.row + before(e.tokens, t)) * a.h + o0 + ch;
        a.hi[to] = __builtin_bit_cast(uint16_t, hi);
        a.lo[to] = __builtin_bit_cast(uint16_t, lo);
      }
      __syncthreads();
    }
  };
  // One half's products.  One group: its activations were loaded ahead.  More:
  // the weights are expanded once, then each group that the expert has tokens in.
  uint64_t tokens = 0;   // of the item's expert (more groups only)
  auto half = [&](const u32x4 (&w)[2], const uint32_t (&s)[2], const u32x4 (&x)[4], int64_t p, int u) {
    if constexpr (NG == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < 2; ++f) acc[0][f] = mfma(expand(w[f], s[f], j), x[j], acc[0][f]);
    } else {
      bf16x8 v[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int f = 0; f < 2; ++f) v[j][f] = expand(w[f], s[f], j);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!((tokens >> (16 * g)) & 0xFFFF)) continue;
        u32x4 y[4];
        load_half(xbuf, xrow[g], p, u, q, a.d, y);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < 2; ++f) acc[g][f] = mfma(v[j][f], y[j], acc[g][f]);
      }
    }
  };
  auto enter = [&]() {
    clear();
    if (NG > 1 && item < items) tokens = uniform_entry(list[item / nt]).tokens;
  };

  enter();
  if (mine == 0) {   // (k has fewer pairs than there are waves)
    for (; item < items; item += gridDim.x) finish();
    return;
  }
  Pair<2> b0, b1;
  u32x4 xa[4], xb[4];
  locate();
  load_next(b0);
  load_next(b1);
  if (NG == 1) load_half(xbuf, xrow[0], wave, 0, q, a.d, xa);
  int i = 0;
  auto consume = [&](Pair<2>& b) {
    const int64_t p = wave + MW * i;
    if (NG == 1) load_half(xbuf, xrow[0], p, 1, q, a.d, xb);
    __builtin_amdgcn_sched_barrier(0);
    half(b.w[0], b.s[0], xa, p, 0);
    if (NG == 1) load_half(xbuf, xrow[0], wave + MW * (i + 1 == mine ? 0 : i + 1), 0, q, a.d, xa);
    __builtin_amdgcn_sched_barrier(0);
    half(b.w[1], b.s[1], xb, p, 1);
    load_next(b);
    __builtin_amdgcn_sched_barrier(0);
    if (++i == mine) {
      finish();
      i = 0;
      item += gridDim.x;
      enter();
    }
  };
  while (item < items) {
    consume(b0);
    if (item >= items) break;
    consume(b1);
  }
}

// Kernel 2: 16 output channels per workgroup.  The units (256 k of an expert's
// activations) of all experts in use lie in a row, which the eight waves share
// in equal runs; a wave adds its experts' sums times g, and the waves' totals are
// added in wave order through LDS.  A token that does not use an expert has
// zeros in its column, and the expert's sum is not added to it (a rejected weight
// row would make it NaN).
template <int NG, int OUT_BF16>
__global__ __launch_bounds__(64 * MW, NG == 1 ? 4 : 2) void moe_down_kernel(const MoeMlp a) {
  __shared__ __attribute__((aligned(16))) float part[MW][16 * NG][20];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int64_t kh = a.h / 2, kb = a.h / 16, o0 = (int64_t)blockIdx.x * 16;
  const uint32_t o = (uint32_t)min((int64_t)c, a.m - 1 - o0), crow = o * (uint32_t)kh + 16 * q, srow = o * (uint32_t)kb + 2 * q;
  const int used = *a.count, per = (int)((a.h + 255) / 256), units = used * per;
  int at = (int)((int64_t)units * wave / MW);
  const int end = (int)((int64_t)units * (wave + 1) / MW);

  // Loads run FD units ahead: unit lp of entry la.
  int la = at / per, lp = at - la * per, lu = at;
  const uint8_t *cp[1], *sp[1];
  auto locate = [&]() {
    if (lu >= end) return;
    const int64_t e = __builtin_amdgcn_readfirstlane(a.entries[la].expert);
    cp[0] = a.dcodes + (e * a.m + o0) * kh;
    sp[0] = a.dscales + (e * a.m + o0) * kb;
  };
  auto load_next = [&](Pair<1>& b) {
    if (lu < end) load_pair<1>(cp, sp, crow, srow, lp, q, a.h, b);
    ++lu;
    if (++lp == per) {
      lp = 0;
      ++la;
      locate();
    }
  };
  constexpr int FD = 4;
  Pair<1> buf[FD];
  locate();
#pragma unroll
  for (int d = 0; d < FD; ++d) load_next(buf[d]);

  f32x4 acc[NG], total[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) acc[g] = total[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  int ea = at / per, ep = at - ea * per;
  Entry e;
  __amdgpu_buffer_rsrc_t hbuf, lbuf;
  uint32_t arow[NG];
  auto enter = [&]() {
    e = uniform_entry(a.entries[ea]);
    const int64_t first = e.row * a.h;
    const uint32_t bytes = (uint32_t)(__popcll(e.tokens) * a.h * 2);
    hbuf = buffer_of(a.hi + first, bytes);
    lbuf = buffer_of(a.lo + first, bytes);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int t = 16 * g + c;
      arow[g] = (e.tokens >> t & 1) ? (uint32_t)(before(e.tokens, t) * a.h * 2) : kNone;
    }
  };
  auto leave = [&]() {
    const float scale = a.dg[e.expert];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int r = 0; r < 4; ++r) total[g][r] += arow[g] != kNone ? acc[g][r] * scale : 0.0f;
      acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  auto consume = [&](Pair<1>& b) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      bf16x8 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = expand(b.w[u][0], b.s[u][0], j);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (NG > 1 && !((e.tokens >> (16 * g)) & 0xFFFF)) continue;
        u32x4 h4[4], l4[4];
        load_half(hbuf, arow[g], ep, u, q, a.h, h4);
        load_half(lbuf, arow[g], ep, u, q, a.h, l4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[g] = mfma(v[j], h4[j], acc[g]);
          acc[g] = mfma(v[j], l4[j], acc[g]);
        }
      }
    }
    load_next(b);
    ++at;
    if (++ep == per || at == end) {
      leave();
      ep = 0;
      ++ea;
      if (at < end) enter();
    }
  };
  if (at < end) {
    enter();
    while (true) {
#pragma unroll
      for (int d = 0; d < FD; ++d) {
        consume(buf[d]);
        if (at >= end) break;
      }
      if (at >= end) break;
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) *(f32x4*)&part[wave][16 * g + c][4 * q] = total[g];
  __syncthreads();
  for (int i = tid; i < 256 * NG; i += 64 * MW) {
    const int t = i >> 4, ch = i & 15;
    if (t >= a.T || o0 + ch >= a.m) continue;
    float v = a.bad[t];
#pragma unroll
    for (int w = 0; w < MW; ++w) v += part[w][t][ch];
    if (OUT_BF16) ((__bf16*)a.out)[t * a.ldo + o0 + ch] = (__bf16)v;
    else ((float*)a.out)[t * a.ldo + o0 + ch] = v;
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// Layout: count, the tokens' `bad`, the entries, the two parts of the activations.
size_t nvfp4_moe_mlp_workspace(int64_t T, int64_t E, int64_t K, int64_t h) {
  return 256 + 256 + up256(std::min(E, T * K) * sizeof(Entry)) + 2 * up256((size_t)(T * K) * h * 2);
}

hipError_t nvfp4_moe_mlp_launch(const uint16_t* X, int64_t T, int64_t d, int64_t ldx, const void* logits, int logits_bf16, int64_t E,
                                int64_t ldl, int K, int renorm, int32_t* ids, float* weights, const uint8_t* ucodes,
                                const uint8_t* uscales, const float* ug, int64_t h, const uint8_t* dcodes, const uint8_t* dscales,
                                const float* dg, int64_t m, void* out, int out_bf16, int64_t ldo, void* ws, hipStream_t s) {
  MoeMlp a{};
  a.X = X; a.logits = logits; a.ids = ids; a.weights = weights;
  a.ucodes = ucodes; a.uscales = uscales; a.ug = ug;
  a.dcodes = dcodes; a.dscales = dscales; a.dg = dg;
  a.out = out; a.ldx = ldx; a.ldl = ldl; a.d = d; a.h = h; a.m = m; a.ldo = ldo;
  a.T = (int)T; a.E = (int)E; a.K = K; a.renorm = renorm;
  char* p = (char*)ws;
  a.count = (int32_t*)p;
  a.bad = (float*)(p + 256);
  a.entries = (Entry*)(p + 512);
  p += 512 + up256(std::min(E, T * K) * sizeof(Entry));
  a.hi = (uint16_t*)p;
  a.lo = (uint16_t*)(p + up256((size_t)(T * K) * h * 2));
  const int64_t items = std::min(E, T * K) * ((h + 15) / 16);
  const dim3 up((unsigned)std::min<int64_t>(items, 512)), down((unsigned)((m + 15) / 16)), block(64 * MW);
  const size_t lds = up_lds(T, E, K);
#define NVQ_UP(L, EPL)                                                                      \
  do {                                                                                      \
    if (T <= 16) hipLaunchKernelGGL((moe_up_kernel<L, EPL, 1>), up, block, lds, s, a);      \
    else if (T <= 32) hipLaunchKernelGGL((moe_up_kernel<L, EPL, 2>), up, block, lds, s, a); \
    else hipLaunchKernelGGL((moe_up_kernel<L, EPL, 4>), up, block, lds, s, a);              \
  } while (0)
  if (logits && logits_bf16) {
    if (E <= 256) NVQ_UP(uint16_t, 4);
    else NVQ_UP(uint16_t, 16);
  } else {
    if (E <= 256) NVQ_UP(float, 4);
    else NVQ_UP(float, 16);
  }
#undef NVQ_UP
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
#define NVQ_DOWN(NG)                                                                                   \
  do {                                                                                                 \
    if (out_bf16) hipLaunchKernelGGL((moe_down_kernel<NG, 1>), down, block, 0, s, a);                  \
    else hipLaunchKernelGGL((moe_down_kernel<NG, 0>), down, block, 0, s, a);                           \
  } while (0)
  if (T <= 16) NVQ_DOWN(1);
  else if (T <= 32) NVQ_DOWN(2);
  else NVQ_DOWN(4);
#undef NVQ_DOWN
  return hipGetLastError();
}

}  // namespace nvq
