// A token's router: its top_k experts and their weights (moe_topk's kernel, and the first step of the few-token layer).
#pragma once

#include "common.h"

namespace nvq {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(uint16_t* p, float v) {
  const __bf16 b = (__bf16)v;   // nearest even, NaN kept
  *p = __builtin_bit_cast(uint16_t, b);
}

// Reductions over LPT = 16 (a DPP row) or 64 lanes, the result in every lane:
// rotations inside a row, then the row and half swaps.  All are vector
// instructions; with the LDS-unit shuffles that __shfl_xor compiles to the
// 256-expert router (65536 tokens, one per wave) took 56 us, with these 35.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int LPT, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, ror16<8>(v));
  v = f(v, ror16<4>(v));
  v = f(v, ror16<2>(v));
  v = f(v, ror16<1>(v));
  if (LPT == 64) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(r[0], r[1]);
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(h[0], h[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPT>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LPT>
__device__ __forceinline__ bool group_any(bool x) {
  const uint64_t all = __ballot(x);
  if (LPT == 64) return all != 0;
  return (all >> (threadIdx.x & 48)) & 0xFFFF;
}

// ---- router -------------------------------------------------------------------
// Elements of a token's row in LPT lanes of EPL: vectors of VW consecutive
// elements (16 bytes at most), one per lane, then the next LPT vectors.
template <typename L, int LPT, int EPL>
struct RowLayout {
  static constexpr int kMost = 16 / (int)sizeof(L);
  static constexpr int VW = EPL < kMost ? EPL : kMost;
  static __device__ __forceinline__ int index(int lane, int i) { return (i / VW) * (LPT * VW) + lane * VW + i % VW; }
};
// The lane's elements as fp32, -inf past E: whole vectors at any element's
// address, the row's last elements one by one.
template <typename L, int LPT, int EPL>
__device__ __forceinline__ void load_row(const L* row, int E, int lane, float (&v)[EPL]) {
  using R = RowLayout<L, LPT, EPL>;
  typedef L Vec __attribute__((ext_vector_type(R::VW), aligned(sizeof(L))));
#pragma unroll
  for (int c = 0; c < EPL / R::VW; ++c) {
    const int e0 = R::index(lane, c * R::VW);
    if (e0 + R::VW <= E) {
      const Vec y = *(const Vec*)(row + e0);
#pragma unroll
      for (int i = 0; i < R::VW; ++i) {
        const L x = y[i];
        v[c * R::VW + i] = load_f(&x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R::VW; ++i) v[c * R::VW + i] = e0 + i < E ? load_f(row + e0 + i) : -__builtin_inff();
    }
  }
}

// LPT lanes per token.  Logits become unsigned keys in the same order (-0 as
// +0); a bf16 key keeps 16 bits of value and holds 65535 - index below them,
// so that the largest key is the largest logit of the lowest index, and one
// maximum a round finds both.  An fp32 round takes the largest key, then the
// lowest index that holds it.  A chosen element's key becomes 0.  A -inf logit is
// never chosen (no key above that of -inf is left); a row with a NaN or +inf
// is rejected.  Weights are a softmax with the row's largest logit
// subtracted, sums in fp32.
// With up to 8 slots (SORTED) a lane first sorts its bf16 keys, of which at
// most 8 can be chosen: a round then is the maximum over the lanes' first keys,
// and the lane whose key was taken moves its others up (28 instructions
// instead of the 70 that look through 16 keys).
// What bounds it: 65536 tokens of 256 bf16 logits are 38 MB, 7.3 us at the copy
// rate; vector instructions (keys, sort, rounds) make it 16 us, 19 without the
// sort.  One token per wave (LPT 64) has a quarter of the elements per lane and a
// shorter chain, for few tokens, many experts or more than 16 slots.
constexpr uint32_t kNegInfKey = 0x007FFFFFu;   // ~bits of -inf
constexpr uint32_t kPosInfKey = 0xFF800000u;   // bits of +inf, top bit set
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// Of a packed bf16 key: the low 16 bits of the value are 0 again.
template <bool PACKED>
__device__ __forceinline__ float logit_of(uint32_t k) {
  return PACKED ? __uint_as_float(__float_as_uint(key_value(k)) & 0xFFFF0000u) : key_value(k);
}

// Exchanges v[I] and v[I + D] into falling order.
template <int I, int D, int EPL>
__device__ __forceinline__ void exchange(uint32_t (&v)[EPL]) {
  const uint32_t a = v[I], b = v[I + D];
  v[I] = max(a, b);
  v[I + D] = min(a, b);
}
// Falling order of v[F .. F + N - 1] by Batcher's odd-even merges: runs of P
// become runs of 2 P by exchanges at distances D = P, P / 2 .. 1, from place I on.
template <int F, int N, int P = 1, int D = 1, int I = 0, int EPL>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[EPL]) {
  if constexpr (P < N) {
    if constexpr (I + D < N) {
      if constexpr (I >= D % P && (I - D % P) / D % 2 == 0 && I / (2 * P) == (I + D) / (2 * P)) exchange<F + I, D>(v);
      sort_keys<F, N, P, D, I + 1>(v);
    } else if constexpr (D > 1) {
      sort_keys<F, N, P, D / 2, 0>(v);
    } else {
      sort_keys<F, N, 2 * P, 2 * P, 0>(v);
    }
  }
}
// The same of a run that rises and falls at most once.
template <int N, int D = N / 2, int I = 0, int EPL>
__device__ __forceinline__ void merge_keys(uint32_t (&v)[EPL]) {
  if constexpr (I < N) {
    if constexpr ((I & D) == 0) exchange<I, D>(v);
    merge_keys<N, D, I + 1>(v);
  } else if constexpr (D > 1) {
    merge_keys<N, D / 2, 0>(v);
  }
}
// The lane's SORTED largest keys in falling order at the front of v (behind them anything).
template <int SORTED, int EPL>
__device__ __forceinline__ void sort_largest(uint32_t (&v)[EPL]) {
  if constexpr (EPL <= SORTED) {
    sort_keys<0, EPL>(v);
  } else {
    static_assert(EPL == 2 * SORTED, "two sorted runs");
    sort_keys<0, SORTED>(v);
    sort_keys<SORTED, SORTED>(v);
#pragma unroll
    for (int i = 0; i < SORTED; ++i) v[i] = max(v[i], v[EPL - 1 - i]);
    merge_keys<SORTED>(v);
  }
}

// The choice of one token by LPT lanes (`lane` of them): lane s gets slot s's
// expert (-1 for none) and weight.
template <typename L, int LPT, int EPL, int SORTED>
__device__ __forceinline__ void route_token(const L* __restrict__ row, int E, int K, int renorm, int lane, int32_t& myid,
                                            float& myweight) {
  using R = RowLayout<L, LPT, EPL>;
  constexpr bool kPacked = sizeof(L) == 2;
  uint32_t key[EPL];
  float rest = 0.0f;   // sum over all experts
  uint32_t best;
  bool bad;
  {
    float v[EPL];
    load_row<L, LPT, EPL>(row, E, lane, v);
    uint32_t own = 0, least = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = order_key(v[i]);
      least = min(least, key[i]);
      if (kPacked) key[i] = (key[i] & 0xFFFF0000u) | (0xFFFFu - (uint32_t)R::index(lane, i));
      own = max(own, key[i]);
    }
    // A NaN's key lies above that of +inf or, with its sign set, below that of -inf.
    bad = group_any<LPT>(own >= kPosInfKey || least < kNegInfKey);
    best = group_max<LPT>(own);
    if (!renorm) {
      const float top = logit_of<kPacked>(best);
#pragma unroll
      for (int i = 0; i < EPL; ++i) rest += expf(v[i] - top);
      rest = group_sum<LPT>(rest);
    }
  }
  if constexpr (SORTED > 0) sort_largest<SORTED>(key);
  const uint32_t none = kPacked ? kNegInfKey | 0xFFFFu : kNegInfKey;   // keys up to this are -inf
  const float top = logit_of<kPacked>(best);
  float myval = -__builtin_inff();
  myid = -1;
  for (int s = 0; s < K; ++s) {
    // (a group with nothing left or a rejected row goes on with the wave and takes nothing)
    const bool take = best > none && !bad;
    uint32_t id, own = 0;
    if (SORTED) {
      id = 0xFFFFu - (best & 0xFFFFu);
      constexpr int N = EPL < SORTED ? EPL : SORTED;
      const bool first = key[0] == best;   // the lane whose first key was taken moves its others up
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t here = key[i], next = i + 1 < N ? key[i + 1] : 0u;
        key[i] = first ? next : here;
      }
      own = key[0];
    } else if (kPacked) {
      id = 0xFFFFu - (best & 0xFFFFu);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        key[i] = key[i] == best ? 0u : key[i];
        own = max(own, key[i]);
      }
    } else {
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)R::index(0, i) : at;
      at += at != 0xFFFFFFFFu ? lane * R::VW : 0;
      id = group_min<LPT>(at);
      const int gone = at == id ? (int)id - lane * R::VW : -1;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        key[i] = R::index(0, i) == gone ? 0u : key[i];
        own = max(own, key[i]);
      }
    }
    if (lane == s && take) {
      myval = logit_of<kPacked>(best);
      myid = (int)id;
    }
    best = group_max<LPT>(own);
  }
  const float ex = myid >= 0 ? expf(myval - top) : 0.0f;
  const float total = renorm ? group_sum<LPT>(ex) : rest;
  myweight = bad ? __builtin_nanf("") : myid >= 0 ? ex / total : 0.0f;
}

}  // namespace nvq
