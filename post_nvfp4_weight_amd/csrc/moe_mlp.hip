// A whole mixture-of-experts MLP with NVFP4 experts for a few tokens (at most
// 64), in two kernels (more than 8 tokens are routed by moe_topk's kernel before them):
//   1. routing (moe_topk's choice, or the caller's), then for each expert in use
//      and each of its tokens  act = w silu(G x) (U x),  w the token's weight;
//   2. out[t] = sum over its experts of g_e D act.
// Q = e2m1 * e4m3 is exact in bf16 and g is applied to the sums.  The
// activation between the products is held as a sum of bf16 parts: two where the
// result is bf16 (16 or more significant bits as long as it is above 2^-110), as one
// bf16 it would be the one value that the layer rounds to 8 bits before its end, for a
// product that waits for weights anyway; three where the result is fp32 (all 24
// bits above 2^-102): against 64 bits 2.1e-7 where two gave 2.4e-6 and fp32 throughout
// gives 1.9e-7 (4096 x 1024), for 64 x 2 of 8 experts 141 us instead of 126, one token 25.4 instead of 24.6.
//
// What bounds it is reading the weights of the experts in use once, and the
// instructions that expand them: 37 tokens x 8 of 256 experts, 2048 x 4096 and 4096 x
// 1024, take 128 and 67 us for 0.74 GB (3.7 TB/s; the vector units are busy 61 % of the
// first kernel), one token 17 and 8 us, most of it latency: the routing, the list of
// experts, then one round of cold weights.  The lanes are dealt as quads.h says (with
// lanes by rows the two kernels took 172 and 134 us for the 37 tokens, where the
// loads alone took 162 and 123).
#include <algorithm>

#include "common.h"
#include "dequant.h"
#include "kernels.h"
#include "quads.h"
#include "router.h"

namespace nvq {

namespace {

// On lambdas: one that is called twice and not inlined keeps what it captures in memory.
#define NVQ_INLINE __attribute__((always_inline))

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

constexpr int MW = 8;              // waves per workgroup of the first kernel
constexpr int down_waves(int NG) { return NG == 1 ? 16 : 8; }   // of the second (groups of 4 tokens need registers)
constexpr int kRoutedTokens = 8;   // up to this many are routed by the first kernel, one per wave
constexpr int kChunk = 512;
constexpr uint32_t kNone = 0x80000000u;   // an offset past every buffer (checked on the host), also with k's offsets added

// An expert and some of its tokens (bits), which are rows `row`, `row` + 1, .. of the activations in rising order.
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
  int parts;          // of an activation
  // workspace
  int32_t* count;     // entries
  float* bad;         // per token: 0, or NaN from the weight of a slot without an expert
  Entry* entries;
  float* scales;      // of each entry: g of its expert in the second product
  uint16_t* act;      // activations, act_row(h) elements per row
};

// Bf16 parts that an activation is the sum of.
constexpr int act_parts(bool out_bf16) { return out_bf16 ? 2 : 3; }
// A row of the activations: chunks of 512, and in each, for each j of a piece's
// four times 8 and for each part, the 16 pieces' 8: what one load takes is 256 bytes in a row.
__host__ __device__ __forceinline__ int64_t act_row(int64_t h, int parts) { return (h + kChunk - 1) / kChunk * kChunk * parts; }
// The first part; the others 128 behind each other.
__device__ __forceinline__ int64_t act_at(int k, int parts) {
  return ((int64_t)(k >> 9) * 512 + ((k >> 3) & 3) * 128) * parts + ((k >> 5) & 15) * 8 + (k & 7);
}

// 512 k of 16 channels.  s[i]: two scales, of the piece's halves (16 bits wide, as
// loaded: a conversion would wait for the load at the loop's end).
struct Chunk {
  u32x4 w[4];
  uint16_t s[4];
};
// Where a lane reads a tile of 16 channels from: cp, sp the tile's first codes
// and scales (the same for all lanes), off[i] and soff[i] the lane's channel i and
// piece in them.  Channels past the last repeat it.
struct TileAt {
  const uint8_t *cp, *sp;
  uint32_t off[4], soff[4];
  __device__ __forceinline__ void set(const uint8_t* codes, const uint8_t* scales, int64_t first, int64_t left, int64_t k, int lane) {
    cp = codes + first * (k / 2);
    sp = scales + first * (k / 16);
    const int a = (lane >> 2) & 3, piece = 4 * (lane >> 4) + (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t ch = (uint32_t)min((int64_t)(4 * a + i), left - 1);
      off[i] = ch * (uint32_t)(k / 2) + 16 * piece;
      soff[i] = ch * (uint32_t)(k / 16) + 2 * piece;
    }
  }
};
// Chunk ch.  REST: k may end inside it: pieces past k read their channel's first
// codes, under zero scales, and one that k ends in the middle of is read from 8 bytes
// before, inside its row, and moved.  The same loads on every path: one that a
// branch may skip makes the compiler wait for those issued behind it, which are
// the ones ahead of time.
template <bool REST>
__device__ __forceinline__ void load_chunk(const TileAt& t, int ch, int64_t k, int lane, Chunk& x) {
  const uint32_t left = REST ? (uint32_t)max((int64_t)0, k - (int64_t)ch * kChunk) : 0, at = 32 * (4 * (lane >> 4) + (lane & 3));
  const bool none = REST && at >= left, half = REST && at + 16 == left;
  const int64_t c0 = (int64_t)ch * 256, s0 = (int64_t)ch * 32;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (REST) {
      const int64_t c = none ? (int64_t)t.off[i] - at / 2 : t.off[i] + c0 - (half ? 8 : 0);
      const int64_t s = none ? (int64_t)t.soff[i] - at / 16 : t.soff[i] + s0 - (half ? 1 : 0);
      x.w[i] = *(const u32x4_any*)(t.cp + c);
      x.s[i] = *(const u16_any*)(t.sp + s);
    } else {
      x.w[i] = *(const u32x4_any*)(t.cp + c0 + t.off[i]);
      x.s[i] = *(const u16_any*)(t.sp + s0 + t.soff[i]);
    }
  }
}
// What load_chunk<true> has loaded, as it stands for (after the wait for it).
template <bool REST>
__device__ __forceinline__ void settle(Chunk& x, int ch, int64_t k, int lane) {
  if (!REST) return;
  const uint32_t left = (uint32_t)max((int64_t)0, k - (int64_t)ch * kChunk), at = 32 * (4 * (lane >> 4) + (lane & 3));
  const bool none = at >= left, half = at + 16 == left;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.w[i][0] = half ? x.w[i][2] : x.w[i][0];
    x.w[i][1] = half ? x.w[i][3] : x.w[i][1];
    x.s[i] = none ? (uint16_t)0 : half ? (uint16_t)(x.s[i] >> 8) : x.s[i];
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
__device__ __forceinline__ f32x4 mfma(bf16x8 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// An entry, the same for the whole wave.  A lane's column
// stands for token number 4 g + (l % 16) / 4 of the entry in group g (-1 for none).
template <int NG>
struct Columns {
  Entry e;
  int token[NG];
  __device__ __forceinline__ void set(const Entry& in, int lane) {
    e.expert = __builtin_amdgcn_readfirstlane(in.expert);
    e.row = __builtin_amdgcn_readfirstlane(in.row);
    e.tokens = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)in.tokens) |
               (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(in.tokens >> 32)) << 32;
    const int mine = (lane >> 2) & 3;
    uint64_t left = e.tokens;
#pragma unroll
    for (int g4 = 0; g4 < NG; ++g4) {
      token[g4] = -1;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (!left) break;
        token[g4] = mine == t ? __builtin_ctzll(left) : token[g4];
        left &= left - 1;
      }
    }
  }
};

__host__ __device__ __forceinline__ int64_t most_entries(int64_t T, int64_t E, int64_t K, int per) {
  return (E < T * K ? E : T * K) + T * K / per;
}
size_t up_lds(int64_t T, int64_t E, int64_t K, int per) { return E * 8 + T * K * 12 + most_entries(T, E, K, per) * (sizeof(Entry) + 4); }

// Kernel 1.  Every workgroup routes all tokens for itself (a launch for it
// alone would cost more), lists the entries (of up to 4 NG tokens), then takes
// items, 16 channels of gate and of up of one entry, in turn with the other workgroups;
// the even waves take gate, the odd ones up, each four a part of k, their
// sums added in wave order through LDS.  Weights are loaded FD chunks ahead.
template <typename L, int EPL, int NG, bool REST>
__global__ __launch_bounds__(64 * MW, 4) void moe_up_kernel(const MoeMlp a) {
  constexpr int KP = MW / 2, FD = NG == 1 ? 2 : 1;
  __shared__ __attribute__((aligned(16))) float part[MW][4 * NG][16];
  __shared__ int s_count;
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  const int slots = a.T * a.K;
  Entry* list = (Entry*)dyn;
  uint64_t* mask = (uint64_t*)(list + most_entries(a.T, a.E, a.K, 4 * NG));
  int32_t* ids = (int32_t*)(mask + a.E);
  float* ws = (float*)(ids + slots);
  float* wrow = ws + slots;   // of each row of the activations: its token's weight
  float* scale = wrow + slots;   // of each entry: its expert's
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
      uint64_t tokens = e0 + lane < a.E ? mask[e0 + lane] : 0;
      const int cnt = __popcll(tokens), ne = (cnt + 4 * NG - 1) / (4 * NG);
      const int incl = wave_inclusive(cnt), nincl = wave_inclusive(ne);
      int row = rows + incl - cnt;
      for (int i = 0; i < ne; ++i, row += 4 * NG) {
        uint64_t part = tokens;
        if (i + 1 < ne) {
          part = 0;
          for (int b = 0; b < 4 * NG; ++b, tokens &= tokens - 1) part |= tokens & -tokens;
        }
        list[n + nincl - ne + i] = Entry{e0 + lane, row, part};
      }
      n += __builtin_amdgcn_readlane(nincl, 63);
      rows += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) s_count = n;
  }
  __syncthreads();
  const int used = __builtin_amdgcn_readfirstlane(s_count);
  for (int i = tid; i < used; i += 64 * MW) {
    const Entry e = list[i];
    scale[i] = a.ug[e.expert];
    if (blockIdx.x == 0) {
      a.entries[i] = e;
      a.scales[i] = a.dg[e.expert];
    }
    int row = e.row;
    for (uint64_t left = e.tokens; left; left &= left - 1, ++row) {
      const int t = __builtin_ctzll(left);
      float w = 0.0f;
      for (int s = 0; s < a.K; ++s) w += ids[t * a.K + s] == e.expert ? ws[t * a.K + s] : 0.0f;
      wrow[row] = w;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (tid == 0) *a.count = used;
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
  if ((int)blockIdx.x >= items) return;
  const int kp = wave >> 1, f = wave & 1;
  const int chunks = (int)((a.d + kChunk - 1) / kChunk), mine = chunks > kp ? (chunks - kp + KP - 1) / KP : 0;   // of k, of the wave
  const __amdgpu_buffer_rsrc_t xbuf = buffer_of(a.X, (uint32_t)(((a.T - 1) * a.ldx + a.d) * 2));
  const int piece = 4 * (lane >> 4) + (lane & 3);

  // What is loaded next: the li-th of the wave's chunks of item `lit`.
  int lit = blockIdx.x, li = 0;
  TileAt tile;
  auto locate = [&](int it) NVQ_INLINE {
    it = min(it, items - 1);   // (behind the last item its weights are loaded again and not used)
    const int at = it / nt;
    const int64_t e = __builtin_amdgcn_readfirstlane(list[at].expert), o0 = 16 * (int64_t)(it - at * nt);
    tile.set(a.ucodes, a.uscales, e * 2 * a.h + f * a.h + o0, a.h - o0, a.d, lane);
  };
  auto load_next = [&](Chunk& b) NVQ_INLINE {
    load_chunk<REST>(tile, kp + KP * li, a.d, lane, b);
    if (++li == mine) {
      li = 0;
      lit += gridDim.x;
      locate(lit);
    }
  };

  f32x4 acc[NG][4];
  auto clear = [&]() NVQ_INLINE {
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  int item = blockIdx.x;
  Columns<NG> cur;
  auto enter = [&](int it, Columns<NG>& cols) NVQ_INLINE {
    it = min(it, items - 1);
    cols.set(list[it / nt], lane);
  };
  u32x4 x[NG][4];
  auto load_x = [&](const Columns<NG>& of, int ch) NVQ_INLINE {   // zeros where there is no token and from k on
    const int k0 = ch * kChunk + 32 * piece;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t row = of.token[g] >= 0 ? (uint32_t)(of.token[g] * a.ldx * 2) : kNone;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[g][j] = load16(xbuf, !REST || k0 + 8 * j < a.d ? row + (uint32_t)(k0 + 8 * j) * 2 : kNone);
    }
  };
  auto finish = [&]() NVQ_INLINE {   // the item's activations
    const int o0 = 16 * (item % nt), n = __popcll(cur.e.tokens);
    const float g1 = scale[item / nt];
#pragma unroll
    for (int g = 0; g < NG; ++g)
      if (4 * g < n) part[wave][4 * g + ((lane >> 2) & 3)][4 * (lane >> 4) + (lane & 3)] = quad_sum(acc[g], lane);
    __syncthreads();
    for (int i = tid; i < 16 * n; i += 64 * MW) {
      const int t = i >> 4, ch = i & 15, k = o0 + ch;
      if (k >= a.h) continue;
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < MW; w += 2) {
        gate += part[w][t][ch];
        up += part[w + 1][t][ch];
      }
      gate *= g1;
      up *= g1;
      const float z = expf(-fabsf(gate)), one = 1.0f / (1.0f + z);
      const float v = gate * (gate >= 0.0f ? one : z * one) * up * wrow[cur.e.row + t];
      uint16_t* to = a.act + (cur.e.row + t) * act_row(a.h, a.parts) + act_at(k, a.parts);
      float rest = v;
      for (int q = 0; q < a.parts; ++q, to += 128) {
        const __bf16 b = (__bf16)rest;
        *to = __builtin_bit_cast(uint16_t, b);
        rest = fabsf((float)b) < __builtin_inff() ? rest - (float)b : 0.0f;   // (an infinity or NaN is in the first part alone)
      }
    }
    __syncthreads();
  };

  clear();
  enter(item, cur);
  if (mine == 0) {   // (k has fewer chunks than there are parts)
    for (; item < items; item += gridDim.x) {
      enter(item, cur);
      finish();
    }
    return;
  }
  // Loads return in the order of their issue, so what is needed first, the
  // activations, goes out ahead of the weights of FD chunks on.
  Chunk buf[FD];
  locate(lit);
#pragma unroll
  for (int b = 0; b < FD; ++b) {
    load_next(buf[b]);
    __builtin_amdgcn_sched_barrier(0);
    if (b == 0) load_x(cur, kp);
    __builtin_amdgcn_sched_barrier(0);
  }
  int i = 0;
  auto consume = [&](Chunk& b) NVQ_INLINE {
    settle<REST>(b, kp + KP * i, a.d, lane);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 v = expand(b.w[n], b.s[n], j);
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[g][n] = mfma(v, x[g][j], acc[g][n]);
      }
    __builtin_amdgcn_sched_barrier(0);
    const bool last = i + 1 == mine;
    Columns<NG> next = cur;
    if (last) enter(item + gridDim.x, next);
    load_x(next, kp + KP * (last ? 0 : i + 1));
    __builtin_amdgcn_sched_barrier(0);
    load_next(b);
    __builtin_amdgcn_sched_barrier(0);
    ++i;
    if (last) {
      finish();
      clear();
      i = 0;
      item += gridDim.x;
      cur = next;
    }
  };
  // (no way out from between the chunks, which would be another path to the first)
  int left = (items - 1 - (int)blockIdx.x) / (int)gridDim.x * mine + mine;
  for (; left >= FD; left -= FD) {
#pragma unroll
    for (int b = 0; b < FD; ++b) consume(buf[b]);
  }
#pragma unroll
  for (int b = 0; b < FD - 1; ++b)
    if (b < left) consume(buf[b]);
}

// Kernel 2: 16 output channels per workgroup.  The units (chunks of an entry's
// activations) of all entries lie in a row, which the waves share in equal
// runs.  A wave adds its entries' sums times g to totals of its own in LDS,
// [token][channel]; the waves' totals are added in wave order.  Columns without
// a token are added nowhere (a rejected weight row makes them NaN).
template <int OUT_BF16, int NG, bool REST>
__global__ __launch_bounds__(64 * down_waves(NG), NG == 1 ? 4 : OUT_BF16 ? 3 : 2) void moe_down_kernel(const MoeMlp a) {
  constexpr int DW = down_waves(NG), FD = 1, PARTS = act_parts(OUT_BF16);
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  float* totals = (float*)dyn;   // [wave][token][16]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t o0 = (int64_t)blockIdx.x * 16, stride = act_row(a.h, PARTS);
  const int used = *a.count, per = (int)((a.h + kChunk - 1) / kChunk);
  Entry* list = (Entry*)(totals + DW * a.T * 16);
  float* scale = (float*)(list + most_entries(a.T, a.E, a.K, 4 * NG));
  for (int i = tid; i < (int)most_entries(a.T, a.E, a.K, 4 * NG); i += 64 * DW) {   // (without waiting for the count)
    list[i] = a.entries[i];
    scale[i] = a.scales[i];
  }
  for (int i = tid; i < DW * a.T * 16; i += 64 * DW) totals[i] = 0.0f;
  float* mine = totals + wave * a.T * 16 + 4 * (lane >> 4) + (lane & 3);
  __syncthreads();
  const int units = used * per;
  int at = (int)((int64_t)units * wave / DW);
  const int end = (int)((int64_t)units * (wave + 1) / DW);

  if (at < end) {
    int ea = at / per, ep = at - ea * per, la = ea, lp = ep;   // unit ep of entry ea; the next to load
    TileAt tile;
    auto locate = [&](int entry) NVQ_INLINE {
      const int64_t e = __builtin_amdgcn_readfirstlane(list[entry].expert);
      tile.set(a.dcodes, a.dscales, e * a.m + o0, a.m - o0, a.h, lane);
    };
    auto load_next = [&](Chunk& b) NVQ_INLINE {
      load_chunk<REST>(tile, lp, a.h, lane, b);
      if (++lp == per) {
        lp = 0;
        la = min(la + 1, used - 1);   // (behind the last entry its weights are loaded again and not used)
        locate(la);
      }
    };
    const int piece = 4 * (lane >> 4) + (lane & 3);
    u32x4 x[NG][4][PARTS];
    auto load_act = [&](const Columns<NG>& of, int p) NVQ_INLINE {   // zeros where there is no token and from h on
      const __amdgpu_buffer_rsrc_t rs = buffer_of(a.act + of.e.row * stride, (uint32_t)(__popcll(of.e.tokens) * stride * 2));
      const int k0 = p * kChunk + 32 * piece;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t row = of.token[g] >= 0 ? (uint32_t)((4 * g + ((lane >> 2) & 3)) * stride * 2 + p * (1024 * PARTS) + piece * 16) : kNone;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t off = !REST || k0 + 8 * j < a.h ? row + j * (256 * PARTS) : kNone;
#pragma unroll
          for (int q = 0; q < PARTS; ++q) x[g][j][q] = load16(rs, off + 256 * q);
        }
      }
    };
    f32x4 acc[NG][4];
    auto clear = [&]() NVQ_INLINE {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[g][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    clear();
    Columns<NG> cur;
    cur.set(list[ea], lane);
    float g2 = scale[ea];
    Chunk buf[FD];
    locate(la);
    // (in the loop's order, as in the first kernel)
#pragma unroll
    for (int b = 0; b < FD; ++b) {
      load_next(buf[b]);
      __builtin_amdgcn_sched_barrier(0);
      if (b == 0) load_act(cur, ep);
      __builtin_amdgcn_sched_barrier(0);
    }
    auto consume = [&](Chunk& b) NVQ_INLINE {
      settle<REST>(b, ep, a.h, lane);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 v = expand(b.w[n], b.s[n], j);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) acc[g][n] = mfma(v, x[g][j][q], acc[g][n]);
        }
      __builtin_amdgcn_sched_barrier(0);
      ++at;
      const bool cross = ep + 1 == per;
      Columns<NG> next = cur;
      float gnext = g2;
      if (cross) {
        ea = min(ea + 1, used - 1);
        next.set(list[ea], lane);
        gnext = scale[ea];
      }
      ep = cross ? 0 : ep + 1;
      load_act(next, ep);
      __builtin_amdgcn_sched_barrier(0);
      load_next(b);
      __builtin_amdgcn_sched_barrier(0);
      if (cross || at == end) {   // the entry's sums to the tokens' totals
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (4 * g >= __popcll(cur.e.tokens)) break;
          const float v = quad_sum(acc[g], lane);
          if (cur.token[g] >= 0) mine[cur.token[g] * 16] += v * g2;
        }
        clear();
      }
      cur = next;
      g2 = gnext;
    };
    int left = end - at;
    for (; left >= FD; left -= FD) {
#pragma unroll
      for (int b = 0; b < FD; ++b) consume(buf[b]);
    }
#pragma unroll
    for (int b = 0; b < FD - 1; ++b)
      if (b < left) consume(buf[b]);
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += 64 * DW) {
    const int t = i >> 4, ch = i & 15;
    if (o0 + ch >= a.m) continue;
    float v = a.bad[t];
#pragma unroll
    for (int w = 0; w < DW; ++w) v += totals[(w * a.T + t) * 16 + ch];
    if (OUT_BF16) ((__bf16*)a.out)[t * a.ldo + o0 + ch] = (__bf16)v;
    else ((float*)a.out)[t * a.ldo + o0 + ch] = v;
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Groups of 4 tokens per entry.  An expert with more tokens than an entry holds
// has its weights read (from the caches) and expanded again for the next one; two
// groups take twice the matrix instructions and registers.  us with one / two / four,
// tokens per expert on average: 37 tokens x 8 of 256 experts (1.2) 203 / 222 / 288,
// 32 x 6 of 64 (3) 117 / 123 / 166, 16 x 2 of 8 (4) 82 / 81 / 103, 64 x 2 of 8 (16)
// 187 / 152 / 155.
int groups(int64_t T, int64_t E, int64_t K) { return T * K < 4 * E ? 1 : 2; }

template <int NG>
hipError_t launch(MoeMlp& a, int logits_bf16, int out_bf16, hipStream_t s) {
  const int64_t items = most_entries(a.T, a.E, a.K, 4 * NG) * ((a.h + 15) / 16);
  const size_t lds = up_lds(a.T, a.E, a.K, 4 * NG);
  const dim3 up((unsigned)std::min<int64_t>(items, 512)), down((unsigned)((a.m + 15) / 16));
#define NVQ_UP(L, EPL)                                                                                          \
  do {                                                                                                          \
    if (a.d % kChunk) hipLaunchKernelGGL((moe_up_kernel<L, EPL, NG, true>), up, dim3(64 * MW), lds, s, a);      \
    else hipLaunchKernelGGL((moe_up_kernel<L, EPL, NG, false>), up, dim3(64 * MW), lds, s, a);                  \
  } while (0)
  // (elements per lane as moe_topk takes them: the sum over all experts has their order)
#define NVQ_UP_BY(L)                   \
  do {                                 \
    if (a.E <= 64) NVQ_UP(L, 1);       \
    else if (a.E <= 128) NVQ_UP(L, 2); \
    else if (a.E <= 256) NVQ_UP(L, 4); \
    else if (a.E <= 512) NVQ_UP(L, 8); \
    else NVQ_UP(L, 16);                \
  } while (0)
  if (!a.logits) NVQ_UP(float, 1);
  else if (logits_bf16) NVQ_UP_BY(uint16_t);
  else NVQ_UP_BY(float);
#undef NVQ_UP_BY
#undef NVQ_UP
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int DW = down_waves(NG);
  const size_t totals = (size_t)DW * a.T * 16 * sizeof(float) + most_entries(a.T, a.E, a.K, 4 * NG) * (sizeof(Entry) + 4);
#define NVQ_DOWN(OUT)                                                                                           \
  do {                                                                                                          \
    if (a.h % kChunk) hipLaunchKernelGGL((moe_down_kernel<OUT, NG, true>), down, dim3(64 * DW), totals, s, a);  \
    else hipLaunchKernelGGL((moe_down_kernel<OUT, NG, false>), down, dim3(64 * DW), totals, s, a);              \
  } while (0)
  if (out_bf16) NVQ_DOWN(1);
  else NVQ_DOWN(0);
#undef NVQ_DOWN
  return hipGetLastError();
}

}  // namespace

// Layout: count, the tokens' `bad`, the entries, their scales, the activations (of as many parts as any result takes).
size_t nvfp4_moe_mlp_workspace(int64_t T, int64_t E, int64_t K, int64_t h) {
  return 512 + up256(most_entries(T, E, K, 4) * sizeof(Entry)) + up256(most_entries(T, E, K, 4) * sizeof(float)) + (size_t)(T * K) * act_row(h, act_parts(false)) * 2;
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
  a.parts = act_parts(out_bf16);
  char* p = (char*)ws;
  a.count = (int32_t*)p;
  a.bad = (float*)(p + 256);
  a.entries = (Entry*)(p + 512);
  a.scales = (float*)((char*)a.entries + up256(most_entries(T, E, K, 4) * sizeof(Entry)));
  a.act = (uint16_t*)((char*)a.scales + up256(most_entries(T, E, K, 4) * sizeof(float)));
  if (logits && T > kRoutedTokens) {
    const hipError_t e = moe_topk_launch(logits, logits_bf16, T, E, ldl, K, renorm, ids, weights, s);
    if (e != hipSuccess) return e;
    a.logits = nullptr;
  }
  return groups(T, E, K) == 1 ? launch<1>(a, logits_bf16, out_bf16, s) : launch<2>(a, logits_bf16, out_bf16, s);
}

}  // namespace nvq
