// The gated activation between the two products of an MLP and its gradient.
// X = [gate | up], s = 1 / (1 + exp(-gate)):
//   forward:  out = gate s up
//   backward: dgate = dout up s (1 + gate (1 - s)),  dup = dout gate s
// in fp32, rounded once.  Both are streams, bound by memory: 3 and 5 values of traffic
// per output, at 5.0 TB/s for 131072 x 1024 bf16 (162 us), the gradient at 5.8 TB/s for
// 5003 x 2060 fp32 (35 us).
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace nvq {

namespace {

// Vectors of 16 bytes at any element's place.
template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T V __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
};
__device__ __forceinline__ float as_f(float v) { return v; }
__device__ __forceinline__ float as_f(__bf16 v) { return (float)v; }

// The first `left` of N elements (the others 0).
template <typename T>
__device__ __forceinline__ typename Vec<T>::V load_part(const T* p, int64_t left) {
  typename Vec<T>::V v;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) v[i] = i < left ? p[i] : (T)0.0f;
  return v;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const typename Vec<T>::V& v, int64_t left) {
  if (left >= Vec<T>::N) {
    *(typename Vec<T>::V*)p = v;
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      if (i < left) p[i] = v[i];
  }
}

// s and 1 - s without overflow on either side.
__device__ __forceinline__ void sigmoid(float g, float& s, float& rest) {
  const float z = expf(-fabsf(g)), a = 1.0f / (1.0f + z), b = z * a;
  s = g >= 0.0f ? a : b;
  rest = g >= 0.0f ? b : a;
  if (g != g) s = rest = g;
}

// Vectors per thread.  us with 1 / 2 / 4: 131072 x 1024 bf16 180 / 179 / 175, the
// gradient of 5003 x 2060 fp32 34 / 35 / 42 (another card than above).
constexpr int SU = 2;

// cpr: vectors per row; units = n cpr.  T in, O out (forward only).
template <typename T, typename O, bool GRAD>
__global__ __launch_bounds__(256) void swiglu_kernel(const T* __restrict__ X, int64_t ldx, const T* __restrict__ dout, int64_t ldd,
                                                     int64_t h, int64_t cpr, int64_t units, O* __restrict__ out, int64_t ldo) {
  constexpr int N = Vec<T>::N;
  for (int64_t base = (int64_t)blockIdx.x * (256 * SU); base < units; base += (int64_t)gridDim.x * (256 * SU)) {
    typename Vec<T>::V g[SU], u[SU], d[SU];
    int64_t row[SU], col[SU];
#pragma unroll
    for (int j = 0; j < SU; ++j) {
      const int64_t i = base + j * 256 + threadIdx.x;
      if (i >= units) continue;
      row[j] = units <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / (uint32_t)cpr) : i / cpr;
      col[j] = (i - row[j] * cpr) * N;
      const T* p = X + row[j] * ldx + col[j];
      const T* q = GRAD ? dout + row[j] * ldd + col[j] : nullptr;
      if (col[j] + N <= h) {
        g[j] = *(const typename Vec<T>::V*)p;
        u[j] = *(const typename Vec<T>::V*)(p + h);
        if (GRAD) d[j] = *(const typename Vec<T>::V*)q;
      } else {
        g[j] = load_part(p, h - col[j]);
        u[j] = load_part(p + h, h - col[j]);
        if (GRAD) d[j] = load_part(q, h - col[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < SU; ++j) {
      const int64_t i = base + j * 256 + threadIdx.x;
      if (i >= units) continue;
      O* o = out + row[j] * ldo + col[j];
      if constexpr (GRAD) {
        typename Vec<T>::V dg, du;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float gv = as_f(g[j][e]), uv = as_f(u[j][e]), dv = as_f(d[j][e]);
          float s, rest;
          sigmoid(gv, s, rest);
          dg[e] = (T)(dv * uv * (s * (1.0f + gv * rest)));
          du[e] = (T)(dv * (gv * s));
        }
        store_vec<T>(o, dg, h - col[j]);
        store_vec<T>(o + h, du, h - col[j]);
      } else {
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float s, rest;
          sigmoid(as_f(g[j][e]), s, rest);
          v[e] = as_f(g[j][e]) * s * as_f(u[j][e]);
        }
        if (col[j] + N <= h) {
          // (8 bf16 in give two vectors of fp32, 4 fp32 in half a vector of bf16)
          typedef O Out __attribute__((ext_vector_type(N), aligned(sizeof(O))));
          Out r;
#pragma unroll
          for (int e = 0; e < N; ++e) r[e] = (O)v[e];
          *(Out*)o = r;
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (col[j] + e < h) o[e] = (O)v[e];
        }
      }
    }
  }
}

template <typename T, typename O, bool GRAD>
hipError_t launch(const void* X, int64_t ldx, const void* dout, int64_t ldd, int64_t n, int64_t h, void* out, int64_t ldo,
                  hipStream_t s) {
  const int64_t cpr = (h + Vec<T>::N - 1) / Vec<T>::N, units = n * cpr;
  const unsigned blocks = (unsigned)std::min<int64_t>((units + 256 * SU - 1) / (256 * SU), 1 << 20);
  hipLaunchKernelGGL((swiglu_kernel<T, O, GRAD>), dim3(blocks), dim3(256), 0, s, (const T*)X, ldx, (const T*)dout, ldd, h, cpr,
                     units, (O*)out, ldo);
  return hipGetLastError();
}

}  // namespace

hipError_t swiglu_launch(const void* X, int x_bf16, int64_t n, int64_t h, int64_t ldx, void* out, int out_bf16, int64_t ldo,
                         hipStream_t s) {
  if (x_bf16) return out_bf16 ? launch<__bf16, __bf16, false>(X, ldx, nullptr, 0, n, h, out, ldo, s)
                              : launch<__bf16, float, false>(X, ldx, nullptr, 0, n, h, out, ldo, s);
  return out_bf16 ? launch<float, __bf16, false>(X, ldx, nullptr, 0, n, h, out, ldo, s)
                  : launch<float, float, false>(X, ldx, nullptr, 0, n, h, out, ldo, s);
}

hipError_t swiglu_backward_launch(const void* dout, int64_t ldd, const void* X, int bf16, int64_t n, int64_t h, int64_t ldx,
                                  void* dX, int64_t lddx, hipStream_t s) {
  return bf16 ? launch<__bf16, __bf16, true>(X, ldx, dout, ldd, n, h, dX, lddx, s)
              : launch<float, float, true>(X, ldx, dout, ldd, n, h, dX, lddx, s);
}

}  // namespace nvq
