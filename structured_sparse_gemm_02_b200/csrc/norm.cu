// Layer norm in front of a pruned linear layer: forward (with an optional
// residual sum, and an int8 output for the fixed-point layers) and backward
// (with the reduction of the weight's gradient).
//
//   h  = x (+ residual, rounded to the activations' type)
//   mu = mean(h), r = 1 / sqrt(mean((h - mu)^2) + eps)
//   y  = (h - mu) r gamma + beta
// backward, with z = (h - mu) r and g = dy gamma:
//   dx = r (g - mean(g) - z mean(g z)) (+ the gradient that reaches h by the residual path)
//   dgamma = sum over rows of dy z, dbeta = sum over rows of dy
//
// Everything is bound by memory: a row is read once, kept in registers (the
// variance is a second pass over the registers, so a large mean costs no
// precision), and written once.  All sums are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gather.cuh"
#include "host.cuh"
#include "sm100.cuh"
#include "spgemm.h"

namespace spg {
namespace norm {

// ---- pairs of fp32 values, which the FMA pipe takes two at a time ----------------------
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_of(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 f2_get(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// 16 bytes of a row as they lie in memory, and as pairs of fp32 values.
template <class T>
struct Vec {
  static constexpr int VE = 16 / sizeof(T), VP = VE / 2;
  uint4 raw;
  __device__ Vec() : raw(make_uint4(0u, 0u, 0u, 0u)) {}
  __device__ __forceinline__ void get(f2 (&v)[VP]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4) {
      v[0] = f2_of(__uint_as_float(w[0]), __uint_as_float(w[1]));
      v[1] = f2_of(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (std::is_same<T, __half>::value) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          v[k] = f2_of(f.x, f.y);
        } else {
          v[k] = f2_of(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
        }
      }
    }
  }
  __device__ __forceinline__ void set(const f2 (&v)[VP]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
      const float2 a = f2_get(v[0]), b = f2_get(v[1]);
      w[0] = __float_as_uint(a.x); w[1] = __float_as_uint(a.y);
      w[2] = __float_as_uint(b.x); w[3] = __float_as_uint(b.y);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = f2_get(v[k]);
        if constexpr (std::is_same<T, __half>::value)
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(f.y), "f"(f.x));
        else
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(f.y), "f"(f.x));
      }
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// How rows meet vectors: SURE < 0: element by element (rows that are not 16-byte
// aligned); otherwise in vectors, of which the first SURE of each thread are
// whole and inside the row, and the others checked (a row's last elements move
// one by one).  A check a vector is a third of the forward kernel's
// instructions, so the kernels exist with none, with one and with all checked.
constexpr int ELEMENTS = -1;

// The first n < VE elements of a row's last vector (all its loads at once: one
// after the other they held the row up by 2 us).
template <class T>
__device__ __forceinline__ uint4 load_last(const T* p, int n) {
  constexpr int VE = Vec<T>::VE;
  if constexpr (sizeof(T) == 4) {
    return make_uint4(n > 0 ? __float_as_uint(p[0]) : 0u, n > 1 ? __float_as_uint(p[1]) : 0u,
                      n > 2 ? __float_as_uint(p[2]) : 0u, 0u);
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
    uint32_t e[VE];
#pragma unroll
    for (int i = 0; i < VE - 1; ++i) e[i] = i < n ? s[i] : 0u;
    e[VE - 1] = 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
}
template <class T>
__device__ __forceinline__ void store_last(T* p, const uint4& v, int n) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) p[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

// VE elements at p, of which the first n are inside the row; the others are 0.
// ONCE: data that is read once, which leaves L1 to the weights.
template <bool VECTORS, bool ONCE, class T>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int n) {
  Vec<T> v;
  if constexpr (!VECTORS) {
    f2 f[Vec<T>::VP];
#pragma unroll
    for (int i = 0; i < Vec<T>::VP; ++i)
      f[i] = f2_of(2 * i < n ? to_f(p[2 * i]) : 0.f, 2 * i + 1 < n ? to_f(p[2 * i + 1]) : 0.f);
    v.set(f);
  } else if (n >= Vec<T>::VE) {
    if constexpr (ONCE)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.raw.x), "=r"(v.raw.y), "=r"(v.raw.z), "=r"(v.raw.w)
                   : "l"(p));
    else
      v.raw = *reinterpret_cast<const uint4*>(p);
  } else {
    v.raw = load_last(p, n);
  }
  return v;
}
template <bool VECTORS, class T>
__device__ __forceinline__ void store_vec(T* p, const f2 (&f)[Vec<T>::VP], int n) {
  if constexpr (!VECTORS) {
#pragma unroll
    for (int i = 0; i < Vec<T>::VP; ++i) {
      const float2 e = f2_get(f[i]);
      if (2 * i < n) p[2 * i] = from_f<T>(e.x);
      if (2 * i + 1 < n) p[2 * i + 1] = from_f<T>(e.y);
    }
  } else {
    Vec<T> v;
    v.set(f);
    if (n >= Vec<T>::VE)
      *reinterpret_cast<uint4*>(p) = v.raw;
    else
      store_last(p, v.raw, n);
  }
}

// VE elements of gamma or beta, in fp32 (W32) or in the activations' type.
template <bool VECTORS, bool W32, class T>
__device__ __forceinline__ void load_weight(f2 (&w)[Vec<T>::VP], const void* p, int c, int n) {
  if constexpr (W32 || sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Vec<T>::VP; k += 2) {
      f2 q[2] = {0ull, 0ull};
      if (2 * k < n)
        load_vec<VECTORS, false>(static_cast<const float*>(p) + c + 2 * k, n - 2 * k).get(q);
      w[k] = q[0];
      w[k + 1] = q[1];
    }
  } else {
    load_vec<VECTORS, false>(static_cast<const T*>(p) + c, n).get(w);
  }
}
template <bool VECTORS, class T>
__device__ __forceinline__ void load_weight(f2 (&w)[Vec<T>::VP], const void* p, int f32, int c, int n) {
  f32 ? load_weight<VECTORS, true, T>(w, p, c, n) : load_weight<VECTORS, false, T>(w, p, c, n);
}

// 0 for the elements of a vector past its row's end.
template <int VP>
__device__ __forceinline__ void clear_past(f2 (&v)[VP], int n) {
  if (n >= 2 * VP) return;
#pragma unroll
  for (int i = 0; i < VP; ++i) {
    const float2 e = f2_get(v[i]);
    v[i] = f2_of(2 * i < n ? e.x : 0.f, 2 * i + 1 < n ? e.y : 0.f);
  }
}

// Threads of the largest block: 16384 columns are 2048 vectors of a 16-bit type
// or 4096 of fp32, at most four a thread.
template <class T, int NV>
constexpr int max_threads() { return sizeof(T) == 4 && NV == 4 ? 1024 : 512; }

// Sum over the 2^lg lanes of a warp that share a row.
__device__ __forceinline__ float lanes_sum(float v, int lg) {
  for (int o = (1 << lg) >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// red[0] + ... + red[n - 1], read in 16-byte pieces (0 up to the next multiple of four).
__device__ __forceinline__ float sum_of(const float* red, int n) {
  float4 s = *reinterpret_cast<const float4*>(red);
  for (int w = 4; w < n; w += 4) {
    const float4 q = *reinterpret_cast<const float4*>(red + w);
    s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
  }
  return (s.x + s.y) + (s.z + s.w);
}
// Sum over the block through `red` (one float a warp, up to a multiple of
// four, the unused ones 0); the caller alternates between two such arrays, so
// one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return sum_of(red, blockDim.x >> 5);
}

struct FwdArgs {
  const void* x;
  const void* res;
  void* h;
  void* y;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  int64_t ldx, ldres, ldh, ldy;
  int M, C, lg, wf32, s8;
  float eps, qscale;
};

// y = (h - mu) rstd gamma + beta of a thread's vectors (v holds h - mu), stored in its type or as int8 codes.
template <class T, int NV, int SURE, bool W32, bool BETA, bool S8>
__device__ __forceinline__ void ln_finish(const FwdArgs& a, f2 (&v)[NV][Vec<T>::VP], int64_t row, int t, int threads,
                                          f2 r2) {
  constexpr int VE = Vec<T>::VE, VP = Vec<T>::VP;
  constexpr bool VECTORS = SURE >= 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
    const int n = k < SURE ? VE : a.C - c;
    if (n <= 0) continue;
    f2 g[VP], b[VP];
    load_weight<VECTORS, W32, T>(g, a.gamma, c, n);
    if constexpr (BETA) load_weight<VECTORS, W32, T>(b, a.beta, c, n);
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const f2 z = f2_mul(v[k][i], r2);
      v[k][i] = BETA ? f2_fma(z, g[i], b[i]) : f2_mul(z, g[i]);
    }
    if constexpr (S8) {
      // clamp(rne(y qscale)): the conversion and the packing saturate at 127 and
      // keep a NaN's 0; -128 is cut off before them by a maximum that passes NaN on
      uint32_t w[VE / 4];
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        int code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = f2_get(f2_mul(v[k][(i + e) / 2], f2_of(a.qscale, a.qscale)));
          float f;
          asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(e & 1 ? y.y : y.x), "f"(-127.f));
          code[e] = __float2int_rn(f);
        }
        uint32_t hi;
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(code[3]), "r"(code[2]), "r"(0));
        asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w[i / 4]) : "r"(code[1]), "r"(code[0]), "r"(hi));
      }
      int8_t* o = static_cast<int8_t*>(a.y) + row * a.ldy + c;
      if (VECTORS && n >= VE) {
        if constexpr (VE == 8)
          *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[VE / 4 - 1]);
        else
          *reinterpret_cast<uint32_t*>(o) = w[0];
      } else {
#pragma unroll
        for (int i = 0; i < VE; ++i)
          if (i < n) o[i] = static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)));
      }
    } else {
      store_vec<VECTORS>(static_cast<T*>(a.y) + row * a.ldy + c, v[k], n);
    }
  }
}

// LANES: a row belongs to 2^lg lanes of a warp, otherwise to the block;
// thread t of the row holds vectors t, t + threads, ... (NV of them).  Bound by
// memory (bf16 [8192, 4096] 26 us, 5.2 TB/s; with a residual 52 us, 5.2 TB/s; fp32 47 us,
// 5.8 TB/s; padded rows of 4097 40 us), and in short rows by the latency of a
// block's own loads (fp16 [12608, 768] 9.0 us, 35 % of the issue slots; int8 codes
// of [6304, 1024] 6.4 us).
template <class T, int NV, int SURE, bool LANES>
__global__ void __launch_bounds__(max_threads<T, NV>(), LANES || sizeof(T) == 4 ? 1 : 2) ln_fwd_kernel(const FwdArgs a) {
  constexpr int VE = Vec<T>::VE, VP = Vec<T>::VP;
  constexpr bool VECTORS = SURE >= 0;
  __shared__ __align__(16) float red[LANES ? 4 : 64];
  const int threads = LANES ? 1 << a.lg : blockDim.x;
  const int t = LANES ? threadIdx.x & (threads - 1) : threadIdx.x;
  int row = blockIdx.x;
  bool live = true;
  if constexpr (LANES) {
    const int64_t r = int64_t(blockIdx.x) * (blockDim.x >> a.lg) + (threadIdx.x >> a.lg);
    live = r < a.M;
    row = live ? int(r) : a.M - 1;  // lanes past the last row follow it and write nothing
  } else {
    for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i] = 0.f;
  }
  griddep_launch_dependents();
  griddep_wait();
  f2 v[NV][VP];
  {
    const T* x = static_cast<const T*>(a.x) + int64_t(row) * a.ldx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = k < SURE ? VE : a.C - c;
      Vec<T> e;
      if (n > 0) e = load_vec<VECTORS, true>(x + c, n);
      e.get(v[k]);
    }
  }
  if constexpr (!LANES) __syncthreads();
  if (a.res) {
    const T* res = static_cast<const T*>(a.res) + int64_t(row) * a.ldres;
    T* h = static_cast<T*>(a.h) + int64_t(row) * a.ldh;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = k < SURE ? VE : a.C - c;
      if (n <= 0) continue;
      f2 r[VP];
      load_vec<VECTORS, true>(res + c, n).get(r);
      // the backward pass reads h as it is stored, so the norm is taken of the rounded sum
      Vec<T> e;
#pragma unroll
      for (int i = 0; i < VP; ++i) v[k][i] = f2_add(v[k][i], r[i]);
      e.set(v[k]);
      e.get(v[k]);
      if (live) store_vec<VECTORS>(h + c, v[k], n);
    }
  }
  f2 s = 0ull;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < VP; ++i) s = f2_add(s, v[k][i]);
  const float inv = 1.f / static_cast<float>(a.C);
  float one = f2_get(s).x + f2_get(s).y;
  const float mu = (LANES ? lanes_sum(one, a.lg) : block_sum(one, red)) * inv;
  const f2 nmu = f2_of(-mu, -mu);
  s = 0ull;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int n = k < SURE ? VE : a.C - (t + k * threads) * VE;
    if (n <= 0) continue;
#pragma unroll
    for (int i = 0; i < VP; ++i) v[k][i] = f2_add(v[k][i], nmu);
    clear_past(v[k], n);
#pragma unroll
    for (int i = 0; i < VP; ++i) s = f2_fma(v[k][i], v[k][i], s);
  }
  one = f2_get(s).x + f2_get(s).y;
  const float rstd = rsqrtf((LANES ? lanes_sum(one, a.lg) : block_sum(one, red + 32)) * inv + a.eps);
  if (!live) return;
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = rstd;
  }
  const f2 r2 = f2_of(rstd, rstd);
  // one copy of the last step for each kind of weights and output, so that its
  // loop has no branch (they cost a third of the kernel's instructions)
  if (a.s8) {
    if (a.wf32) a.beta ? ln_finish<T, NV, SURE, true, true, true>(a, v, row, t, threads, r2)
                       : ln_finish<T, NV, SURE, true, false, true>(a, v, row, t, threads, r2);
    else a.beta ? ln_finish<T, NV, SURE, false, true, true>(a, v, row, t, threads, r2)
                : ln_finish<T, NV, SURE, false, false, true>(a, v, row, t, threads, r2);
  } else {
    if (a.wf32) a.beta ? ln_finish<T, NV, SURE, true, true, false>(a, v, row, t, threads, r2)
                       : ln_finish<T, NV, SURE, true, false, false>(a, v, row, t, threads, r2);
    else a.beta ? ln_finish<T, NV, SURE, false, true, false>(a, v, row, t, threads, r2)
                : ln_finish<T, NV, SURE, false, false, false>(a, v, row, t, threads, r2);
  }
}

struct BwdArgs {
  const void* dy;
  const void* x;
  const void* dh;
  void* dx;
  const void* gamma;
  const float* mean;
  const float* rstd;
  float* part;  // [gridDim.x][2][C]
  int64_t lddy, ldx, lddh, lddx;
  int M, C, lg, wf32, stages;
  uint32_t* err;
};

// A row's elements of one thread on their way through the backward pass.
//   g = dy gamma and z = (x - mu) rstd; the sums of g and g z over the row,
//   dy z and dy added to the columns' sums; then
//   dx = rstd (g - mean(g) - z mean(g z)) (+ dh)
template <class T, int NV>
struct BwdRow {
  static constexpr int VP = Vec<T>::VP;
  f2 g[NV][VP], z[NV][VP];
  f2 s1, s2;
  __device__ __forceinline__ void clear() { s1 = s2 = 0ull; }
  __device__ __forceinline__ void take(int k, const Vec<T>& x, const Vec<T>& dy, const f2 (&ga)[VP], float mu,
                                       float rstd, f2 (&dg)[VP], f2 (&db)[VP], int n) {
    const f2 r2 = f2_of(rstd, rstd), nm = f2_of(-mu, -mu);
    f2 d[VP];
    x.get(z[k]);
    dy.get(d);
#pragma unroll
    for (int i = 0; i < VP; ++i) z[k][i] = f2_mul(f2_add(z[k][i], nm), r2);
    clear_past(z[k], n);
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      g[k][i] = f2_mul(d[i], ga[i]);
      s1 = f2_add(s1, g[k][i]);
      s2 = f2_fma(g[k][i], z[k][i], s2);
      dg[i] = f2_fma(d[i], z[k][i], dg[i]);
      db[i] = f2_add(db[i], d[i]);
    }
  }
  // vector 0 of a row that is not held: g and z once more
  __device__ __forceinline__ void again(const Vec<T>& x, const Vec<T>& dy, const f2 (&ga)[VP], float mu, float rstd) {
    const f2 r2 = f2_of(rstd, rstd), nm = f2_of(-mu, -mu);
    x.get(z[0]);
    dy.get(g[0]);
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      z[0][i] = f2_mul(f2_add(z[0][i], nm), r2);
      g[0][i] = f2_mul(g[0][i], ga[i]);
    }
  }
  // the row's means m1, m2 (of g and g z) -> dx of vector k
  __device__ __forceinline__ void give(int k, float m1, float m2, float rstd, const f2 (&dh)[VP],
                                       f2 (&dx)[VP]) const {
    const f2 r2 = f2_of(rstd, rstd), a = f2_of(-m1, -m1), b = f2_of(-m2, -m2);
#pragma unroll
    for (int i = 0; i < VP; ++i) dx[i] = f2_fma(f2_fma(z[k][i], b, f2_add(g[k][i], a)), r2, dh[i]);
  }
};

// The block's partial sums of the columns.
template <class T, int NV>
__device__ __forceinline__ void store_part(float* p, int C, int t, int threads, const f2 (&dg)[NV][Vec<T>::VP],
                                           const f2 (&db)[NV][Vec<T>::VP]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * Vec<T>::VE;
#pragma unroll
    for (int i = 0; i < Vec<T>::VP; ++i) {
      const float2 g = f2_get(dg[k][i]), b = f2_get(db[k][i]);
      if (c + 2 * i < C) {
        p[c + 2 * i] = g.x;
        p[C + c + 2 * i] = b.x;
      }
      if (c + 2 * i + 1 < C) {
        p[c + 2 * i + 1] = g.y;
        p[C + c + 2 * i + 1] = b.y;
      }
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... (LANES: groups of rows, one to
// 2^lg lanes); the columns' sums stay in registers over all of them and go to
// the block's own rows of `part` at the end, so the order of every sum is
// fixed.  The next row's loads are issued before this row's sums.  Serves rows
// of up to 32 vectors (bf16 [60000, 64] 11 us), fp32 rows of more than 8192
// columns, and rows that are not 16-byte aligned; those cost a load an element
// (bf16 [8192, 4097] 260 us).
template <class T, int NV, bool VECTORS, bool LANES>
__global__ void __launch_bounds__(max_threads<T, NV>()) ln_bwd_kernel(const BwdArgs a) {
  constexpr int VE = Vec<T>::VE, VP = Vec<T>::VP;
  __shared__ __align__(16) float red[LANES ? 4 : 128];
  const int threads = LANES ? 1 << a.lg : blockDim.x;
  const int group = LANES ? threadIdx.x >> a.lg : 0, groups = LANES ? blockDim.x >> a.lg : 1;
  const int t = LANES ? threadIdx.x & (threads - 1) : threadIdx.x;
  if constexpr (!LANES) {
    for (int i = threadIdx.x; i < 128; i += blockDim.x) red[i] = 0.f;
    __syncthreads();
  }
  griddep_launch_dependents();
  griddep_wait();
  f2 ga[NV][VP], dg[NV][VP], db[NV][VP];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
#pragma unroll
    for (int i = 0; i < VP; ++i) ga[k][i] = dg[k][i] = db[k][i] = 0ull;
    if (c < a.C) load_weight<VECTORS, T>(ga[k], a.gamma, a.wf32, c, a.C - c);
  }
  const float inv = 1.f / static_cast<float>(a.C);
  const int64_t step = int64_t(gridDim.x) * groups;
  Vec<T> x[NV], dy[NV];
  float mun = 0.f, rstdn = 0.f;
  auto fetch = [&](int64_t row) {
    if (row >= a.M) return;
    mun = a.mean[row];
    rstdn = a.rstd[row];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      if (c >= a.C) continue;
      x[k] = load_vec<VECTORS, true>(static_cast<const T*>(a.x) + row * a.ldx + c, a.C - c);
      dy[k] = load_vec<VECTORS, true>(static_cast<const T*>(a.dy) + row * a.lddy + c, a.C - c);
    }
  };
  const int64_t first = int64_t(blockIdx.x) * groups;
  fetch(first + group);
  int turn = 0;
  for (int64_t base = first; base < a.M; base += step) {
    const int64_t row = base + group;
    const bool live = row < a.M;
    const float mu = mun, rstd = rstdn;
    BwdRow<T, NV> r;
    r.clear();
    if (live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int n = a.C - (t + k * threads) * VE;
        if (n > 0) r.take(k, x[k], dy[k], ga[k], mu, rstd, dg[k], db[k], n);
      }
    }
    fetch(row + step);
    float s1 = f2_get(r.s1).x + f2_get(r.s1).y, s2 = f2_get(r.s2).x + f2_get(r.s2).y;
    if constexpr (LANES) {
      s1 = lanes_sum(s1, a.lg);
      s2 = lanes_sum(s2, a.lg);
    } else {
      s1 = block_sum(s1, red + 64 * turn);
      s2 = block_sum(s2, red + 64 * turn + 32);
      turn ^= 1;
    }
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = a.C - c;
      if (n <= 0) continue;
      f2 h[VP];
#pragma unroll
      for (int i = 0; i < VP; ++i) h[i] = 0ull;
      if (a.dh) load_vec<VECTORS, true>(static_cast<const T*>(a.dh) + row * a.lddh + c, n).get(h);
      r.give(k, s1 * inv, s2 * inv, rstd, h, h);
      store_vec<VECTORS>(static_cast<T*>(a.dx) + row * a.lddx + c, h, n);
    }
  }
  if constexpr (LANES) {
    // groups of lanes that share their columns: summed in the order of the groups
    extern __shared__ float cols[];  // [groups][2][threads * VE]
    const int W = threads * VE;
    store_part<T, NV>(cols + size_t(group) * 2 * W, W, t, threads, dg, db);
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * W; j += blockDim.x) {
      float s = 0.f;
      for (int w = 0; w < groups; ++w) s += cols[size_t(w) * 2 * W + j];
      const int which = j >= W, c = j - which * W;
      if (c < a.C) a.part[(int64_t(blockIdx.x) * 2 + which) * a.C + c] = s;
    }
  } else {
    store_part<T, NV>(a.part + int64_t(blockIdx.x) * 2 * a.C, a.C, t, threads, dg, db);
  }
}

// The same for whole vectors, a block a row: x, dy and dh of the next rows come
// by bulk copies into a ring of `stages` rows (an SM has to have some 50 KB of
// reads under way to draw the memory's full rate, more than a block holds in
// registers).  Up to two vectors a thread a row stays in registers, so its
// stage is free at the barrier of its own sums; with four, which would not
// fit, it is read from the ring twice, and gamma with it, and the stage is free
// at the next row's barrier.  bf16 [8192, 4096] 50 us (4.0 TB/s; by loads into registers
// 68 us), with dh 57 us (4.7 TB/s); [2048, 16384] 84 us: there the barrier of a
// row of 512 threads is what bounds it.
template <class T, int NV, int SURE, bool DH>
__global__ void __launch_bounds__(512) ln_bwd_ring_kernel(const BwdArgs a) {
  constexpr int VE = Vec<T>::VE, VP = Vec<T>::VP;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float red[2][2][16];  // two turns of the sums of g and of g z, one float a warp
  __shared__ uint64_t full[16];
  const int threads = blockDim.x, t = threadIdx.x;
  for (int i = t; i < 64; i += threads) red[0][0][i] = 0.f;
  // whole vectors come through the ring; a row's last elements are read directly
  const uint32_t row_bytes = uint32_t(a.C) * sizeof(T) / 16 * 16;
  const uint32_t stage_bytes = row_bytes * (DH ? 3 : 2);
  if (t == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  auto fetch = [&](int64_t row, int s) {  // one thread
    uint8_t* to = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], stage_bytes);
    bulk_load(smem_addr(to), static_cast<const T*>(a.x) + row * a.ldx, row_bytes, &full[s]);
    bulk_load(smem_addr(to + row_bytes), static_cast<const T*>(a.dy) + row * a.lddy, row_bytes, &full[s]);
    if (DH) bulk_load(smem_addr(to + 2 * row_bytes), static_cast<const T*>(a.dh) + row * a.lddh, row_bytes, &full[s]);
  };
  const int64_t step = gridDim.x;
  if (t == 0)
    for (int s = 0; s < a.stages; ++s)
      if (blockIdx.x + s * step < a.M) fetch(blockIdx.x + s * step, s);
  constexpr bool kHold = NV <= 2;
  constexpr int NH = kHold ? NV : 1;
  f2 ga[NH][VP], dg[NV][VP], db[NV][VP];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      dg[k][i] = db[k][i] = 0ull;
      if constexpr (kHold) ga[k][i] = 0ull;
    }
    if constexpr (kHold) {
      if (k < SURE || c < a.C) load_weight<true, T>(ga[k], a.gamma, a.wf32, c, k < SURE ? VE : a.C - c);
    }
  }
  const float inv = 1.f / static_cast<float>(a.C);
  int s = 0, turn = 0;
  uint32_t phase = 0;
  float mu = 0.f, rstd = 0.f;
  if (blockIdx.x < a.M) {
    mu = a.mean[blockIdx.x];
    rstd = a.rstd[blockIdx.x];
  }
  int never = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += step) {
    mbar_wait(&full[s], phase, &never, a.err, ERR_WAIT_FULL);
    const uint8_t* from = ring + s * stage_bytes;
    BwdRow<T, NH> r;
    r.clear();
    Vec<T> dh[NH];
    // vector c of x, dy or dh (the i-th part of the stage)
    auto read = [&](int i, const void* p, int64_t ld, int c, int n) {
      Vec<T> v;
      if (n >= VE)
        v.raw = *reinterpret_cast<const uint4*>(from + i * row_bytes + c * sizeof(T));
      else
        v.raw = load_last(static_cast<const T*>(p) + row * ld + c, n);
      return v;
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = k < SURE ? VE : a.C - c;
      if (n <= 0) continue;
      const int kh = kHold ? k : 0;
      const Vec<T> x = read(0, a.x, a.ldx, c, n), dy = read(1, a.dy, a.lddy, c, n);
      if constexpr (kHold) {
        if (DH) dh[k] = read(2, a.dh, a.lddh, c, n);
      } else {
        load_weight<true, T>(ga[0], a.gamma, a.wf32, c, n);
      }
      r.take(kh, x, dy, ga[kh], mu, rstd, dg[k], db[k], n);
    }
    const float mc = mu, rs = rstd;
    if (row + step < a.M) {
      mu = a.mean[row + step];
      rstd = a.rstd[row + step];
    }
    const float w1 = warp_sum(f2_get(r.s1).x + f2_get(r.s1).y), w2 = warp_sum(f2_get(r.s2).x + f2_get(r.s2).y);
    if ((t & 31) == 0) {
      red[turn][0][t >> 5] = w1;
      red[turn][1][t >> 5] = w2;
    }
    __syncthreads();
    if (t == 0) {  // the stage that every thread is done with: this row's, or the one before it
      const int64_t next = row + (kHold ? a.stages : a.stages - 1) * step;
      if (next < a.M && (kHold || row != blockIdx.x)) fetch(next, kHold ? s : s ? s - 1 : a.stages - 1);
    }
    const float m1 = sum_of(red[turn][0], threads >> 5) * inv, m2 = sum_of(red[turn][1], threads >> 5) * inv;
    turn ^= 1;
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = k < SURE ? VE : a.C - c;
      if (n <= 0) continue;
      f2 h[VP];
#pragma unroll
      for (int i = 0; i < VP; ++i) h[i] = 0ull;
      if constexpr (kHold) {
        if (DH) dh[k].get(h);
        r.give(k, m1, m2, rs, h, h);
      } else {
        const Vec<T> x = read(0, a.x, a.ldx, c, n), dy = read(1, a.dy, a.lddy, c, n);
        if (DH) {
          dh[0] = read(2, a.dh, a.lddh, c, n);
          dh[0].get(h);
        }
        load_weight<true, T>(ga[0], a.gamma, a.wf32, c, n);
        r.again(x, dy, ga[0], mc, rs);
        r.give(0, m1, m2, rs, h, h);
      }
      store_vec<true>(dx + c, h, n);
    }
    if (++s == a.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  store_part<T, NV>(a.part + int64_t(blockIdx.x) * 2 * a.C, a.C, t, threads, dg, db);
}

// The same with a warp a row (up to 128 vectors), so no barrier a row: each
// warp has its own ring, and the warps' column sums are added in their order
// at the end.  fp16 [12608, 768] 19 us; a row took the block kernel 1.5 us a block.
constexpr int bwd_warps(int es, int nv) { return es == 4 || nv == 2 ? 16 : 8; }  // what the registers allow
template <class T, int NV, int SURE, bool DH>
__global__ void __launch_bounds__(32 * bwd_warps(sizeof(T), NV)) ln_bwd_warp_kernel(const BwdArgs a) {
  constexpr int VE = Vec<T>::VE, VP = Vec<T>::VP, kBwdWarps = bwd_warps(sizeof(T), NV);
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t bars[kBwdWarps][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // whole vectors come through the ring; a row's last elements are read directly
  const uint32_t row_bytes = uint32_t(a.C) * sizeof(T) / 16 * 16;
  const uint32_t stage_bytes = row_bytes * (DH ? 3 : 2);
  uint8_t* ring = smem + size_t(warp) * a.stages * stage_bytes;
  uint64_t* full = bars[warp];
  if (lane == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  __syncwarp();
  griddep_launch_dependents();
  griddep_wait();
  auto fetch = [&](int64_t row, int s) {  // one lane
    uint8_t* to = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], stage_bytes);
    bulk_load(smem_addr(to), static_cast<const T*>(a.x) + row * a.ldx, row_bytes, &full[s]);
    bulk_load(smem_addr(to + row_bytes), static_cast<const T*>(a.dy) + row * a.lddy, row_bytes, &full[s]);
    if (DH) bulk_load(smem_addr(to + 2 * row_bytes), static_cast<const T*>(a.dh) + row * a.lddh, row_bytes, &full[s]);
  };
  const int64_t step = int64_t(gridDim.x) * kBwdWarps;
  const int64_t first = int64_t(blockIdx.x) * kBwdWarps + warp;
  if (lane == 0)
    for (int s = 0; s < a.stages; ++s)
      if (first + s * step < a.M) fetch(first + s * step, s);
  f2 ga[NV][VP], dg[NV][VP], db[NV][VP];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (lane + 32 * k) * VE;
#pragma unroll
    for (int i = 0; i < VP; ++i) ga[k][i] = dg[k][i] = db[k][i] = 0ull;
    if (k < SURE || c < a.C) load_weight<true, T>(ga[k], a.gamma, a.wf32, c, k < SURE ? VE : a.C - c);
  }
  const float inv = 1.f / static_cast<float>(a.C);
  int s = 0;
  uint32_t phase = 0;
  float mu = 0.f, rstd = 0.f;
  if (first < a.M) {
    mu = a.mean[first];
    rstd = a.rstd[first];
  }
  int never = 0;
  for (int64_t row = first; row < a.M; row += step) {
    mbar_wait(&full[s], phase, &never, a.err, ERR_WAIT_FULL);
    const uint8_t* from = ring + s * stage_bytes;
    // vector c of x, dy or dh (the i-th part of the stage)
    auto read = [&](int i, const void* p, int64_t ld, int c, int n) {
      Vec<T> v;
      if (n >= VE)
        v.raw = *reinterpret_cast<const uint4*>(from + i * row_bytes + c * sizeof(T));
      else
        v.raw = load_last(static_cast<const T*>(p) + row * ld + c, n);
      return v;
    };
    BwdRow<T, NV> r;
    r.clear();
    Vec<T> dh[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + 32 * k) * VE;
      const int n = k < SURE ? VE : a.C - c;
      if (n <= 0) continue;
      const Vec<T> x = read(0, a.x, a.ldx, c, n), dy = read(1, a.dy, a.lddy, c, n);
      if (DH) dh[k] = read(2, a.dh, a.lddh, c, n);
      r.take(k, x, dy, ga[k], mu, rstd, dg[k], db[k], n);
    }
    const float rs = rstd;
    if (row + step < a.M) {
      mu = a.mean[row + step];
      rstd = a.rstd[row + step];
    }
    const float m1 = warp_sum(f2_get(r.s1).x + f2_get(r.s1).y) * inv;
    const float m2 = warp_sum(f2_get(r.s2).x + f2_get(r.s2).y) * inv;
    __syncwarp();  // every lane has read its part of the stage, dh too, before it is filled again
    if (lane == 0 && row + a.stages * step < a.M) fetch(row + a.stages * step, s);
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (lane + 32 * k) * VE;
      const int n = k < SURE ? VE : a.C - c;
      if (n <= 0) continue;
      f2 h[VP];
#pragma unroll
      for (int i = 0; i < VP; ++i) h[i] = 0ull;
      if (DH) dh[k].get(h);
      r.give(k, m1, m2, rs, h, h);
      store_vec<true>(dx + c, h, n);
    }
    if (++s == a.stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  __syncthreads();  // every warp is done with its ring
  float* cols = reinterpret_cast<float*>(smem);  // [warps][2][C]
  store_part<T, NV>(cols + size_t(warp) * 2 * a.C, a.C, lane, 32, dg, db);
  __syncthreads();
  for (int j = threadIdx.x; j < 2 * a.C; j += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kBwdWarps; ++w) v += cols[size_t(w) * 2 * a.C + j];
    a.part[int64_t(blockIdx.x) * 2 * a.C + j] = v;
  }
}

// dgamma and dbeta from the blocks' partial sums: 32 columns a block, the
// partial rows dealt to its warps, each sum in a fixed order.
__global__ void __launch_bounds__(1024) ln_colsum_kernel(const float* part, int rows, int C, void* dgamma, void* dbeta,
                                                         int kind) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // column of the 2 C of a partial row
  griddep_launch_dependents();
  griddep_wait();
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < 2 * C)
    for (int r0 = warp; r0 < rows; r0 += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (r0 + 32 * k < rows) s[k] += part[int64_t(r0 + 32 * k) * 2 * C + c];
    }
  sm[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (warp == 0 && c < 2 * C) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += sm[w][lane];
    void* out = c < C ? dgamma : dbeta;
    const int i = c < C ? c : c - C;
    if (out) {
      if (kind == SPG_F32) static_cast<float*>(out)[i] = v;
      else if (kind == SPG_F16) static_cast<__half*>(out)[i] = from_f<__half>(v);
      else static_cast<__nv_bfloat16*>(out)[i] = from_f<__nv_bfloat16>(v);
    }
  }
}

constexpr int kMaxC = 16384;

int esize(int dtype) { return dtype == SPG_F32 ? 4 : 2; }

// How a row is dealt to threads.
struct Shape {
  bool lanes;   // to 2^lg lanes of a warp, otherwise to the block
  int lg;
  int nv;       // vectors a thread
  int threads;  // of the block
};

constexpr int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

constexpr int lg_of(int nvec) {
  int lg = 0;
  while ((1 << lg) < nvec && lg < 5) ++lg;
  return lg;
}

// Up to four vectors a lane a row stays in one warp (no barrier); beyond that
// a block with four vectors a thread, so that a row's two block sums weigh little.
constexpr Shape fwd_shape(int C, int es) {
  const int nvec = (C * es + 15) / 16;
  if (nvec <= 128) return {true, lg_of(nvec), (nvec + 31) / 32, 128};
  return {false, 0, 4, round32((nvec + 3) / 4)};
}

// One vector a lane where that holds the row (several rows a warp where it is
// shorter); a warp with up to four a lane; otherwise two or four vectors a thread of a block.
constexpr Shape bwd_shape(int C, int es) {
  const int nvec = (C * es + 15) / 16;
  if (nvec <= 32) return {true, lg_of(nvec), 1, 256};
  if (nvec <= 128) {
    const int nv = (nvec + 31) / 32;
    return {true, 5, nv, 32 * bwd_warps(es, nv)};
  }
  const int nv = nvec <= 1024 ? 2 : 4;
  return {false, 0, nv, round32((nvec + nv - 1) / nv)};
}

// Blocks of the backward kernel: as many as are resident, so that each leaves
// one row of partial sums and no more, and a row group each at least.
constexpr int bwd_per_sm(const Shape& s) {
  return s.lanes ? (s.nv == 1 ? 3 : 1) : s.threads > 256 ? 1 : s.threads > 128 ? 2 : 4;
}
int bwd_blocks(int64_t M, const Shape& s) {
  const int64_t groups = s.lanes ? s.threads >> s.lg : 1;
  const int64_t work = (M + groups - 1) / groups;
  const int64_t cap = int64_t(sm_count()) * bwd_per_sm(s);
  return static_cast<int>(work < cap ? work : cap);
}

// The vectors of each thread that are whole and inside the row: all `nv`, all
// but the last, or (0) none to be sure of.
constexpr int sure_vectors(const Shape& s, int C, int es) {
  const int threads = s.lanes ? 1 << s.lg : s.threads, whole = C * es / 16;
  return whole >= threads * s.nv && C * es % 16 == 0 ? s.nv : whole >= threads * (s.nv - 1) ? s.nv - 1 : 0;
}

// Rows of `row_bytes` in a ring fit a block's share of shared memory at least twice.
constexpr bool ring_fits(const Shape& s, int64_t row_bytes) {
  return s.threads <= 512 && (224 * 1024 / bwd_per_sm(s) - 1024) / row_bytes >= 2;
}

// What the choices below rest on, for every row length: a row in a warp's lanes,
// and a row of the backward pass, leaves no vector but the last of a thread in
// question, and 16-bit rows always fit the ring (with dh, three matrices).
constexpr bool dealt_as_chosen(int es, int first, int last) {
  for (int C = first; C <= last; ++C) {
    const Shape f = fwd_shape(C, es), b = bwd_shape(C, es);
    if (f.lanes && sure_vectors(f, C, es) < f.nv - 1) return false;
    if (sure_vectors(b, C, es) < b.nv - 1) return false;
    if (es == 2 && !b.lanes && !ring_fits(b, int64_t(C) * es / 16 * 16 * 3)) return false;
  }
  return true;
}
static_assert(dealt_as_chosen(2, 1, 8192) && dealt_as_chosen(2, 8193, kMaxC), "16-bit rows");
static_assert(dealt_as_chosen(4, 1, 8192) && dealt_as_chosen(4, 8193, kMaxC), "fp32 rows");

using FwdKernel = void (*)(const FwdArgs);
template <class T, int NV, bool LANES>
FwdKernel fwd_kernel(int sure) {
  if (sure == NV) return ln_fwd_kernel<T, NV, NV, LANES>;
  if (sure < 0) return ln_fwd_kernel<T, NV, ELEMENTS, LANES>;
  if constexpr (!LANES)
    if (sure < NV - 1) return ln_fwd_kernel<T, NV, 0, LANES>;
  return ln_fwd_kernel<T, NV, NV - 1, LANES>;
}

template <class T>
cudaError_t launch_fwd(const FwdArgs& a, const Shape& s, bool vectors, int64_t blocks, cudaStream_t st) {
  const int sure = vectors ? sure_vectors(s, a.C, sizeof(T)) : ELEMENTS;
  const FwdKernel k = !s.lanes    ? fwd_kernel<T, 4, false>(sure)
                      : s.nv == 1 ? fwd_kernel<T, 1, true>(sure)
                      : s.nv == 2 ? fwd_kernel<T, 2, true>(sure)
                      : s.nv == 3 ? fwd_kernel<T, 3, true>(sure)
                                  : fwd_kernel<T, 4, true>(sure);
  // Large batches are not launched ahead of the previous kernel's end: an SM that
  // never idles keeps that kernel's share of shared memory (the pruned layers'
  // is nearly all of it), and the loads under way are limited by what it leaves
  // to L1.  A square fp16 layer and the norm behind it, in plain order against ahead:
  // [8192, 4096] 151 / 154 us, [4096, 4096] with a residual 97 / 100; at the limit no
  // difference ([9456, 1024] with a residual 33.0 / 32.9, [6304, 1024] 26.2 / 26.2); below it
  // [6304, 1024] without a residual 20.8 / 20.6, [12608, 768] 24.2 / 23.9.
  const int64_t read = int64_t(a.M) * a.C * sizeof(T) * (a.res ? 2 : 1);
  if (read > (int64_t(32) << 20)) {
    k<<<static_cast<unsigned>(blocks), s.threads, 0, st>>>(a);
    return cudaGetLastError();
  }
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(s.threads), 0, st, a);
}

using BwdKernel = void (*)(const BwdArgs);
template <class T, int NV>
BwdKernel ring_kernel(int sure, bool dh) {
  return sure == NV ? (dh ? ln_bwd_ring_kernel<T, NV, NV, true> : ln_bwd_ring_kernel<T, NV, NV, false>)
                    : (dh ? ln_bwd_ring_kernel<T, NV, NV - 1, true> : ln_bwd_ring_kernel<T, NV, NV - 1, false>);
}
template <class T, int NV>
BwdKernel warp_kernel(int sure, bool dh) {
  return sure == NV ? (dh ? ln_bwd_warp_kernel<T, NV, NV, true> : ln_bwd_warp_kernel<T, NV, NV, false>)
                    : (dh ? ln_bwd_warp_kernel<T, NV, NV - 1, true> : ln_bwd_warp_kernel<T, NV, NV - 1, false>);
}

template <class T>
cudaError_t launch_bwd(const BwdArgs& a, const Shape& s, bool vectors, int blocks, cudaStream_t st) {
  const int sure = sure_vectors(s, a.C, sizeof(T));
  const bool dh = a.dh != nullptr;
  const int64_t row = int64_t(a.C) * sizeof(T) / 16 * 16 * (dh ? 3 : 2);  // bytes of a row in a ring
  BwdKernel k;
  size_t smem = 0;
  BwdArgs b = a;
  if (s.lanes && s.nv == 1) {
    k = vectors ? ln_bwd_kernel<T, 1, true, true> : ln_bwd_kernel<T, 1, false, true>;
    smem = size_t(s.threads) * 2 * Vec<T>::VE * sizeof(float);
  } else if (s.lanes && !vectors) {  // the block kernel, with the warp kernel's blocks
    Shape q = s;
    q.lanes = false;
    q.nv = 1;
    q.threads = round32((a.C * int(sizeof(T)) + 15) / 16);
    return launch_bwd<T>(a, q, false, blocks, st);
  } else if (s.lanes) {
    // one block an SM; two stages of the longest rows (2 KB) take 16 * 2 * 6 KB
    const int64_t stage = row * (s.threads / 32);
    const int64_t stages = 200 * 1024 / stage;
    b.stages = stages > 8 ? 8 : static_cast<int>(stages);
    const int64_t sums = int64_t(s.threads / 32) * 2 * a.C * 4;
    smem = size_t(b.stages * stage > sums ? b.stages * stage : sums);
    k = s.nv == 2 ? warp_kernel<T, 2>(sure, dh) : s.nv == 3 ? warp_kernel<T, 3>(sure, dh) : warp_kernel<T, 4>(sure, dh);
  } else {
    // the ring, where at least two rows of it fit the block's share of shared memory
    if (vectors && ring_fits(s, row)) {
      const int64_t stages = (224 * 1024 / bwd_per_sm(s) - 1024) / row;
      b.stages = stages > 16 ? 16 : static_cast<int>(stages);
      smem = size_t(b.stages * row);
      k = s.nv == 2 ? ring_kernel<T, 2>(sure, dh) : ring_kernel<T, 4>(sure, dh);
    } else if (sizeof(T) == 4 && vectors) {  // rows of more than 8192 columns
      k = ln_bwd_kernel<float, 4, true, false>;
    } else {
      k = s.nv == 1   ? ln_bwd_kernel<T, 1, false, false>
          : s.nv == 2 ? ln_bwd_kernel<T, 2, false, false>
                      : ln_bwd_kernel<T, 4, false, false>;
    }
  }
  if (smem > 40 * 1024) {  // 48 KB with the static arrays
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k, dim3(blocks), dim3(s.threads), smem, st, b);
}

bool vec_ok(const void* p, int64_t ld, int es) { return p == nullptr || (aligned(p, 16) && (ld * es) % 16 == 0); }

bool is_act(int d) { return d == SPG_F16 || d == SPG_BF16 || d == SPG_F32; }

// An output in place of an input keeps its rows where they are.
bool other_pitch(const void* in, int64_t ldin, const void* out, int64_t ldout) {
  return in && in == out && ldin != ldout;
}

// What the two forward entry points share.
spg_status fwd(const void* X, int64_t ldx, const void* res, int64_t ldres, void* H, int64_t ldh, const void* gamma,
               const void* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd, int64_t M, int64_t C,
               int dtype, int wdtype, int s8, float qscale, cudaStream_t st) {
  if (!is_act(dtype) || (wdtype != dtype && wdtype != SPG_F32)) return SPG_ERR_INVALID_ARG;
  if (M < 0 || C <= 0 || ldx < C || ldy < C || (res && ldres < C) || (res && ldh < C)) return SPG_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !(eps < 3.0e38f) || !gamma) return SPG_ERR_INVALID_ARG;
  if ((res == nullptr) != (H == nullptr) && M != 0) return SPG_ERR_INVALID_ARG;
  if (M != 0 && (!X || !Y)) return SPG_ERR_INVALID_ARG;
  if (C > kMaxC || M >= (int64_t(1) << 31)) return SPG_ERR_UNSUPPORTED_SHAPE;
  const int es = esize(dtype), wes = esize(wdtype);
  if (!aligned(X, es) || !aligned(res, es) || !aligned(H, es) || !aligned(Y, s8 ? 1 : es) || !aligned(gamma, wes) ||
      !aligned(beta, wes) || !aligned(mean, 4) || !aligned(rstd, 4))
    return SPG_ERR_MISALIGNED;
  if (M == 0) return SPG_OK;
  if (Y == H || other_pitch(X, ldx, H, ldh) || other_pitch(res, ldres, H, ldh) ||
      (s8 ? Y == X || Y == res : other_pitch(X, ldx, Y, ldy) || other_pitch(res, ldres, Y, ldy)))
    return SPG_ERR_INVALID_ARG;
  spg_status rc = check_device();
  if (rc != SPG_OK) return rc;
  const Shape s = fwd_shape(int(C), es);
  const FwdArgs b{X,   res, H,      Y,      gamma, beta,              mean, rstd, ldx,   ldres,
                  ldh, ldy, int(M), int(C), s.lg,  wdtype == SPG_F32, s8,   eps,  qscale};
  const int64_t rows = s.lanes ? s.threads >> s.lg : 1;
  const int64_t blocks = (M + rows - 1) / rows;
  // vectors in rows that start on 16-byte boundaries; otherwise element by element
  const bool al = vec_ok(X, ldx, es) && vec_ok(res, ldres, es) && vec_ok(H, ldh, es) &&
                  (s8 ? aligned(Y, 8) && ldy % 8 == 0 : vec_ok(Y, ldy, es)) && aligned(gamma, 16) && aligned(beta, 16);
  const cudaError_t e = dtype == SPG_F32   ? launch_fwd<float>(b, s, al, blocks, st)
                        : dtype == SPG_F16 ? launch_fwd<__half>(b, s, al, blocks, st)
                                           : launch_fwd<__nv_bfloat16>(b, s, al, blocks, st);
  return e == cudaSuccess ? launch_status() : SPG_ERR_CUDA;
}

}  // namespace norm
}  // namespace spg

extern "C" {

spg_status layernorm(const void* X, int64_t ldx, const void* res, int64_t ldres, void* H, int64_t ldh,
                     const void* gamma, const void* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
                     int64_t M, int64_t C, spg_dtype dtype, spg_dtype wdtype, spg_stream_t stream) {
  return spg::norm::fwd(X, ldx, res, ldres, H, ldh, gamma, beta, eps, Y, ldy, mean, rstd, M, C, dtype, wdtype, 0, 1.f,
                        reinterpret_cast<cudaStream_t>(stream));
}

spg_status layernorm_s8(const void* X, int64_t ldx, const void* res, int64_t ldres, void* H, int64_t ldh,
                        const void* gamma, const void* beta, float eps, float qscale, int8_t* Yq, int64_t ldy,
                        int64_t M, int64_t C, spg_dtype dtype, spg_dtype wdtype, spg_stream_t stream) {
  if (!(qscale > 0.f) || !(qscale < 3.0e38f)) return SPG_ERR_INVALID_ARG;
  return spg::norm::fwd(X, ldx, res, ldres, H, ldh, gamma, beta, eps, Yq, ldy, nullptr, nullptr, M, C, dtype, wdtype,
                        1, qscale, reinterpret_cast<cudaStream_t>(stream));
}

size_t layernorm_bwd_workspace_size(int64_t M, int64_t C, spg_dtype dtype) {
  using namespace spg::norm;
  if (M <= 0 || C <= 0 || C > kMaxC || M >= (int64_t(1) << 31) || !is_act(dtype)) return 0;
  return size_t(bwd_blocks(M, bwd_shape(int(C), esize(dtype)))) * 2 * size_t(C) * sizeof(float);
}

spg_status layernorm_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, const float* mean,
                         const float* rstd, const void* gamma, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                         void* dgamma, void* dbeta, void* workspace, size_t ws_bytes, int64_t M, int64_t C,
                         spg_dtype dtype, spg_dtype wdtype, spg_stream_t stream) {
  using namespace spg;
  using namespace spg::norm;
  if (!is_act(dtype) || (wdtype != dtype && wdtype != SPG_F32)) return SPG_ERR_INVALID_ARG;
  if (M < 0 || C <= 0 || lddy < C || ldx < C || lddx < C || (dH && lddh < C)) return SPG_ERR_INVALID_ARG;
  if (!gamma || !dgamma) return SPG_ERR_INVALID_ARG;
  if (M != 0 && (!dY || !X || !mean || !rstd || !dX || !workspace)) return SPG_ERR_INVALID_ARG;
  if (C > kMaxC || M >= (int64_t(1) << 31)) return SPG_ERR_UNSUPPORTED_SHAPE;
  const int es = esize(dtype), wes = esize(wdtype);
  if (!aligned(dY, es) || !aligned(X, es) || !aligned(dH, es) || !aligned(dX, es) || !aligned(gamma, wes) ||
      !aligned(dgamma, wes) || !aligned(dbeta, wes) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 16))
    return SPG_ERR_MISALIGNED;
  if (ws_bytes < layernorm_bwd_workspace_size(M, C, dtype)) return SPG_ERR_INVALID_ARG;
  if (M != 0 && (other_pitch(dY, lddy, dX, lddx) || other_pitch(X, ldx, dX, lddx) || other_pitch(dH, lddh, dX, lddx)))
    return SPG_ERR_INVALID_ARG;
  spg_status rc = check_device();
  if (rc != SPG_OK) return rc;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const Shape s = bwd_shape(int(C), es);
  int blocks = 0;
  if (M != 0) {
    blocks = bwd_blocks(M, s);
    uint32_t* err = device_error_word();
    if (!err) return SPG_ERR_CUDA;
    const BwdArgs a{dY,  X,    dH,   dX,     gamma,  mean, rstd, static_cast<float*>(workspace), lddy,
                    ldx, lddh, lddx, int(M), int(C), s.lg, wdtype == SPG_F32, 0, err};
    const bool al = vec_ok(dY, lddy, es) && vec_ok(X, ldx, es) && vec_ok(dH, lddh, es) && vec_ok(dX, lddx, es) &&
                    aligned(gamma, 16);
    const cudaError_t e = dtype == SPG_F32   ? launch_bwd<float>(a, s, al, blocks, st)
                          : dtype == SPG_F16 ? launch_bwd<__half>(a, s, al, blocks, st)
                                             : launch_bwd<__nv_bfloat16>(a, s, al, blocks, st);
    if (e != cudaSuccess) return SPG_ERR_CUDA;
  }
  // no rows: the sums over them are zero
  if (launch_pdl(ln_colsum_kernel, dim3(static_cast<unsigned>((2 * C + 31) / 32)), dim3(1024), 0, st,
                 static_cast<const float*>(workspace), blocks, int(C), dgamma, dbeta, int(wdtype)) != cudaSuccess)
    return SPG_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
