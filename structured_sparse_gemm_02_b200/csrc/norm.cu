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

#include "host.cuh"
#include "sm100.cuh"
#include "spgemm.h"

namespace spg {
namespace norm {

// One 16-byte vector of a row: VE elements of T as they lie in memory.
template <class T>
struct Vec {
  static constexpr int VE = 16 / sizeof(T);
  union {
    uint4 raw;
    T e[VE];
  };
  __device__ Vec() : raw(make_uint4(0u, 0u, 0u, 0u)) {}
  // elements [0, n) from p; a whole vector in one load where AL says that p is 16-byte aligned
  template <bool AL>
  __device__ __forceinline__ void load(const T* p, int n) {
    if (AL && n >= VE) {
      raw = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i < n) e[i] = p[i];
    }
  }
  template <bool AL>
  __device__ __forceinline__ void store(T* p, int n) const {
    if (AL && n >= VE) {
      *reinterpret_cast<uint4*>(p) = raw;
    } else {
#pragma unroll
      for (int i = 0; i < VE; ++i)
        if (i < n) p[i] = e[i];
    }
  }
};

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

// VE elements of gamma or beta, in the activations' type or in fp32; 0 where the pointer is null.
template <class T>
__device__ __forceinline__ void load_weight(float (&w)[Vec<T>::VE], const void* p, int f32, int c, int n) {
#pragma unroll
  for (int i = 0; i < Vec<T>::VE; ++i)
    w[i] = (p == nullptr || i >= n) ? 0.f
           : f32                    ? static_cast<const float*>(p)[c + i]
                                    : to_f(static_cast<const T*>(p)[c + i]);
}

// Threads of the largest block: 16384 columns are 2048 vectors of a 16-bit type
// or 4096 of fp32, at most four a thread.
template <class T, int NV>
constexpr int max_threads() { return sizeof(T) == 4 && NV == 4 ? 1024 : 512; }

// Sums over the threads of a row: `tpr` lanes of a warp (a power of two), or
// the whole block through shared memory.  The two halves of `red` alternate,
// so one barrier a reduction is enough.
struct RowSum {
  float2* red;  // 2 x 32
  int tpr;      // 0: the block
  int turn;
  __device__ float2 operator()(float2 v) {
    const int width = tpr ? tpr : 32;
    for (int o = width >> 1; o; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (tpr) return v;
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float2* r = red + 32 * turn;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    v = r[0];
    for (int w = 1; w < warps; ++w) {
      v.x += r[w].x;
      v.y += r[w].y;
    }
    return v;
  }
};

struct FwdArgs {
  const void* x;
  const void* res;
  void* h;
  void* y;
  const void* gamma;
  const void* beta;
  float* mean;
  float* rstd;
  int64_t ldx, ldres, ldh, ldy, M;
  int C, tpr, wf32, s8;
  float eps, qscale;
};

// A row belongs to `tpr` lanes of a warp (tpr > 0) or to the block (tpr = 0);
// thread t of the row holds vectors t, t + threads, ... (NV of them).
template <class T, int NV, bool AL>
__global__ void __launch_bounds__(max_threads<T, NV>()) ln_fwd_kernel(const FwdArgs a) {
  constexpr int VE = Vec<T>::VE;
  __shared__ float2 red[64];
  const int threads = a.tpr ? a.tpr : blockDim.x;
  const int t = threadIdx.x % threads;
  const int64_t row0 = a.tpr ? int64_t(blockIdx.x) * (blockDim.x / threads) + threadIdx.x / threads : blockIdx.x;
  const bool live = row0 < a.M;
  const int64_t row = live ? row0 : a.M - 1;  // lanes past the last row follow it and write nothing
  griddep_launch_dependents();
  griddep_wait();
  RowSum sum{red, a.tpr, 0};
  float v[NV][VE];
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
    const int n = a.C - c;
    Vec<T> x;
    if (n > 0) {
      x.template load<AL>(static_cast<const T*>(a.x) + row * a.ldx + c, n);
      if (a.res) {
        Vec<T> r;
        r.template load<AL>(static_cast<const T*>(a.res) + row * a.ldres + c, n);
        // the backward pass reads h as it is stored, so the norm is taken of the rounded sum
#pragma unroll
        for (int i = 0; i < VE; ++i) x.e[i] = from_f<T>(to_f(x.e[i]) + to_f(r.e[i]));
        if (live) x.template store<AL>(static_cast<T*>(a.h) + row * a.ldh + c, n);
      }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      v[k][i] = to_f(x.e[i]);
      s += v[k][i];
    }
  }
  const float inv = 1.f / static_cast<float>(a.C);
  const float mu = sum(make_float2(s, 0.f)).x * inv;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int n = a.C - (t + k * threads) * VE;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      v[k][i] -= mu;
      q += i < n ? v[k][i] * v[k][i] : 0.f;
    }
  }
  const float rstd = rsqrtf(sum(make_float2(q, 0.f)).x * inv + a.eps);
  if (!live) return;
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = rstd;
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
    const int n = a.C - c;
    if (n <= 0) continue;
    float g[VE], b[VE];
    load_weight<T>(g, a.gamma, a.wf32, c, n);
    load_weight<T>(b, a.beta, a.wf32, c, n);
    if (a.s8) {
      // clamp(rne(y qscale)); a NaN gives code 0
      uint32_t w[VE / 4];
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float y = fmaf(v[k][i] * rstd, g[i], b[i]) * a.qscale;
        const int code = max(-127, min(127, __float2int_rn(y)));
        w[i / 4] = (i % 4 ? w[i / 4] : 0u) | (static_cast<uint32_t>(code & 0xFF) << (8 * (i % 4)));
      }
      int8_t* o = static_cast<int8_t*>(a.y) + row * a.ldy + c;
      if (AL && n >= VE) {
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
      Vec<T> o;
#pragma unroll
      for (int i = 0; i < VE; ++i) o.e[i] = from_f<T>(fmaf(v[k][i] * rstd, g[i], b[i]));
      o.template store<AL>(static_cast<T*>(a.y) + row * a.ldy + c, n);
    }
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
  int64_t lddy, ldx, lddh, lddx, M;
  int C, tpr, wf32;
};

// Rows as in ln_fwd_kernel, a block taking rows blockIdx.x, blockIdx.x + gridDim.x, ...
// (in groups of blockDim.x / tpr); the columns' sums stay in registers over
// all its rows and go to the block's own rows of `part` at the end, so the
// order of every sum is fixed.
template <class T, int NV, bool AL>
__global__ void __launch_bounds__(max_threads<T, NV>()) ln_bwd_kernel(const BwdArgs a) {
  constexpr int VE = Vec<T>::VE;
  __shared__ float2 red[64];
  const int threads = a.tpr ? a.tpr : blockDim.x;
  const int group = threadIdx.x / threads, groups = blockDim.x / threads;
  const int t = threadIdx.x % threads;
  griddep_launch_dependents();
  griddep_wait();
  RowSum sum{red, a.tpr, 0};
  // up to 16 columns a thread gamma stays in registers; beyond that it would
  // push the sums out of them, and is read again (from L1) with every row
  constexpr bool kKeep = NV * VE <= 16;
  float g[kKeep ? NV : 1][VE], dg[NV][VE], db[NV][VE];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
    if constexpr (kKeep) load_weight<T>(g[k], a.gamma, a.wf32, c, a.C - c);
#pragma unroll
    for (int i = 0; i < VE; ++i) dg[k][i] = db[k][i] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(a.C);
  for (int64_t base = int64_t(blockIdx.x) * groups; base < a.M; base += int64_t(gridDim.x) * groups) {
    const bool live = base + group < a.M;
    const int64_t row = live ? base + group : a.M - 1;
    Vec<T> x[NV], dy[NV];
    const float mu = a.mean[row], rstd = a.rstd[row];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = a.C - c;
      if (n > 0 && live) {
        x[k].template load<AL>(static_cast<const T*>(a.x) + row * a.ldx + c, n);
        dy[k].template load<AL>(static_cast<const T*>(a.dy) + row * a.lddy + c, n);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int kg = kKeep ? k : 0;
      const int c = (t + k * threads) * VE;
      const int n = a.C - c;
      if constexpr (!kKeep) load_weight<T>(g[kg], a.gamma, a.wf32, c, n);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float d = to_f(dy[k].e[i]);
        const float z = live && i < n ? (to_f(x[k].e[i]) - mu) * rstd : 0.f;
        s.x = fmaf(d, g[kg][i], s.x);
        s.y = fmaf(d * g[kg][i], z, s.y);
        dg[k][i] = fmaf(d, z, dg[k][i]);
        db[k][i] += d;
      }
    }
    s = sum(s);
    const float m1 = s.x * inv, m2 = s.y * inv;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (t + k * threads) * VE;
      const int n = a.C - c;
      const int kg = kKeep ? k : 0;
      if (n <= 0) continue;
      if constexpr (!kKeep) load_weight<T>(g[kg], a.gamma, a.wf32, c, n);
      Vec<T> o, h;
      if (a.dh) h.template load<AL>(static_cast<const T*>(a.dh) + row * a.lddh + c, n);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        const float z = (to_f(x[k].e[i]) - mu) * rstd;
        float d = rstd * (fmaf(to_f(dy[k].e[i]), g[kg][i], -m1) - z * m2);
        if (a.dh) d += to_f(h.e[i]);
        o.e[i] = from_f<T>(d);
      }
      o.template store<AL>(static_cast<T*>(a.dx) + row * a.lddx + c, n);
    }
  }
  // groups of lanes that share their columns: summed in the order of the groups
  if (a.tpr) {
    extern __shared__ float cols[];  // [groups][2][threads * VE], NV = 1
    float* mine = cols + size_t(group) * 2 * threads * VE;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      mine[t * VE + i] = dg[0][i];
      mine[(threads + t) * VE + i] = db[0][i];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * threads * VE; j += blockDim.x) {
      float s = 0.f;
      for (int w = 0; w < groups; ++w) s += cols[size_t(w) * 2 * threads * VE + j];
      const int which = j / (threads * VE), c = j % (threads * VE);
      if (c < a.C) a.part[(int64_t(blockIdx.x) * 2 + which) * a.C + c] = s;
    }
    return;
  }
  float* p = a.part + int64_t(blockIdx.x) * 2 * a.C;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (t + k * threads) * VE;
#pragma unroll
    for (int i = 0; i < VE; ++i)
      if (c + i < a.C) {
        p[c + i] = dg[k][i];
        p[a.C + c + i] = db[k][i];
      }
  }
}

// dgamma and dbeta from the blocks' partial sums: 32 columns a block, the
// partial rows dealt to its warps, each sum in a fixed order.
__global__ void __launch_bounds__(512) ln_colsum_kernel(const float* part, int rows, int C, void* dgamma, void* dbeta,
                                                        int kind) {
  __shared__ float sm[16][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // column of the 2 C of a partial row
  griddep_launch_dependents();
  griddep_wait();
  float s = 0.f;
  if (c < 2 * C)
    for (int r = warp; r < rows; r += 16) s += part[int64_t(r) * 2 * C + c];
  sm[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * C) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sm[w][lane];
    void* out = c < C ? dgamma : dbeta;
    const int i = c < C ? c : c - C;
    if (out) {
      if (kind == SPG_F32) static_cast<float*>(out)[i] = s;
      else if (kind == SPG_F16) static_cast<__half*>(out)[i] = from_f<__half>(s);
      else static_cast<__nv_bfloat16*>(out)[i] = from_f<__nv_bfloat16>(s);
    }
  }
}

constexpr int kMaxC = 16384;

int esize(int dtype) { return dtype == SPG_F32 ? 4 : 2; }

// How a row is dealt to threads: lanes of one warp where NV vectors each are
// enough for it, else a block.
struct Shape {
  int tpr;      // lanes of a warp, or 0: the block
  int nv;       // vectors a thread
  int threads;  // of the block
};

int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

Shape fwd_shape(int C, int es) {
  const int nvec = (C * es + 15) / 16;
  if (nvec <= 32) {
    int tpr = 1;
    while (tpr < nvec) tpr *= 2;
    return {tpr, 1, 128};
  }
  if (nvec <= 128) return {32, (nvec + 31) / 32, 128};
  const int nv = nvec <= 512 ? 2 : 4;
  return {0, nv, round32((nvec + nv - 1) / nv)};
}

Shape bwd_shape(int C, int es) {
  const int nvec = (C * es + 15) / 16;
  if (nvec <= 32) {
    int tpr = 1;
    while (tpr < nvec) tpr *= 2;
    return {tpr, 1, 128};
  }
  const int nv = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  return {0, nv, round32((nvec + nv - 1) / nv)};
}

// Blocks of the backward kernel: enough to fill the device, a row group each
// at least.
int bwd_blocks(int64_t M, const Shape& s) {
  const int64_t groups = s.tpr ? s.threads / s.tpr : 1;
  const int64_t work = (M + groups - 1) / groups;
  const int64_t per_sm = 1024 / s.threads;
  const int64_t cap = int64_t(sm_count()) * (per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm);
  return static_cast<int>(work < cap ? work : cap);
}

template <class T, bool AL>
cudaError_t launch_fwd(const FwdArgs& a, const Shape& s, int64_t blocks, cudaStream_t st) {
  void (*k)(const FwdArgs) = s.nv == 1   ? ln_fwd_kernel<T, 1, AL>
                             : s.nv == 2 ? ln_fwd_kernel<T, 2, AL>
                             : s.nv == 3 ? ln_fwd_kernel<T, 3, AL>
                                         : ln_fwd_kernel<T, 4, AL>;
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(s.threads), 0, st, a);
}

template <class T, bool AL>
cudaError_t launch_bwd(const BwdArgs& a, const Shape& s, int blocks, cudaStream_t st) {
  void (*k)(const BwdArgs) = s.nv == 1   ? ln_bwd_kernel<T, 1, AL>
                             : s.nv == 2 ? ln_bwd_kernel<T, 2, AL>
                                         : ln_bwd_kernel<T, 4, AL>;
  const size_t smem = s.tpr ? size_t(s.threads) * 2 * Vec<T>::VE * sizeof(float) : 0;
  return launch_pdl(k, dim3(blocks), dim3(s.threads), smem, st, a);
}

bool vec_ok(const void* p, int64_t ld, int es) { return p == nullptr || (aligned(p, 16) && (ld * es) % 16 == 0); }

bool is_act(int d) { return d == SPG_F16 || d == SPG_BF16 || d == SPG_F32; }

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
  spg_status rc = check_device();
  if (rc != SPG_OK) return rc;
  const FwdArgs a{X,   res, H,   Y, gamma,         beta,          mean, rstd, ldx, ldres, ldh,
                  ldy, M, int(C), 0, wdtype == SPG_F32, s8, eps, qscale};
  Shape s = fwd_shape(int(C), es);
  FwdArgs b = a;
  b.tpr = s.tpr;
  const int64_t rows = s.tpr ? s.threads / s.tpr : 1;
  const int64_t blocks = (M + rows - 1) / rows;
  // rows that start on 16-byte boundaries move in 16-byte vectors, others element by element
  const bool al = vec_ok(X, ldx, es) && vec_ok(res, ldres, es) && vec_ok(H, ldh, es) &&
                  (s8 ? aligned(Y, 8) && ldy % 8 == 0 : vec_ok(Y, ldy, es));
  cudaError_t e;
  if (dtype == SPG_F32) e = al ? launch_fwd<float, true>(b, s, blocks, st) : launch_fwd<float, false>(b, s, blocks, st);
  else if (dtype == SPG_F16)
    e = al ? launch_fwd<__half, true>(b, s, blocks, st) : launch_fwd<__half, false>(b, s, blocks, st);
  else
    e = al ? launch_fwd<__nv_bfloat16, true>(b, s, blocks, st) : launch_fwd<__nv_bfloat16, false>(b, s, blocks, st);
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
  spg_status rc = check_device();
  if (rc != SPG_OK) return rc;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const Shape s = bwd_shape(int(C), es);
  int blocks = 0;
  if (M != 0) {
    blocks = bwd_blocks(M, s);
    const BwdArgs a{dY,  X,    dH,  dX,   gamma, mean,   rstd,  static_cast<float*>(workspace), lddy,
                    ldx, lddh, lddx, M, int(C), s.tpr, wdtype == SPG_F32};
    const bool al = vec_ok(dY, lddy, es) && vec_ok(X, ldx, es) && vec_ok(dH, lddh, es) && vec_ok(dX, lddx, es);
    cudaError_t e;
    if (dtype == SPG_F32) e = al ? launch_bwd<float, true>(a, s, blocks, st) : launch_bwd<float, false>(a, s, blocks, st);
    else if (dtype == SPG_F16)
      e = al ? launch_bwd<__half, true>(a, s, blocks, st) : launch_bwd<__half, false>(a, s, blocks, st);
    else
      e = al ? launch_bwd<__nv_bfloat16, true>(a, s, blocks, st) : launch_bwd<__nv_bfloat16, false>(a, s, blocks, st);
    if (e != cudaSuccess) return SPG_ERR_CUDA;
  }
  // no rows: the sums over them are zero
  if (launch_pdl(ln_colsum_kernel, dim3(static_cast<unsigned>((2 * C + 31) / 32)), dim3(512), 0, st,
                 static_cast<const float*>(workspace), blocks, int(C), dgamma, dbeta, int(wdtype)) != cudaSuccess)
    return SPG_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
