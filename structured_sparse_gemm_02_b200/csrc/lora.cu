// Low-rank adapters of many requests beside one shared (pruned) projection,
// forward and backward.  Row m uses adapter l = index[m], or none:
//
//   v = x A_l^T,  y = base + s_l v B_l^T              (A_l [R, K], B_l [N, R])
//   u = s_l dy B_l,  dx = dbase + u A_l
//   dA_l = sum over l's rows of u^T x,  dB_l = s_l sum over l's rows of dy^T v
//
// A plan (one small kernel per batch) groups the rows by adapter; every product
// then runs on tiles of up to 128 rows of one adapter, whose rows TMA gathers
// by index.  Three tcgen05 kernels cover all products:
//   shrink  P = T G^T for T = X (G = A_l) or T = dY (G = B_l^T)
//   expand  Y = base + s P G^T for G = B_l or G = A_l^T
//   wgrad   dG = s T^T P for (X, U) and (dY, V)
// R is at most 128, so each of them is bound by the reads and writes of its
// large matrix.  V and U are rounded to the activations' type between the
// products: V is saved for the backward pass as any activation is, and both
// are operands of the tensor cores; every sum is fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gather.cuh"
#include "host.cuh"
#include "sm100.cuh"
#include "spgemm.h"

namespace spg {
namespace lora {

constexpr int kTile = 128;  // rows of a tile: the M of one MMA
constexpr int kMaxL = 8192;
constexpr int kMaxR = 128;

// ---- the plan ---------------------------------------------------------------------
// int32 words: [0] number of tiles; start[L + 2] (rows of each adapter, then
// those without one, as positions); perm[M] (the row at each position, the
// rows of a group ascending); tiles {adapter or -1, first position, rows, 0}.
struct Plan {
  int* hdr;
  int* start;
  int* perm;
  int4* tiles;
};

__host__ __device__ inline int64_t round4(int64_t v) { return (v + 3) / 4 * 4; }

inline int64_t max_tiles(int64_t M, int64_t L) { return M / kTile + (L + 1 < M ? L + 1 : M); }

inline size_t plan_ints(int64_t M, int64_t L) {
  return static_cast<size_t>(4 + round4(L + 2) + round4(M) + 4 * max_tiles(M, L));
}

inline Plan plan_view(const int32_t* p, int64_t M, int64_t L) {
  int* b = const_cast<int*>(p);
  return Plan{b, b + 4, b + 4 + round4(L + 2), reinterpret_cast<int4*>(b + 4 + round4(L + 2) + round4(M))};
}

// Groups the rows by adapter, in one block.  Each warp takes a strip of
// consecutive rows and counts its own occurrences of every adapter (lanes that
// share one vote, the lowest adds), so the order of a group's rows does not
// depend on timing.
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* __restrict__ index, int M, int L, int warps,
                                                    Plan p) {
  extern __shared__ int cnt[];  // [warps][L + 1]
  __shared__ int2 wsum[32];
  __shared__ int2 carry;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = L + 1;
  griddep_launch_dependents();
  griddep_wait();
  for (int i = threadIdx.x; i < warps * G; i += blockDim.x) cnt[i] = 0;
  if (threadIdx.x == 0) carry = make_int2(0, 0);
  __syncthreads();
  const int strip = (M + warps * 32 - 1) / (warps * 32) * 32;
  const int r0 = warp * strip, r1 = min(M, r0 + strip);
  if (warp < warps) {
    for (int r = r0; r < r1; r += 32) {
      const int row = r + lane;
      int a = -1;
      if (row < r1) {
        a = index[row];
        if (a < 0 || a >= L) a = L;
      }
      const unsigned same = __match_any_sync(0xffffffffu, a);
      if (a >= 0 && lane == __ffs(same) - 1) cnt[warp * G + a] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // rows and tiles before each group: a block scan over 1024 groups at a time
  for (int g0 = 0; g0 < G; g0 += blockDim.x) {
    const int g = g0 + threadIdx.x;
    int rows = 0;
    if (g < G)
      for (int w = 0; w < warps; ++w) rows += cnt[w * G + g];
    const int2 own = make_int2(rows, (rows + kTile - 1) / kTile);
    int2 v = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
      if (lane >= o) {
        v.x += x;
        v.y += y;
      }
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    int2 base = carry;
    for (int w = 0; w < warp; ++w) {
      base.x += wsum[w].x;
      base.y += wsum[w].y;
    }
    v.x += base.x - own.x;  // exclusive
    v.y += base.y - own.y;
    if (g < G) {
      p.start[g] = v.x;
      if (g == L) {
        p.start[G] = v.x + rows;
        p.hdr[0] = v.y + own.y;
      }
      for (int t = 0; t < own.y; ++t)
        p.tiles[v.y + t] =
            make_int4(g < L ? g : -1, v.x + t * kTile, min(kTile, rows - t * kTile), 0);
      int at = v.x;
      for (int w = 0; w < warps; ++w) {
        const int n = cnt[w * G + g];
        cnt[w * G + g] = at;
        at += n;
      }
    }
    __syncthreads();
    if (threadIdx.x == blockDim.x - 1) carry = make_int2(v.x + own.x, v.y + own.y);
    __syncthreads();
  }
  if (warp < warps) {
    for (int r = r0; r < r1; r += 32) {
      const int row = r + lane;
      int a = -1;
      if (row < r1) {
        a = index[row];
        if (a < 0 || a >= L) a = L;
      }
      const unsigned same = __match_any_sync(0xffffffffu, a);
      int at = 0;
      if (a >= 0) at = cnt[warp * G + a];
      __syncwarp();
      if (a >= 0) {
        p.perm[at + __popc(same & ((1u << lane) - 1))] = row;
        if (lane == __ffs(same) - 1) cnt[warp * G + a] = at + __popc(same);
      }
      __syncwarp();
    }
  }
}

// ---- shared pieces ------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint16_t pack1(float v) {
  return static_cast<uint16_t>(pack2<BF16>(v, 0.f) & 0xFFFFu);
}
template <bool BF16>
__device__ __forceinline__ float unpack1(uint16_t v) {
  return unpack2<BF16>(v).x;
}

// Bounded wait that ignores the abort flag (teardown, and the one wait that everything else follows).
__device__ __forceinline__ void tail_wait(uint64_t* bar, uint32_t parity, uint32_t* err) {
  int never = 0;
  mbar_wait(bar, parity, &never, err, ERR_WAIT_TAIL);
}

// Barriers of a block and its tensor memory, behind the operand ring.
struct Ring {
  uint64_t* full;
  uint64_t* empty;
  uint64_t* done;
  uint64_t* aux;
  uint32_t* tmem;
  volatile int* abort_flag;
};
constexpr int kMaxStages = 8;
constexpr int kBarBytes = (2 * kMaxStages + 2) * 8 + 16;

__device__ __forceinline__ Ring ring_at(uint8_t* p) {
  Ring r;
  r.full = reinterpret_cast<uint64_t*>(p);
  r.empty = r.full + kMaxStages;
  r.done = r.empty + kMaxStages;
  r.aux = r.done + 1;
  r.tmem = reinterpret_cast<uint32_t*>(r.aux + 1);
  r.abort_flag = reinterpret_cast<volatile int*>(r.tmem + 1);
  return r;
}

__device__ __forceinline__ void ring_init(const Ring& r, uint32_t tmem_cols, int warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&r.full[s], 1);
      mbar_init(&r.empty[s], 1);
    }
    mbar_init(r.done, 1);
    mbar_init(r.aux, 1);
    *r.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(r.tmem, tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now: a dependent kernel that takes tensor memory before it waits for
  // this one must not get ahead of a block of this one that still needs its own.
  griddep_launch_dependents();
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__host__ __device__ inline int round16(int r) { return (r + 15) & ~15; }
// Tensor-memory columns for n accumulator columns: a power of two, at least 32.
__host__ __device__ inline uint32_t tmem_cols(int n) { return n <= 32 ? 32u : n <= 64 ? 64u : n <= 128 ? 128u : 256u; }

// The 128-byte-swizzled tiles below are rows of 64 elements (128 bytes), eight
// rows to a 1024-byte group.  Read with the row as the MMA's M or N index they
// are K-major; with the row as its K index, M- or N-major: then the leading
// offset steps between tiles of 64 columns and the stride offset between
// groups of eight rows.
__device__ __forceinline__ uint64_t desc_k_major(const void* p) {
  return smem_desc(smem_addr(p), 16, 1024, LAYOUT_SW128);
}
__device__ __forceinline__ uint64_t desc_mn_major(const void* p, uint32_t next64) {
  return smem_desc(smem_addr(p), next64, 1024, LAYOUT_SW128);
}

// Rows 4 lane .. 4 lane + 3 of a tile for one gather; positions past its end
// name a row past the matrix, which reads as zeros.
__device__ __forceinline__ int4 tile_rows(const int* perm, int pos, int count, int j, int M) {
  int4 r;
  r.x = j + 0 < count ? perm[pos + j + 0] : M;
  r.y = j + 1 < count ? perm[pos + j + 1] : M;
  r.z = j + 2 < count ? perm[pos + j + 2] : M;
  r.w = j + 3 < count ? perm[pos + j + 3] : M;
  return r;
}

// ---- shrink: P [rows][R] = T [rows][D] . G^T ----------------------------------------
// One cluster a tile; its blocks split D in steps of 64, accumulate their
// parts in tensor memory and add them through distributed shared memory in
// the order of the ranks.  Warp 0 gathers T rows and loads G, one thread of
// warp 1 issues the MMAs, all four warps read the accumulators.
//   GMN false: G = A_l [R][D], a [64][R rows] box, K-major
//   GMN true:  G = B_l [D][R], boxes of 64 rows x 64 columns, N-major
struct ShrinkArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  void* P;
  int64_t ldp;
  int M, D, R, stages, gbytes;
  uint32_t* err;
};

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(128) shrink_kernel(const __grid_constant__ CUtensorMap tmT,
                                                     const __grid_constant__ CUtensorMap tmG, const ShrinkArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = cluster_nctarank(), rank = cluster_ctarank();
  griddep_wait();
  const int tile = blockIdx.x / cs;
  if (tile >= a.plan.hdr[0]) return;
  const int4 t = a.plan.tiles[tile];
  const int adapter = t.x, pos = t.y, count = t.z;
  const int R = a.R, vecs = R / 8;
  uint16_t* P = static_cast<uint16_t*>(a.P);
  if (adapter < 0) {  // rows without an adapter: zeros
    if (rank == 0)
      for (int i = threadIdx.x; i < count * vecs; i += blockDim.x)
        *reinterpret_cast<uint4*>(P + int64_t(a.plan.perm[pos + i / vecs]) * a.ldp + (i % vecs) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int Rn = round16(R);
  const int stage_bytes = kTile * 128 + a.gbytes;
  const Ring ring = ring_at(smem + a.stages * stage_bytes);
  ring_init(ring, tmem_cols(Rn), warp);
  const uint32_t tmem = *ring.tmem;
  const int nkb = (a.D + 63) / 64;
  const int kb0 = int(int64_t(nkb) * rank / cs), n = int(int64_t(nkb) * (rank + 1) / cs) - kb0;

  if (warp == 0) {
    const int groups = (count + 3) / 4;
    const int4 rows = tile_rows(a.plan.perm, pos, count, 4 * lane, a.M);
    const uint32_t tx = groups * 512 + a.gbytes;
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % a.stages;
      const uint32_t use = i / a.stages;
      if (use > 0 && !mbar_wait_warp(&ring.empty[s], (use - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      const int k = (kb0 + i) * 64;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], tx);
      __syncwarp();
      if (lane < groups) tma_gather4(st + lane * 512, &tmT, k, rows, &ring.full[s]);
      if (lane == 0) {
        if constexpr (GMN) {
          tma_load_3d(st + kTile * 128, &tmG, 0, k, adapter, &ring.full[s]);
          if (R > 64) tma_load_3d(st + kTile * 128 + 8192, &tmG, 64, k, adapter, &ring.full[s]);
        } else {
          tma_load_3d(st + kTile * 128, &tmG, k, 0, adapter, &ring.full[s]);
        }
      }
      __syncwarp();
    }
    if (lane == 0)  // nothing is in flight when the block goes on
      for (int q = i > a.stages ? i - a.stages : 0; q < i; ++q)
        tail_wait(&ring.full[q % a.stages], (q / a.stages) & 1, a.err);
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = instr_desc_major(BF16, kTile, Rn, 0, GMN ? 1 : 0);
      for (int i = 0; i < n; ++i) {
        const int s = i % a.stages;
        if (!mbar_wait(&ring.full[s], (i / a.stages) & 1, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
        tc_fence_after();
        uint8_t* st = smem + s * stage_bytes;
        const uint64_t ad = desc_k_major(st);
        const uint64_t bd = GMN ? desc_mn_major(st + kTile * 128, 8192) : desc_k_major(st + kTile * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma(tmem, ad + ((32 * k) >> 4), bd + ((GMN ? 2048 * k : 32 * k) >> 4), idesc, (i | k) != 0);
        tc_commit(&ring.empty[s]);
      }
      tc_commit(ring.done);
    }
    __syncwarp();
  }
  tail_wait(ring.done, 0, a.err);
  __syncwarp();
  __syncthreads();  // the ring is idle: it takes the partial sums
  tc_fence_after();
  const int pitch = R + 4;  // floats; rows of 16-byte vectors that no two lanes of a quarter warp share banks in
  float* part = reinterpret_cast<float*>(smem);
  if (32 * warp < count) {
    float* mine = part + (32 * warp + lane) * pitch;
    for (int c = 0; c < R; c += 8) {
      uint32_t r[8];
      tmem_ld_32x32b_x8(tmem + (uint32_t(32 * warp) << 16) + c, r);
      tmem_ld_wait(r);
      *reinterpret_cast<uint4*>(mine + c) = make_uint4(r[0], r[1], r[2], r[3]);
      *reinterpret_cast<uint4*>(mine + c + 4) = make_uint4(r[4], r[5], r[6], r[7]);
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols(Rn));
  }
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  const int per = kTile / cs;
  for (int i = threadIdx.x; i < per * vecs; i += blockDim.x) {
    const int row = rank * per + i / vecs, c = (i % vecs) * 8;
    if (row >= count) break;
    const uint32_t at = smem_addr(part + row * pitch + c);
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
    for (int q = 0; q < cs; ++q) {
      const uint32_t from = mapa_shared(at, q);
      const float4 x = ld_cluster_f4(from), y = ld_cluster_f4(from + 16);
      lo.x += x.x; lo.y += x.y; lo.z += x.z; lo.w += x.w;
      hi.x += y.x; hi.y += y.y; hi.z += y.z; hi.w += y.w;
    }
    uint4 o;
    o.x = pack2<BF16>(lo.x * scale, lo.y * scale);
    o.y = pack2<BF16>(lo.z * scale, lo.w * scale);
    o.z = pack2<BF16>(hi.x * scale, hi.y * scale);
    o.w = pack2<BF16>(hi.z * scale, hi.w * scale);
    *reinterpret_cast<uint4*>(P + int64_t(a.plan.perm[pos + row]) * a.ldp + c) = o;
  }
  __syncwarp();
  cluster_sync();  // no block leaves while another may still read its shared memory
}

// ---- expand: Y [rows][C] = base + s P [rows][R] . G^T ---------------------------------
// One block a tile and 128 columns.  The rows of base come in by bulk copies
// (one a row) while the MMA runs, the sum is rounded in place and goes out the
// same way; the columns behind the last multiple of 8 move element by element.
//   GMN false: G = B_l [C][R];  GMN true: G = A_l [R][C]
struct ExpandArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  const void* base;    // nullptr: 0
  void* Y;
  int64_t ldb, ldy;
  int M, C, R;
  uint32_t* err;
};

constexpr int kExpCols = 128;
constexpr int kExpPitch = kExpCols * 2 + 16;  // bytes of a staged row: 16-byte accesses of eight lanes miss each other

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(128) expand_kernel(const __grid_constant__ CUtensorMap tmP,
                                                     const __grid_constant__ CUtensorMap tmG, const ExpandArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  if (int(blockIdx.y) >= a.plan.hdr[0]) return;
  const int4 t = a.plan.tiles[blockIdx.y];
  const int adapter = t.x, pos = t.y, count = t.z;
  const int n0 = blockIdx.x * kExpCols;
  const int cols = min(kExpCols, a.C - n0);
  const bool live = int(threadIdx.x) < count;
  const int64_t row = live ? a.plan.perm[pos + threadIdx.x] : 0;
  const uint16_t* base = static_cast<const uint16_t*>(a.base);
  uint16_t* Y = static_cast<uint16_t*>(a.Y);
  if (adapter < 0) {  // rows without an adapter: base as it is
    if (base == Y) return;
    for (int r = warp; r < count; r += 4) {
      const int64_t from = a.plan.perm[pos + r];
      for (int c = lane * 4; c < cols; c += 128) {
        uint16_t* o = Y + from * a.ldy + n0 + c;
        const uint16_t* b = base + from * a.ldb + n0 + c;
        if (c + 4 <= cols)
          *reinterpret_cast<uint2*>(o) = base ? *reinterpret_cast<const uint2*>(b) : make_uint2(0u, 0u);
        else
          for (int e = 0; e < cols - c; ++e) o[e] = base ? b[e] : uint16_t(0);
      }
    }
    return;
  }
  const int Rn = round16(a.R);
  const int halves = a.R > 64 ? 2 : 1;
  uint8_t* Ps = smem;
  uint8_t* Gs = Ps + halves * kTile * 128;
  const int gbytes = GMN ? 2 * Rn * 128 : halves * kExpCols * 128;
  uint8_t* Ys = Gs + gbytes;
  const Ring ring = ring_at(Ys + kTile * kExpPitch);
  ring_init(ring, kExpCols, warp);
  const uint32_t tmem = *ring.tmem;
  const int bulk = cols / 8 * 8;  // columns that move in 16-byte pieces
  uint8_t* mine = Ys + threadIdx.x * kExpPitch;
  if (warp == 0) {
    const int groups = (count + 3) / 4;
    const int4 rows = tile_rows(a.plan.perm, pos, count, 4 * lane, a.M);
    if (lane == 0) {
      if (base && bulk) mbar_arrive_expect_tx(ring.aux, uint32_t(count) * bulk * 2);
      mbar_arrive_expect_tx(&ring.full[0], halves * groups * 512 + gbytes);
    }
    __syncwarp();
    for (int h = 0; h < halves; ++h)
      if (lane < groups) tma_gather4(Ps + h * kTile * 128 + lane * 512, &tmP, 64 * h, rows, &ring.full[0]);
    if (lane == 0) {
      if constexpr (GMN) {
        tma_load_3d(Gs, &tmG, n0, 0, adapter, &ring.full[0]);
        tma_load_3d(Gs + Rn * 128, &tmG, n0 + 64, 0, adapter, &ring.full[0]);
      } else {
        for (int h = 0; h < halves; ++h)
          tma_load_3d(Gs + h * kExpCols * 128, &tmG, 64 * h, n0, adapter, &ring.full[0]);
      }
    }
    __syncwarp();
  }
  if (base && bulk && live) bulk_load(smem_addr(mine), base + row * a.ldb + n0, bulk * 2, ring.aux);
  if (warp == 1) {
    if (lane == 0) {
      tail_wait(&ring.full[0], 0, a.err);
      tc_fence_after();
      const uint32_t idesc = instr_desc_major(BF16, kTile, kExpCols, 0, GMN ? 1 : 0);
      for (int k = 0; k < Rn / 16; ++k) {
        const uint64_t ad = desc_k_major(Ps + (k >> 2) * kTile * 128) + ((32 * (k & 3)) >> 4);
        const uint64_t bd = GMN ? desc_mn_major(Gs + 2048 * k, Rn * 128)
                                : desc_k_major(Gs + (k >> 2) * kExpCols * 128) + ((32 * (k & 3)) >> 4);
        tc_mma(tmem, ad, bd, idesc, k != 0);
      }
      tc_commit(ring.done);
    }
    __syncwarp();
  }
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  tail_wait(ring.done, 0, a.err);
  if (base && bulk) tail_wait(ring.aux, 0, a.err);
  __syncwarp();
  tc_fence_after();
  if (32 * warp < count) {
#pragma unroll 1
    for (int c = 0; c < cols; c += 32) {
      uint32_t h[32];
      tmem_ld_32x32b_x32(tmem + (uint32_t(32 * warp) << 16) + c, h);
      tmem_ld_wait(h);
      if (live) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int at = c + 8 * v;
          if (at + 8 <= cols) {
            uint4 b = make_uint4(0u, 0u, 0u, 0u);
            if (base) b = *reinterpret_cast<const uint4*>(mine + at * 2);
            uint32_t* bw = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack2<BF16>(bw[e]);
              bw[e] = pack2<BF16>(fmaf(scale, __uint_as_float(h[8 * v + 2 * e]), f.x),
                                  fmaf(scale, __uint_as_float(h[8 * v + 2 * e + 1]), f.y));
            }
            *reinterpret_cast<uint4*>(mine + at * 2) = b;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (at + e < cols) {
                const float f = base ? unpack1<BF16>(base[row * a.ldb + n0 + at + e]) : 0.f;
                Y[row * a.ldy + n0 + at + e] = pack1<BF16>(fmaf(scale, __uint_as_float(h[8 * v + e]), f));
              }
          }
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  if (live && bulk) {
    fence_proxy_async_smem();
    bulk_store(Y + row * a.ldy + n0, smem_addr(mine), bulk * 2);
    bulk_commit();
    bulk_wait_all<0>();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kExpCols);
  }
}

// ---- wgrad: dG_l [C][R] = s_l sum over l's rows of T[m][c] P[m][r] ----------------------
// One cluster a block of 256 columns of T and an adapter; its blocks split
// the adapter's rows in chunks of 64 and add their sums as shrink_kernel does.
// Both operands are read with the row as the MMA's K index.
//   OT false: dG is [C][R] (dB);  OT true: [R][C] (dA)
struct WgradArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  void* dG;
  int M, C, R, stages;
  uint32_t* err;
};

constexpr int kWgCols = 256;

template <bool BF16, bool OT>
__global__ void __launch_bounds__(128) wgrad_kernel(const __grid_constant__ CUtensorMap tmT,
                                                    const __grid_constant__ CUtensorMap tmP, const WgradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = cluster_nctarank(), rank = cluster_ctarank();
  griddep_wait();
  const int adapter = blockIdx.y;
  const int c0 = int(blockIdx.x / cs) * kWgCols;
  const int cols = min(kWgCols, a.C - c0);
  const int R = a.R, vecs = R / 8;
  const int start = a.plan.start[adapter], rows = a.plan.start[adapter + 1] - start;
  uint16_t* dG = static_cast<uint16_t*>(a.dG) + int64_t(adapter) * a.C * R;
  if (rows == 0) {  // an adapter without rows: zeros
    if (rank == 0) {
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (OT) {
        for (int i = threadIdx.x; i < R * (cols / 8); i += blockDim.x)
          *reinterpret_cast<uint4*>(dG + int64_t(i / (cols / 8)) * a.C + c0 + (i % (cols / 8)) * 8) = z;
      } else {
        for (int i = threadIdx.x; i < cols * vecs; i += blockDim.x)
          *reinterpret_cast<uint4*>(dG + int64_t(c0 + i / vecs) * R + (i % vecs) * 8) = z;
      }
    }
    return;
  }
  const int Rn = round16(R), halves = R > 64 ? 2 : 1;
  const int subs = (cols + 63) / 64;  // tiles of 64 columns inside the matrix
  const int tbytes = (kWgCols / 64) * 8192;
  const int stage_bytes = tbytes + halves * 8192;
  const int part_bytes = kWgCols * (R + 4) * 4;
  const int ring_bytes = a.stages * stage_bytes;
  const Ring ring = ring_at(smem + (ring_bytes > part_bytes ? ring_bytes : part_bytes));
  const uint32_t tcols = tmem_cols(2 * Rn);
  ring_init(ring, tcols, warp);
  const uint32_t tmem = *ring.tmem;
  const int chunks = (rows + 63) / 64;
  const int q0 = int(int64_t(chunks) * rank / cs), n = int(int64_t(chunks) * (rank + 1) / cs) - q0;

  if (warp == 0) {
    const uint32_t tx = (subs + halves) * 8192;
    const int group = lane & 15;
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % a.stages;
      const uint32_t use = i / a.stages;
      const int at = (q0 + i) * 64;
      const int4 r = tile_rows(a.plan.perm, start + at, rows - at, 4 * group, a.M);
      if (use > 0 && !mbar_wait_warp(&ring.empty[s], (use - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], tx);
      __syncwarp();
      for (int j = lane >> 4; j < subs; j += 2)
        tma_gather4(st + j * 8192 + group * 512, &tmT, c0 + 64 * j, r, &ring.full[s]);
      if ((lane >> 4) < halves)
        tma_gather4(st + tbytes + (lane >> 4) * 8192 + group * 512, &tmP, 64 * (lane >> 4), r, &ring.full[s]);
      __syncwarp();
    }
    if (lane == 0)
      for (int q = i > a.stages ? i - a.stages : 0; q < i; ++q)
        tail_wait(&ring.full[q % a.stages], (q / a.stages) & 1, a.err);
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = instr_desc_major(BF16, 128, Rn, 1, 1);
      for (int i = 0; i < n; ++i) {
        const int s = i % a.stages;
        if (!mbar_wait(&ring.full[s], (i / a.stages) & 1, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
        tc_fence_after();
        uint8_t* st = smem + s * stage_bytes;
        const uint64_t bd = desc_mn_major(st + tbytes, 8192);
        for (int h = 0; h < 2 && 128 * h < cols; ++h) {
          const uint64_t ad = desc_mn_major(st + h * 16384, 8192);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma(tmem + h * Rn, ad + ((2048 * k) >> 4), bd + ((2048 * k) >> 4), idesc, (i | k) != 0);
        }
        tc_commit(&ring.empty[s]);
      }
      tc_commit(ring.done);
    }
    __syncwarp();
  }
  tail_wait(ring.done, 0, a.err);
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const int pitch = R + 4;
  float* part = reinterpret_cast<float*>(smem);
  if (n > 0) {
    for (int h = 0; h < 2 && 128 * h < cols; ++h) {
      float* mine = part + (128 * h + 32 * warp + lane) * pitch;
      for (int c = 0; c < R; c += 8) {
        uint32_t r[8];
        tmem_ld_32x32b_x8(tmem + (uint32_t(32 * warp) << 16) + h * Rn + c, r);
        tmem_ld_wait(r);
        *reinterpret_cast<uint4*>(mine + c) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(mine + c + 4) = make_uint4(r[4], r[5], r[6], r[7]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  const int per = kWgCols / cs;  // columns this block adds up
  for (int i = threadIdx.x; i < per * vecs; i += blockDim.x) {
    // a vector of 8 sums: 8 r of one column, or 8 columns of one r
    int c, r;
    if constexpr (OT) {
      r = i / (per / 8);
      c = rank * per + (i % (per / 8)) * 8;
    } else {
      c = rank * per + i / vecs;
      r = (i % vecs) * 8;
    }
    if (c >= cols) continue;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int q = 0; q < cs; ++q) {
      if (int(int64_t(chunks) * (q + 1) / cs) == int(int64_t(chunks) * q / cs)) continue;  // a block without rows
      const uint32_t from = mapa_shared(smem_addr(part + c * pitch + r), q);
      if constexpr (OT) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += ld_cluster_f(from + e * pitch * 4);
      } else {
        const float4 x = ld_cluster_f4(from), y = ld_cluster_f4(from + 16);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
    }
    uint4 o;
    o.x = pack2<BF16>(v[0] * scale, v[1] * scale);
    o.y = pack2<BF16>(v[2] * scale, v[3] * scale);
    o.z = pack2<BF16>(v[4] * scale, v[5] * scale);
    o.w = pack2<BF16>(v[6] * scale, v[7] * scale);
    *reinterpret_cast<uint4*>(OT ? dG + int64_t(r) * a.C + c0 + c : dG + int64_t(c0 + c) * R + r) = o;
  }
  __syncwarp();
  cluster_sync();
}

// ---- host ---------------------------------------------------------------------------
// Shared-memory budget of a ring: two blocks an SM.
constexpr int kRingBudget = 100 * 1024;

template <class K>
spg_status prepare(K kern, int smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess ? SPG_OK
                                                                                                      : SPG_ERR_CUDA;
}

// T rows for gathers: boxes of one row of 64 columns.
bool rows_map(CUtensorMap* m, const void* p, int64_t cols, int64_t rows, int64_t ld) {
  return make_tmap_2d(m, p, 2, uint64_t(cols), uint64_t(rows), uint64_t(ld) * 2, 64, 1, true);
}

template <bool BF16, bool GMN>
spg_status shrink(const void* T, int64_t ldt, const void* G, const float* scale, const Plan& plan, void* P, int64_t ldp,
                  int64_t M, int64_t D, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  const int Rn = round16(int(R));
  CUtensorMap tmT, tmG;
  if (!rows_map(&tmT, T, D, M, ldt)) return SPG_ERR_CUDA;
  if (!(GMN ? make_tmap_3d(&tmG, G, R, D, L, 64, 64) : make_tmap_3d(&tmG, G, D, R, L, 64, Rn))) return SPG_ERR_CUDA;
  const int gbytes = GMN ? (R > 64 ? 16384 : 8192) : Rn * 128;
  const int stage = kTile * 128 + gbytes;
  int stages = kRingBudget / stage;
  stages = stages > kMaxStages ? kMaxStages : stages;
  // blocks of a cluster: enough to fill the device with the tiles of full
  // groups, each with at least two steps of its own
  const int64_t tiles = max_tiles(M, L), nkb = (D + 63) / 64;
  const int64_t busy = (M + kTile - 1) / kTile;
  int cs = 1;
  while (cs < 8 && busy * cs < 2 * sm_count() && nkb >= 4 * cs) cs *= 2;
  const int ring = stages * stage, part = kTile * (int(R) + 4) * 4;
  if (part > ring) return SPG_ERR_UNSUPPORTED_SHAPE;
  const int smem = ring + kBarBytes + 1024;
  auto kern = shrink_kernel<BF16, GMN>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const ShrinkArgs a{plan, scale, P, ldp, int(M), int(D), int(R), stages, gbytes, err};
  return launch_pdl_cluster(kern, dim3(unsigned(tiles * cs)), dim3(128), smem, cs, st, tmT, tmG, a) == cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

template <bool BF16, bool GMN>
spg_status expand(const void* P, int64_t ldp, const void* G, const float* scale, const Plan& plan, const void* base,
                  int64_t ldb, void* Y, int64_t ldy, int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err,
                  cudaStream_t st) {
  const int Rn = round16(int(R)), halves = R > 64 ? 2 : 1;
  CUtensorMap tmP, tmG;
  if (!rows_map(&tmP, P, R, M, ldp)) return SPG_ERR_CUDA;
  if (!(GMN ? make_tmap_3d(&tmG, G, C, R, L, 64, Rn) : make_tmap_3d(&tmG, G, R, C, L, 64, kExpCols)))
    return SPG_ERR_CUDA;
  const int smem = halves * kTile * 128 + (GMN ? 2 * Rn * 128 : halves * kExpCols * 128) + kTile * kExpPitch +
                   kBarBytes + 1024;
  auto kern = expand_kernel<BF16, GMN>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const ExpandArgs a{plan, scale, base, Y, ldb, ldy, int(M), int(C), int(R), err};
  const dim3 grid(unsigned((C + kExpCols - 1) / kExpCols), unsigned(max_tiles(M, L)));
  return launch_pdl(kern, grid, dim3(128), smem, st, tmP, tmG, a) == cudaSuccess ? launch_status() : SPG_ERR_CUDA;
}

template <bool BF16, bool OT>
spg_status wgrad(const void* T, int64_t ldt, const void* P, int64_t ldp, const float* scale, const Plan& plan, void* dG,
                 int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  CUtensorMap tmT, tmP;
  if (!rows_map(&tmT, T, C, M, ldt) || !rows_map(&tmP, P, R, M, ldp)) return SPG_ERR_CUDA;
  const int stage = (kWgCols / 64 + (R > 64 ? 2 : 1)) * 8192;
  const int stages = 204800 / stage;
  const int64_t blocks = (C + kWgCols - 1) / kWgCols;
  const int64_t groups = L < 4 ? L : 4;
  int cs = 1;
  while (cs < 8 && blocks * groups * cs < 2 * sm_count() && M / groups >= 128 * cs) cs *= 2;
  const int ring = stages * stage, part = kWgCols * (int(R) + 4) * 4;
  const int smem = (ring > part ? ring : part) + kBarBytes + 1024;
  auto kern = wgrad_kernel<BF16, OT>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const WgradArgs a{plan, scale, dG, int(M), int(C), int(R), stages, err};
  return launch_pdl_cluster(kern, dim3(unsigned(blocks * cs), unsigned(L)), dim3(128), smem, cs, st, tmT, tmP, a) ==
                 cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

bool mat_ok(const void* p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// Sizes, pointers and alignment that the forward and backward calls share.
spg_status validate(const void* X, int64_t ldx, const void* A, const void* B, const float* scale, const int32_t* plan,
                    const void* V, int64_t ldv, int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                    spg_dtype dtype) {
  if (dtype != SPG_F16 && dtype != SPG_BF16) return SPG_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || K <= 0 || R <= 0 || L <= 0 || ldx < K || ldv < R) return SPG_ERR_INVALID_ARG;
  if (!A || !B || (M != 0 && (!X || !V || !plan))) return SPG_ERR_INVALID_ARG;
  if (K % 8 || R % 8 || R > kMaxR || L > kMaxL) return SPG_ERR_UNSUPPORTED_SHAPE;
  const int64_t lim = int64_t(1) << 31;
  if (M >= (int64_t(1) << 22) || N >= lim - 256 || K >= lim - 256) return SPG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(scale, 4) || !aligned(plan, 16)) return SPG_ERR_MISALIGNED;
  if (M != 0 && (!mat_ok(X, ldx) || !mat_ok(V, ldv))) return SPG_ERR_MISALIGNED;
  return SPG_OK;
}

template <bool BF16>
spg_status forward(const void* X, int64_t ldx, const void* A, const void* B, const float* scale, const Plan& plan,
                   void* V, int64_t ldv, const void* base, int64_t ldbase, void* Y, int64_t ldy, int64_t M, int64_t N,
                   int64_t K, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  spg_status rc = shrink<BF16, false>(X, ldx, A, nullptr, plan, V, ldv, M, K, R, L, err, st);
  if (rc != SPG_OK) return rc;
  return expand<BF16, false>(V, ldv, B, scale, plan, base, ldbase, Y, ldy, M, N, R, L, err, st);
}

template <bool BF16>
spg_status backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* V, int64_t ldv, const void* A,
                    const void* B, const float* scale, const Plan& plan, const void* dbase, int64_t lddb, void* dX,
                    int64_t lddx, void* dA, void* dB, void* U, int64_t M, int64_t N, int64_t K, int64_t R, int64_t L,
                    uint32_t* err, cudaStream_t st) {
  spg_status rc = shrink<BF16, true>(dY, lddy, B, scale, plan, U, R, M, N, R, L, err, st);
  if (rc == SPG_OK) rc = wgrad<BF16, false>(dY, lddy, V, ldv, scale, plan, dB, M, N, R, L, err, st);
  if (rc == SPG_OK) rc = wgrad<BF16, true>(X, ldx, U, R, nullptr, plan, dA, M, K, R, L, err, st);
  if (rc == SPG_OK && dX)
    rc = expand<BF16, true>(U, R, A, nullptr, plan, dbase, lddb, dX, lddx, M, K, R, L, err, st);
  return rc;
}

}  // namespace lora
}  // namespace spg

extern "C" {

size_t lora_plan_size(int64_t M, int64_t L) {
  using namespace spg::lora;
  if (M < 0 || L <= 0 || L > kMaxL || M >= (int64_t(1) << 22)) return 0;
  return plan_ints(M, L) * sizeof(int32_t);
}

spg_status lora_plan(const int32_t* index, int64_t M, int64_t L, int32_t* plan, size_t plan_bytes,
                     spg_stream_t stream) {
  using namespace spg;
  using namespace spg::lora;
  if (M < 0 || L <= 0 || !plan || (M != 0 && !index)) return SPG_ERR_INVALID_ARG;
  if (L > kMaxL || M >= (int64_t(1) << 22)) return SPG_ERR_UNSUPPORTED_SHAPE;
  if (plan_bytes < lora_plan_size(M, L)) return SPG_ERR_INVALID_ARG;
  if (!aligned(index, 4) || !aligned(plan, 16)) return SPG_ERR_MISALIGNED;
  spg_status rc = check_device();
  if (rc != SPG_OK) return rc;
  // counters of one warp a row of shared memory: as many warps as fit and have rows
  const int64_t G = L + 1;
  int64_t warps = 196608 / (4 * G);
  const int64_t need = (M + 31) / 32;
  warps = warps > 32 ? 32 : warps;
  warps = warps > need ? (need > 0 ? need : 1) : warps;
  const int smem = int(warps * G * 4);
  if (smem > 48 * 1024 && prepare(plan_kernel, smem) != SPG_OK) return SPG_ERR_CUDA;
  // every group needs a thread of its own in the scan, every strip a warp
  const int64_t threads = ((G > warps * 32 ? G : warps * 32) + 31) / 32 * 32;
  if (launch_pdl(plan_kernel, dim3(1), dim3(unsigned(threads > 1024 ? 1024 : threads)), smem,
                 reinterpret_cast<cudaStream_t>(stream), index, int(M), int(L), int(warps),
                 plan_view(plan, M, L)) != cudaSuccess)
    return SPG_ERR_CUDA;
  return launch_status();
}

spg_status lora_f16(const void* X, int64_t ldx, const void* A, const void* B, const float* scale, const int32_t* plan,
                    void* V, int64_t ldv, const void* base, int64_t ldbase, void* Y, int64_t ldy, int64_t M, int64_t N,
                    int64_t K, int64_t R, int64_t L, spg_dtype dtype, spg_stream_t stream) {
  using namespace spg;
  using namespace spg::lora;
  spg_status rc = validate(X, ldx, A, B, scale, plan, V, ldv, M, N, K, R, L, dtype);
  if (rc != SPG_OK) return rc;
  if (ldy < N || (base && ldbase < N) || (M != 0 && !Y) || (base == Y && base && ldbase != ldy))
    return SPG_ERR_INVALID_ARG;
  if (M == 0) return SPG_OK;
  if (!mat_ok(Y, ldy) || (base && !mat_ok(base, ldbase))) return SPG_ERR_MISALIGNED;
  rc = check_device();
  if (rc != SPG_OK) return rc;
  uint32_t* err = device_error_word();
  if (!err) return SPG_ERR_CUDA;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  const Plan p = plan_view(plan, M, L);
  return dtype == SPG_BF16
             ? forward<true>(X, ldx, A, B, scale, p, V, ldv, base, ldbase, Y, ldy, M, N, K, R, L, err, st)
             : forward<false>(X, ldx, A, B, scale, p, V, ldv, base, ldbase, Y, ldy, M, N, K, R, L, err, st);
}

size_t lora_bwd_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R, int64_t L) {
  (void)N;
  (void)K;
  (void)L;
  return M > 0 && R > 0 ? (size_t(M) * size_t(R) * 2 + 255) / 256 * 256 : 0;
}

spg_status lora_f16_bwd(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* V, int64_t ldv,
                        const void* A, const void* B, const float* scale, const int32_t* plan, const void* dbase,
                        int64_t lddbase, void* dX, int64_t lddx, void* dA, void* dB, void* workspace, size_t ws_bytes,
                        int64_t M, int64_t N, int64_t K, int64_t R, int64_t L, spg_dtype dtype, spg_stream_t stream) {
  using namespace spg;
  using namespace spg::lora;
  spg_status rc = validate(X, ldx, A, B, scale, plan, V, ldv, M, N, K, R, L, dtype);
  if (rc != SPG_OK) return rc;
  if (lddy < N || !dA || !dB || (dX && lddx < K) || (dX && dbase && lddbase < K) ||
      (dX && dX == dbase && lddx != lddbase))
    return SPG_ERR_INVALID_ARG;
  if (!aligned(dA, 16) || !aligned(dB, 16)) return SPG_ERR_MISALIGNED;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // no rows: the sums over them are zero
    rc = check_device();
    if (rc != SPG_OK) return rc;
    if (cudaMemsetAsync(dA, 0, size_t(L) * R * K * 2, st) != cudaSuccess ||
        cudaMemsetAsync(dB, 0, size_t(L) * N * R * 2, st) != cudaSuccess)
      return SPG_ERR_CUDA;
    return SPG_OK;
  }
  if (!dY || !workspace || ws_bytes < lora_bwd_workspace_size(M, N, K, R, L)) return SPG_ERR_INVALID_ARG;
  if (!mat_ok(dY, lddy) || (dX && !mat_ok(dX, lddx)) || (dX && dbase && !mat_ok(dbase, lddbase)) ||
      !aligned(workspace, 16))
    return SPG_ERR_MISALIGNED;
  rc = check_device();
  if (rc != SPG_OK) return rc;
  uint32_t* err = device_error_word();
  if (!err) return SPG_ERR_CUDA;
  const Plan p = plan_view(plan, M, L);
  return dtype == SPG_BF16 ? backward<true>(dY, lddy, X, ldx, V, ldv, A, B, scale, p, dbase, lddbase, dX, lddx, dA, dB,
                                            workspace, M, N, K, R, L, err, st)
                           : backward<false>(dY, lddy, X, ldx, V, ldv, A, B, scale, p, dbase, lddbase, dX, lddx, dA,
                                             dB, workspace, M, N, K, R, L, err, st);
}

}  // extern "C"
