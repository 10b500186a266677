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
  uint64_t* more;  // eight further barriers (expand_kernel)
  uint32_t* tmem;
  volatile int* abort_flag;
};
constexpr int kMaxStages = 8;
constexpr int kBarBytes = (2 * kMaxStages + 9) * 8 + 16;

__device__ __forceinline__ Ring ring_at(uint8_t* p) {
  Ring r;
  r.full = reinterpret_cast<uint64_t*>(p);
  r.empty = r.full + kMaxStages;
  r.done = r.empty + kMaxStages;
  r.more = r.done + 1;
  r.tmem = reinterpret_cast<uint32_t*>(r.more + 8);
  r.abort_flag = reinterpret_cast<volatile int*>(r.tmem + 1);
  return r;
}

// `readers` arrivals free a stage; `more`: arrivals of the further barriers.
__device__ __forceinline__ void ring_init(const Ring& r, uint32_t tmem_cols, int warp, int readers = 1,
                                          const int* more = nullptr) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&r.full[s], 1);
      mbar_init(&r.empty[s], readers);
    }
    mbar_init(r.done, 1);
    for (int i = 0; more && i < 8; ++i) mbar_init(&r.more[i], more[i]);
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

// The rows of a tile as a producer warp loads them, 32 at a time.  Consecutive
// rows of the matrix (requests come as runs of rows) move as one box; others
// are gathered four by four, which TMA does at about half the rate (shrink of
// dY [8192, 16384] 118 us by gathers alone, 83 us with boxes).
struct TileRows {
  int4 rows;      // lane: positions 4 lane .. 4 lane + 3; a row past the matrix (zeros) past the end
  unsigned runs;  // bit g: rows 32 g .. are consecutive
  int count;
};

__device__ __forceinline__ TileRows tile_rows(const int* perm, int pos, int count, int lane, int M) {
  TileRows t;
  const int j = 4 * lane, first = j & ~31;
  t.count = count;
  t.rows.x = j + 0 < count ? perm[pos + j + 0] : M;
  t.rows.y = j + 1 < count ? perm[pos + j + 1] : M;
  t.rows.z = j + 2 < count ? perm[pos + j + 2] : M;
  t.rows.w = j + 3 < count ? perm[pos + j + 3] : M;
  const int want = __shfl_sync(0xffffffffu, t.rows.x, lane & ~7) + j - first;
  const bool run = (j + 0 >= count || t.rows.x == want) && (j + 1 >= count || t.rows.y == want + 1) &&
                   (j + 2 >= count || t.rows.z == want + 2) && (j + 3 >= count || t.rows.w == want + 3);
  const unsigned lanes = __ballot_sync(0xffffffffu, run);
  t.runs = 0;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int n = count - 32 * g;
    // ZERO-filled ends and short groups are gathered: a box would read past them
    if (((lanes >> (8 * g)) & 0xFFu) == 0xFFu && n > 0) t.runs |= 1u << g;
  }
  return t;
}

// Loads 64 columns from x of the tile's rows (32 groups of `rowb` bytes a row)
// to dst.  exact: only the tile's rows may be read as anything but zeros, as
// where the row is summed over.  Returns the bytes to expect, the same on
// every lane; `issue` false only counts.
template <bool EXACT>
__device__ __forceinline__ bool as_box(const TileRows& t, int g) {
  const int n = t.count - 32 * g;
  return (t.runs >> g & 1u) && (EXACT ? n >= 32 : n > 16);
}
template <bool EXACT>
__device__ __forceinline__ uint32_t rows_bytes(const TileRows& t, int groups, uint32_t rowb) {
  uint32_t b = 0;
  for (int g = 0; g < groups; ++g) {
    const int n = t.count - 32 * g;
    if (as_box<EXACT>(t, g)) b += 32 * rowb;
    else if (EXACT) b += 32 * rowb;
    else if (n > 0) b += uint32_t((n < 32 ? n + 3 : 32) / 4) * 4 * rowb;
  }
  return b;
}
template <bool EXACT>
__device__ __forceinline__ void rows_load(const TileRows& t, int groups, uint32_t rowb, uint8_t* dst,
                                          const CUtensorMap* box, const CUtensorMap* one, int x, uint64_t* bar,
                                          int lane) {
  const int g = lane >> 3;
  const int n = t.count - 32 * g;
  if (g < groups) {
    if (as_box<EXACT>(t, g)) {
      if ((lane & 7) == 0) tma_load_2d(dst + g * 32 * rowb, box, x, t.rows.x, bar);
    } else if (EXACT || 4 * (lane & 7) < n) {
      tma_gather4(dst + lane * 4 * rowb, one, x, t.rows, bar);
    }
  }
}

// Layout of a K-major operand whose rows hold R elements: rows of 32, 64 or
// 128 bytes (two tiles of 128 where R > 64), swizzled over their own width.
__host__ __device__ inline int row_bytes_of(int R) { return R <= 16 ? 32 : R <= 32 ? 64 : 128; }
__device__ __forceinline__ uint64_t desc_rows(const void* p, int rowb, uint32_t next) {
  return smem_desc(smem_addr(p), next, 8 * rowb, rowb == 32 ? LAYOUT_SW32 : rowb == 64 ? LAYOUT_SW64 : LAYOUT_SW128);
}

// ---- shrink: P [rows][R] = T [rows][D] . G^T ----------------------------------------
// One cluster a tile; its blocks split D in steps of 64, accumulate their
// parts in tensor memory and add them through distributed shared memory in
// the order of the ranks.  Warp 0 gathers T rows and loads G, one thread of
// warp 1 issues the MMAs, all four warps read the accumulators.
//   GMN false: G = A_l [R][D], a box of R rows of 64 columns, K-major
//   GMN true:  G = B_l [D][R], a box of 64 rows (two where R > 64), N-major
struct ShrinkArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  void* P;
  int64_t ldp;
  int M, D, R, stages, gbytes, rowb;
  uint32_t* err;
};

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(128) shrink_kernel(const __grid_constant__ CUtensorMap tmT,
                                                     const __grid_constant__ CUtensorMap tmT1,
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
    const TileRows rows = tile_rows(a.plan.perm, pos, count, lane, a.M);
    const uint32_t tx = rows_bytes<false>(rows, 4, 128) + a.gbytes;
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % a.stages;
      const uint32_t use = i / a.stages;
      if (use > 0 && !mbar_wait_warp(&ring.empty[s], (use - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      const int k = (kb0 + i) * 64;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], tx);
      __syncwarp();
      rows_load<false>(rows, 4, 128, st, &tmT, &tmT1, k, &ring.full[s], lane);
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
        const uint64_t bd = GMN ? desc_rows(st + kTile * 128, a.rowb, 8192) : desc_k_major(st + kTile * 128);
        const int bstep = (GMN ? 16 * a.rowb : 32) >> 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma(tmem, ad + ((32 * k) >> 4), bd + k * bstep, idesc, (i | k) != 0);
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
// A block of work is a tile and 128 columns; each SM's block takes an equal,
// consecutive share of them all and keeps the loads of the next ones under
// way (one block a tile and 128 columns, started anew each time, took 165 us
// for [8192, 16384] where this one's traffic takes 82).
//   warp 0    producer: base and G of the next blocks into the ring, P of the
//             next tile into one of two slots
//   warp 1    MMAs (one thread), tensor memory
//   warps 2-9 two a quarter of the rows, 64 columns each: accumulator + base
//             from the ring, rounded in place and stored from there (a box
//             where the rows are consecutive, else coalesced stores)
//   GMN false: G = B_l [C][R];  GMN true: G = A_l [R][C]
struct ExpandArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  const void* base;    // nullptr: 0
  void* Y;
  int64_t ldb, ldy;
  int M, C, R, stages, rowb, pbytes, gbytes;
  uint32_t* err;
};

constexpr int kExpCols = 128;
constexpr int kExpThreads = 320;
constexpr int kYBytes = kTile * kExpCols * 2;

// The consecutive share of the blocks of work that this thread block takes,
// one by one: column block nb of tile `tile`.
struct Share {
  int left, tile, nb, nblk;
  bool fresh;  // the first block of its tile here
  __device__ Share(int tiles, int nblk_) : nblk(nblk_), fresh(true) {
    const int64_t total = int64_t(tiles) * nblk_;
    const int64_t w = total * blockIdx.x / gridDim.x;
    left = int(total * (blockIdx.x + 1) / gridDim.x - w);
    tile = int(w / nblk_);
    nb = int(w - int64_t(tile) * nblk_);
  }
  __device__ bool more() const { return left > 0; }
  __device__ bool last_of_tile() const { return left == 1 || nb + 1 == nblk; }
  __device__ void next() {
    --left;
    fresh = false;
    if (++nb == nblk) {
      nb = 0;
      ++tile;
      fresh = true;
    }
  }
};

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(kExpThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmG,
                  const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB1,
                  const __grid_constant__ CUtensorMap tmY, const ExpandArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stage_bytes = kYBytes + a.gbytes;
  uint8_t* Ps = smem + a.stages * stage_bytes;  // two slots
  const Ring ring = ring_at(Ps + 2 * a.pbytes);
  uint64_t* acc_full = ring.more;       // two accumulators
  uint64_t* acc_empty = ring.more + 2;
  uint64_t* p_full = ring.more + 4;     // two slots of P
  uint64_t* p_empty = ring.more + 6;
  const int counts[8] = {1, 1, 8, 8, 1, 1, 1, 1};
  griddep_wait();
  ring_init(ring, 2 * kExpCols, warp, 8, counts);
  const uint32_t tmem = *ring.tmem;
  const int halves = a.R > 64 ? 2 : 1;
  const int Rn = round16(a.R);
  Share w(a.plan.hdr[0], (a.C + kExpCols - 1) / kExpCols);
  const bool has_base = a.base != nullptr;
  const bool in_place = a.base == a.Y;
  // Every role walks the same blocks: i counts those that are not skipped
  // (rows without an adapter whose base is already in place), p those tiles
  // that need a slot of P.
  if (warp == 0) {
    int i = 0, p = 0;
    int4 t = make_int4(-1, 0, 0, 0);
    TileRows rows;
    uint32_t bytes = 0;
    for (; w.more(); w.next()) {
      const int n0 = w.nb * kExpCols;
      if (w.fresh) {
        t = a.plan.tiles[w.tile];
        rows = tile_rows(a.plan.perm, t.y, t.z, lane, a.M);
        bytes = rows_bytes<false>(rows, 4, 128);
      }
      if (t.x < 0 && in_place) continue;
      if (w.fresh && t.x >= 0) {
        const int slot = p & 1;
        if (p >= 2 && !mbar_wait_warp(&p_empty[slot], ((p >> 1) - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
        const int fours = (t.z + 3) / 4;
        if (lane == 0) mbar_arrive_expect_tx(&p_full[slot], halves * fours * 4 * a.rowb);
        __syncwarp();
        for (int h = 0; h < halves; ++h)
          if (lane < fours)
            tma_gather4(Ps + slot * a.pbytes + h * kTile * a.rowb + lane * 4 * a.rowb, &tmP, 64 * h, rows.rows,
                        &p_full[slot]);
        ++p;
      }
      const int s = i % a.stages;
      const int use = i / a.stages;
      if (use > 0 && !mbar_wait_warp(&ring.empty[s], (use - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      const int subs = a.C - n0 > 64 ? 2 : 1;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], (has_base ? subs * bytes : 0u) + (t.x >= 0 ? a.gbytes : 0));
      __syncwarp();
      if (has_base)
        for (int j = 0; j < subs; ++j)
          rows_load<false>(rows, 4, 128, st + j * kTile * 128, &tmB, &tmB1, n0 + 64 * j, &ring.full[s], lane);
      if (t.x >= 0 && lane == 0) {
        uint8_t* g = st + kYBytes;
        if constexpr (GMN) {
          tma_load_3d(g, &tmG, n0, 0, t.x, &ring.full[s]);
          tma_load_3d(g + Rn * 128, &tmG, n0 + 64, 0, t.x, &ring.full[s]);
        } else {
          for (int h = 0; h < halves; ++h)
            tma_load_3d(g + h * kExpCols * a.rowb, &tmG, 64 * h, n0, t.x, &ring.full[s]);
        }
      }
      __syncwarp();
      ++i;
    }
    if (lane == 0) {  // nothing is in flight when the block ends
      for (int q = i > a.stages ? i - a.stages : 0; q < i; ++q)
        tail_wait(&ring.full[q % a.stages], (q / a.stages) & 1, a.err);
      for (int q = p > 2 ? p - 2 : 0; q < p; ++q) tail_wait(&p_full[q & 1], (q >> 1) & 1, a.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = instr_desc_major(BF16, kTile, kExpCols, 0, GMN ? 1 : 0);
      int i = 0, p = 0, adapter = -1;
      for (; w.more(); w.next()) {
        if (w.fresh) adapter = a.plan.tiles[w.tile].x;
        if (adapter < 0 && in_place) continue;
        if (w.fresh && adapter >= 0) {
          if (!mbar_wait(&p_full[p & 1], (p >> 1) & 1, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
          ++p;
        }
        const int s = i % a.stages, b = i & 1;
        if (!mbar_wait(&ring.full[s], (i / a.stages) & 1, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
        if (i >= 2 && !mbar_wait(&acc_empty[b], ((i >> 1) - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_ACC_FREE)) break;
        tc_fence_after();
        if (adapter >= 0) {
          const uint8_t* P = Ps + ((p - 1) & 1) * a.pbytes;
          const uint8_t* G = smem + s * stage_bytes + kYBytes;
          const int ksub = a.rowb / 32;  // MMA steps in a row of an operand tile
          for (int k = 0; k < Rn / 16; ++k) {
            const int h = k / ksub, kk = k - h * ksub;
            const uint64_t ad = desc_rows(P + h * kTile * a.rowb, a.rowb, 16) + ((32 * kk) >> 4);
            const uint64_t bd = GMN ? desc_mn_major(G + 2048 * k, Rn * 128)
                                    : desc_rows(G + h * kExpCols * a.rowb, a.rowb, 16) + ((32 * kk) >> 4);
            tc_mma(tmem + b * kExpCols, ad, bd, idesc, k != 0);
          }
          if (w.last_of_tile()) tc_commit(&p_empty[(p - 1) & 1]);
        }
        tc_commit(&acc_full[b]);
        ++i;
      }
      tc_commit(ring.done);
    }
    __syncwarp();
    tail_wait(ring.done, 0, a.err);
  } else {
    const int quad = warp & 3, sub = (warp - 2) >> 2;
    uint16_t* Y = static_cast<uint16_t*>(a.Y);
    int i = 0, pending = -1;
    int4 t = make_int4(-1, 0, 0, 0);
    int mine = 0;       // this lane's row
    bool run = false;   // the warp's 32 rows are consecutive, and all there
    int rows_here = 0;
    float scale = 0.f;
    for (; w.more(); w.next()) {
      const int n0 = w.nb * kExpCols + 64 * sub;
      if (w.fresh) {
        t = a.plan.tiles[w.tile];
        rows_here = t.z - 32 * quad;
        mine = lane < rows_here ? a.plan.perm[t.y + 32 * quad + lane] : 0;
        const int first = __shfl_sync(0xffffffffu, mine, 0);
        run = rows_here >= 32 && __all_sync(0xffffffffu, mine == first + lane);
        scale = t.x < 0 ? 0.f : a.scale ? a.scale[t.x] : 1.f;
      }
      if (t.x < 0 && in_place) continue;
      const int s = i % a.stages, b = i & 1;
      // the copied rows' own barrier, then the accumulator's
      bool ok = mbar_wait_warp(&ring.full[s], (i / a.stages) & 1, ring.abort_flag, a.err, ERR_WAIT_ACC);
      ok = ok && mbar_wait_warp(&acc_full[b], (i >> 1) & 1, ring.abort_flag, a.err, ERR_WAIT_ACC);
      if (!ok) break;
      tc_fence_after();
      const int cols = min(64, a.C - n0);
      uint8_t* buf = smem + s * stage_bytes + sub * kTile * 128 + quad * 32 * 128;
      bool boxed = false;
      if (rows_here > 0 && cols > 0) {
        uint8_t* row = buf + lane * 128;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t h[32];
          if (t.x >= 0) {
            tmem_ld_32x32b_x32(tmem + (uint32_t(32 * quad) << 16) + b * kExpCols + 64 * sub + c, h);
            tmem_ld_wait(h);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) h[e] = 0u;
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            // 16-byte piece v of the row's 64 columns, where the swizzle puts it
            uint4* at = reinterpret_cast<uint4*>(row + (((c / 8 + v) ^ (lane & 7)) << 4));
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (has_base) x = *at;
            uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
            if (t.x >= 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<BF16>(xw[e]);
                xw[e] = pack2<BF16>(fmaf(scale, __uint_as_float(h[8 * v + 2 * e]), f.x),
                                    fmaf(scale, __uint_as_float(h[8 * v + 2 * e + 1]), f.y));
              }
            }
            *at = x;
          }
        }
        boxed = run && cols == 64;
        if (boxed) {
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
      if (boxed) {
        if (lane == 0) {
          tma_store_2d_saddr(&tmY, smem_addr(buf), n0, mine);
          bulk_commit();
          // the stage of the store before this one, once that has left shared memory
          if (pending >= 0) {
            bulk_wait_read<1>();
            mbar_arrive(&ring.empty[pending]);
          }
        }
        pending = s;
      } else {
        if (rows_here > 0 && cols > 0) {
          // eight lanes a row, four rows at a time
          for (int r = 0; r < 32; r += 4) {
            const int rr = r + (lane >> 3), c = (lane & 7) * 8;
            const int64_t to = __shfl_sync(0xffffffffu, mine, rr);
            if (rr < rows_here && c < cols) {
              const uint4 x = *reinterpret_cast<const uint4*>(buf + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
              uint16_t* o = Y + to * a.ldy + n0 + c;
              if (c + 8 <= cols) {
                *reinterpret_cast<uint4*>(o) = x;
              } else {
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 7; ++e)
                  if (c + e < cols) o[e] = static_cast<uint16_t>(xw[e >> 1] >> (16 * (e & 1)));
              }
            }
          }
        }
        // generic reads of the stage come before the copies that refill it
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (pending >= 0) {
            bulk_wait_read<0>();
            mbar_arrive(&ring.empty[pending]);
          }
          mbar_arrive(&ring.empty[s]);
        }
        pending = -1;
      }
      ++i;
    }
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kExpCols);
  }
}

// ---- wgrad: dG_l [C][R] = s_l sum over l's rows of T[m][c] P[m][r] ----------------------
// One cluster a block of kWgCols columns of T and an adapter; its blocks split
// the adapter's rows in chunks of 64 and add their sums as shrink_kernel does.
// Both operands are read with the row as the MMA's K index.
//   OT false: dG is [C][R] (dB);  OT true: [R][C] (dA)
struct WgradArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  void* dG;
  int M, C, R, stages, rowb;
  uint32_t* err;
};

constexpr int kWgCols = 128;

template <bool BF16, bool OT>
__global__ void __launch_bounds__(128) wgrad_kernel(const __grid_constant__ CUtensorMap tmT,
                                                    const __grid_constant__ CUtensorMap tmT1,
                                                    const __grid_constant__ CUtensorMap tmP,
                                                    const __grid_constant__ CUtensorMap tmP1, const WgradArgs a) {
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
  const int pbytes = 64 * a.rowb;
  const int stage_bytes = tbytes + halves * pbytes;
  const int part_bytes = kWgCols * (R + 4) * 4;
  const int ring_bytes = a.stages * stage_bytes;
  const Ring ring = ring_at(smem + (ring_bytes > part_bytes ? ring_bytes : part_bytes));
  const uint32_t tcols = tmem_cols(Rn);
  ring_init(ring, tcols, warp);
  const uint32_t tmem = *ring.tmem;
  const int chunks = (rows + 63) / 64;
  const int q0 = int(int64_t(chunks) * rank / cs), n = int(int64_t(chunks) * (rank + 1) / cs) - q0;

  if (warp == 0) {
    const uint32_t tx = subs * 8192 + halves * pbytes;
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % a.stages;
      const uint32_t use = i / a.stages;
      const int at = (q0 + i) * 64;
      const TileRows r = tile_rows(a.plan.perm, start + at, min(64, rows - at), lane, a.M);
      if (use > 0 && !mbar_wait_warp(&ring.empty[s], (use - 1) & 1, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], tx);
      __syncwarp();
      for (int j = 0; j < subs; ++j)
        rows_load<true>(r, 2, 128, st + j * 8192, &tmT, &tmT1, c0 + 64 * j, &ring.full[s], lane);
      for (int h = 0; h < halves; ++h)
        rows_load<true>(r, 2, a.rowb, st + tbytes + h * pbytes, &tmP, &tmP1, 64 * h, &ring.full[s], lane);
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
        const uint64_t ad = desc_mn_major(st, 8192), bd = desc_rows(st + tbytes, a.rowb, pbytes);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma(tmem, ad + ((2048 * k) >> 4), bd + ((16 * a.rowb * k) >> 4), idesc, (i | k) != 0);
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
template <class K>
spg_status prepare(K kern, int smem) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess ? SPG_OK
                                                                                                      : SPG_ERR_CUDA;
}

// Rows of a matrix: boxes of 32 rows, and single rows for gathers, of `rowb` bytes.
bool rows_maps(CUtensorMap* box, CUtensorMap* one, const void* p, int64_t cols, int64_t rows, int64_t ld, int rowb) {
  return make_tmap_2d_swz(box, p, 2, uint64_t(cols), uint64_t(rows), uint64_t(ld) * 2, rowb / 2, 32, rowb) &&
         make_tmap_2d_swz(one, p, 2, uint64_t(cols), uint64_t(rows), uint64_t(ld) * 2, rowb / 2, 1, rowb);
}

constexpr int kRingBudget = 100 * 1024;  // shared memory of a ring where two blocks share an SM

template <bool BF16, bool GMN>
spg_status shrink(const void* T, int64_t ldt, const void* G, const float* scale, const Plan& plan, void* P, int64_t ldp,
                  int64_t M, int64_t D, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  const int Rn = round16(int(R)), rowb = row_bytes_of(int(R));
  CUtensorMap tmT, tmT1, tmG;
  if (!rows_maps(&tmT, &tmT1, T, D, M, ldt, 128)) return SPG_ERR_CUDA;
  if (!(GMN ? make_tmap_3d(&tmG, G, R, D, L, 64, rowb) : make_tmap_3d(&tmG, G, D, R, L, Rn, 128))) return SPG_ERR_CUDA;
  const int gbytes = GMN ? 64 * rowb * (R > 64 ? 2 : 1) : Rn * 128;
  const int stage = kTile * 128 + gbytes;
  int stages = kRingBudget / stage;
  stages = stages > kMaxStages ? kMaxStages : stages;
  // blocks of a cluster: as many as let every tile of full groups be resident
  // at once (two blocks an SM), each with at least two steps of its own
  const int64_t tiles = max_tiles(M, L), nkb = (D + 63) / 64;
  const int64_t busy = (M + kTile - 1) / kTile;
  int cs = 1;
  while (cs < 8 && busy * 2 * cs <= 2 * sm_count() && nkb >= 4 * cs) cs *= 2;
  const int ring = stages * stage, part = kTile * (int(R) + 4) * 4;
  const int smem = (ring > part ? ring : part) + kBarBytes + 1024;
  if (part > ring) return SPG_ERR_UNSUPPORTED_SHAPE;
  auto kern = shrink_kernel<BF16, GMN>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const ShrinkArgs a{plan, scale, P, ldp, int(M), int(D), int(R), stages, gbytes, rowb, err};
  return launch_pdl_cluster(kern, dim3(unsigned(tiles * cs)), dim3(128), smem, cs, st, tmT, tmT1, tmG, a) ==
                 cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

template <bool BF16, bool GMN>
spg_status expand(const void* P, int64_t ldp, const void* G, const float* scale, const Plan& plan, const void* base,
                  int64_t ldb, void* Y, int64_t ldy, int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err,
                  cudaStream_t st) {
  const int Rn = round16(int(R)), halves = R > 64 ? 2 : 1, rowb = row_bytes_of(int(R));
  CUtensorMap tmP, tmP32, tmG, tmB, tmB1, tmY, tmY1;
  if (!rows_maps(&tmP32, &tmP, P, R, M, ldp, rowb) || !rows_maps(&tmY, &tmY1, Y, C, M, ldy, 128) ||
      !rows_maps(&tmB, &tmB1, base ? base : Y, C, M, base ? ldb : ldy, 128))
    return SPG_ERR_CUDA;
  if (!(GMN ? make_tmap_3d(&tmG, G, C, R, L, Rn, 128) : make_tmap_3d(&tmG, G, R, C, L, kExpCols, rowb)))
    return SPG_ERR_CUDA;
  const int pbytes = halves * kTile * rowb;
  const int gbytes = GMN ? 2 * Rn * 128 : halves * kExpCols * rowb;
  const int fixed = 2 * pbytes + kBarBytes + 1024;
  int stages = (232448 - fixed) / (kYBytes + gbytes);
  stages = stages > kMaxStages ? kMaxStages : stages;
  const int smem = stages * (kYBytes + gbytes) + fixed;
  auto kern = expand_kernel<BF16, GMN>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const ExpandArgs a{plan, scale, base, Y, ldb, ldy, int(M), int(C), int(R), stages, rowb, pbytes, gbytes, err};
  const int64_t work = max_tiles(M, L) * ((C + kExpCols - 1) / kExpCols);
  const int64_t blocks = work < sm_count() ? work : sm_count();
  return launch_pdl(kern, dim3(unsigned(blocks)), dim3(kExpThreads), smem, st, tmP, tmG, tmB, tmB1, tmY, a) ==
                 cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

template <bool BF16, bool OT>
spg_status wgrad(const void* T, int64_t ldt, const void* P, int64_t ldp, const float* scale, const Plan& plan, void* dG,
                 int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  const int rowb = row_bytes_of(int(R));
  CUtensorMap tmT, tmT1, tmP, tmP1;
  if (!rows_maps(&tmT, &tmT1, T, C, M, ldt, 128) || !rows_maps(&tmP, &tmP1, P, R, M, ldp, rowb)) return SPG_ERR_CUDA;
  const int stage = (kWgCols / 64) * 8192 + (R > 64 ? 2 : 1) * 64 * rowb;
  int stages = kRingBudget / stage;
  stages = stages > kMaxStages ? kMaxStages : stages;
  const int64_t blocks = (C + kWgCols - 1) / kWgCols;
  const int64_t groups = L < 4 ? L : 4;
  int cs = 1;
  while (cs < 8 && blocks * groups * cs < 4 * sm_count() && M / groups >= 256 * cs) cs *= 2;
  const int ring = stages * stage, part = kWgCols * (int(R) + 4) * 4;
  const int smem = (ring > part ? ring : part) + kBarBytes + 1024;
  auto kern = wgrad_kernel<BF16, OT>;
  if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const WgradArgs a{plan, scale, dG, int(M), int(C), int(R), stages, rowb, err};
  return launch_pdl_cluster(kern, dim3(unsigned(blocks * cs), unsigned(L)), dim3(128), smem, cs, st, tmT, tmT1, tmP,
                            tmP1, a) == cudaSuccess
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
