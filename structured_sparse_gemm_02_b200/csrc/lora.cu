// Low-rank adapters of many requests beside one shared (pruned) projection,
// forward and backward.  Row m uses adapter l = index[m], or none:
//
//   v = x A_l^T,  y = base + s_l v B_l^T              (A_l [R, K], B_l [N, R])
//   u = s_l dy B_l,  dx = dbase + u A_l
//   dA_l = sum over l's rows of u^T x,  dB_l = s_l sum over l's rows of dy^T v
//
// A plan (one small kernel per batch) groups the rows by adapter; every product
// then runs on tiles of up to 128 rows of one adapter, whose rows TMA gathers
// by index.  Three kinds of kernels cover all products:
//   shrink  P = T G^T for T = X (G = A_l) or T = dY (G = B_l^T): tcgen05
//   expand  Y = base + s P G^T for G = B_l or G = A_l^T: mma.sync up to R = 32
//           and for few rows, tcgen05 beyond
//   wgrad   dG = s T^T P for (X, U) and (dY, V): tcgen05
// The two that read dY run as one launch.
// R is at most 128, so each of them is bound by the reads and writes of its
// large matrix.  V and U are rounded to the activations' type between the
// products: V is saved for the backward pass as any activation is, and both
// are operands of the tensor cores; every sum is fp32.  Against 64 bits that
// leaves Y where it is with V in fp32 (bf16, R = 64: 1.6e-3 relative, the
// rounding of Y itself) and takes dX and dA from 1.7e-3 to 2.3e-3 (fp16
// 2.1e-4 to 2.9e-4); U as a high and a low half would undo it, for twice the
// operands of wgrad and expand.
//
// A block of a cluster may wait for tensor memory while another block of it
// holds some, so such blocks, of several streams too, must never use up an SM's
// tensor memory between them: those of shrink, wgrad and dual take at least
// kSmemPerColumn bytes of shared memory for each column.  Beside a block of the
// pruned layers' kernels, which take nearly all of an SM's, none fits.  Blocks of
// the expand kernels wait for no other block.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "gather.cuh"
#include "host.cuh"
#include "sm100.cuh"
#include "spgemm.h"

namespace spg {
namespace lora {

constexpr int kTile = 128;  // rows of a tile: the M of one MMA
constexpr int kMaxL = 8192;
constexpr int kMaxR = 128;
constexpr int64_t kMaxPitch = int64_t(1) << 31;  // pitches in bytes fit 32 bits

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
// depend on timing.  The kernel may start before the one that writes `index`
// has ended, so index is not read as data that never changes (no __restrict__).
// Bound by latency: 8192 rows 5.4 us, 64 rows 2.4 us.
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* index, int M, int L, int warps, Plan p) {
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
  const int r0 = warp * strip, r1 = warp < warps ? min(M, r0 + strip) : r0;
  // the group of a row, -1 past the strip; the first kHeld steps of a strip are
  // read once, all at the same time
  constexpr int kHeld = 8;
  auto group_at = [&](int row) {
    if (row >= r1) return -1;
    const int a = index[row];
    return a < 0 || a >= L ? L : a;
  };
  int held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = group_at(r0 + 32 * k + lane);
  auto count = [&](int a) {
    const unsigned same = __match_any_sync(0xffffffffu, a);
    if (a >= 0 && lane == __ffs(same) - 1) cnt[warp * G + a] += __popc(same);
    __syncwarp();
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (r0 + 32 * k < r1) count(held[k]);
  for (int r = r0 + 32 * kHeld; r < r1; r += 32) count(group_at(r + lane));
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
  auto place = [&](int row, int a) {
    const unsigned same = __match_any_sync(0xffffffffu, a);
    int at = 0;
    if (a >= 0) at = cnt[warp * G + a];
    __syncwarp();
    if (a >= 0) {
      p.perm[at + __popc(same & ((1u << lane) - 1))] = row;
      if (lane == __ffs(same) - 1) cnt[warp * G + a] = at + __popc(same);
    }
    __syncwarp();
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (r0 + 32 * k < r1) place(r0 + 32 * k + lane, held[k]);
  for (int r = r0 + 32 * kHeld; r < r1; r += 32) place(r + lane, group_at(r + lane));
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
  uint32_t* tmem;
  volatile int* abort_flag;
};
// A role's place in a ring of n: slot and the parity of its use of the slot
// (kept, as a division a step costs a single thread more than the step).  A
// fresh barrier passes a wait for parity 1.
struct Turn {
  int n, s = 0;
  uint32_t ph = 0;
  __device__ explicit Turn(int n_) : n(n_) {}
  __device__ __forceinline__ void next() {
    if (++s == n) {
      s = 0;
      ph ^= 1u;
    }
  }
};
constexpr int kMaxStages = 8;
constexpr int kBarBytes = (2 * kMaxStages + 1) * 8 + 8;

__device__ __forceinline__ Ring ring_at(uint8_t* p) {
  Ring r;
  r.full = reinterpret_cast<uint64_t*>(p);
  r.empty = r.full + kMaxStages;
  r.done = r.empty + kMaxStages;
  r.tmem = reinterpret_cast<uint32_t*>(r.done + 1);
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
  // Only now: a dependent kernel takes its tensor memory before it waits for this
  // one, and must not get ahead of a block of this one that still needs its own.
  griddep_launch_dependents();
}

__host__ __device__ inline int round16(int r) { return (r + 15) & ~15; }
// Tensor-memory columns for n accumulator columns: a power of two, at least 32.
__host__ __device__ inline uint32_t tmem_cols(int n) { return n <= 32 ? 32u : n <= 64 ? 64u : 128u; }
constexpr int kSmemPerColumn = 228 * 1024 / 512;  // of an SM, for 512 columns
// Shared memory of a block with `bytes` of ring or sums and n accumulator columns.
__host__ inline int block_smem(int bytes, int n) {
  const int all = bytes + kBarBytes + 1024, least = int(tmem_cols(n)) * kSmemPerColumn;
  return all > least ? all : least;
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

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
// are gathered four by four, which takes TMA longer (shrink of [8192, 4096], rank
// 16: rows in runs 20 us, in no order 29 us).
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

// `rowb` bytes of each of the tile's rows, in `groups` groups of 32 rows, from
// column x to dst.  EXACT: only the tile's rows may be read as anything but
// zeros, as where the row is summed over.  rows_bytes: the bytes to expect, the
// same on every lane.
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
// warp 1 issues the MMAs, all four warps read the accumulators.  Bound by the
// reading of T: [8192, 4096], rank 16 20 us, [8192, 16384] 51 us (5.3 TB/s).
//   GMN false: G = A_l [R][D], a box of R rows of 64 columns, K-major
//   GMN true:  G = B_l [D][R], a box of 64 rows (two where R > 64), N-major
struct ShrinkArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  void* P;
  int64_t ldp;
  int M, D, R, stages, trows, gbytes, rowb;
  uint32_t* err;
};

// Bytes of a shrink's ring: its last stage is read as a whole tile.
__host__ __device__ inline int ring_of(int stages, int stage) {
  return stages * stage + (stage < kTile * 128 ? kTile * 128 - stage : 0);
}

template <bool BF16, bool GMN>
__device__ __forceinline__ void shrink_body(uint8_t* smem, const CUtensorMap& tmT, const CUtensorMap& tmT1,
                                            const CUtensorMap& tmG, const ShrinkArgs& a, int tile) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cs = cluster_nctarank(), rank = cluster_ctarank();
  const int R = a.R, vecs = R / 8;
  const int Rn = round16(R);
  // A tile has at most a.trows rows (M, where that is less than a whole tile); the
  // MMA reads 128, the others from whatever follows, and nobody reads their sums
  const int tbytes = a.trows * 128, stage_bytes = tbytes + a.gbytes;
  const int ring_bytes = ring_of(a.stages, stage_bytes), part_bytes = kTile * (R + 4) * 4;
  const Ring ring = ring_at(smem + (ring_bytes > part_bytes ? ring_bytes : part_bytes));
  ring_init(ring, tmem_cols(Rn), warp);
  const uint32_t tmem = *ring.tmem;
  griddep_wait();
  const int4 t = tile < a.plan.hdr[0] ? a.plan.tiles[tile] : make_int4(-1, 0, 0, 0);
  const int adapter = t.x, pos = t.y, count = t.z;
  uint16_t* P = static_cast<uint16_t*>(a.P);
  if (adapter < 0) {  // rows without an adapter: zeros; past the last tile: nothing
    if (warp == 1) tmem_dealloc(tmem, tmem_cols(Rn));
    if (rank == 0)
      for (int i = threadIdx.x; i < count * vecs; i += blockDim.x)
        *reinterpret_cast<uint4*>(P + int64_t(a.plan.perm[pos + i / vecs]) * a.ldp + (i % vecs) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int nkb = (a.D + 63) / 64;
  const int kb0 = int(int64_t(nkb) * rank / cs), n = int(int64_t(nkb) * (rank + 1) / cs) - kb0;

  if (warp == 0) {
    const TileRows rows = tile_rows(a.plan.perm, pos, count, lane, a.M);
    const uint32_t tx = rows_bytes<false>(rows, 4, 128) + a.gbytes;
    int i = 0;
    for (Turn r(a.stages); i < n; ++i, r.next()) {
      const int s = r.s;
      if (!mbar_wait_warp(&ring.empty[s], r.ph ^ 1u, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
      uint8_t* st = smem + s * stage_bytes;
      const int k = (kb0 + i) * 64;
      if (lane == 0) mbar_arrive_expect_tx(&ring.full[s], tx);
      __syncwarp();
      rows_load<false>(rows, 4, 128, st, &tmT, &tmT1, k, &ring.full[s], lane);
      if (lane == 0) {
        if constexpr (GMN) {
          tma_load_3d(st + tbytes, &tmG, 0, k, adapter, &ring.full[s]);
          if (R > 64) tma_load_3d(st + tbytes + 8192, &tmG, 64, k, adapter, &ring.full[s]);
        } else {
          tma_load_3d(st + tbytes, &tmG, k, 0, adapter, &ring.full[s]);
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
      const uint64_t ad0 = desc_k_major(smem);
      const uint64_t bd0 = GMN ? desc_rows(smem + tbytes, a.rowb, 8192) : desc_k_major(smem + tbytes);
      const int bstep = (GMN ? 16 * a.rowb : 32) >> 4;
      Turn r(a.stages);
      for (int i = 0; i < n; ++i, r.next()) {
        if (!mbar_wait(&ring.full[r.s], r.ph, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
        tc_fence_after();
        const uint64_t ad = ad0 + ((r.s * stage_bytes) >> 4), bd = bd0 + ((r.s * stage_bytes) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc_mma(tmem, ad + ((32 * k) >> 4), bd + k * bstep, idesc, (i | k) != 0);
        tc_commit(&ring.empty[r.s]);
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

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(128) shrink_kernel(const __grid_constant__ CUtensorMap tmT,
                                                     const __grid_constant__ CUtensorMap tmT1,
                                                     const __grid_constant__ CUtensorMap tmG, const ShrinkArgs a) {
  extern __shared__ uint8_t smem_raw[];
  shrink_body<BF16, GMN>(align1024(smem_raw), tmT, tmT1, tmG, a, blockIdx.x / cluster_nctarank());
}

// ---- expand in registers ------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight 16-bit columns from c of a row of C, those past its end 0 (or unwritten).
__device__ __forceinline__ uint4 load_cols8(const uint16_t* row, int c, int C) {
  if (c + 8 <= C) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (c + e < C) w[e >> 1] |= static_cast<uint32_t>(row[c + e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_cols8(uint16_t* row, int c, int C, const uint4& v) {
  if (c + 8 <= C) {
    *reinterpret_cast<uint4*>(row + c) = v;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (c + e < C) row[c + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
  }
}

constexpr int kRegCols = 64;  // columns of a warp
// Warps of a block: `RG` (1 or 4) take the tile's groups of 32 rows between
// them, 4 / 2 blocks of columns side by side.
template <int RG>
struct RegShape {
  static constexpr int CG = RG == 1 ? 4 : 2;
  static constexpr int WARPS = RG * CG;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int COLS = CG * kRegCols;
  static constexpr int PITCH = COLS * 2 + 16;  // bytes of a staged row of G
  static constexpr int STAGES = RG == 1 ? 2 : 1;
  static constexpr int BASE = WARPS * (STAGES * 4096 + kTile * 4);
};

struct ExpandRegArgs {
  Plan plan;
  const float* scale;  // nullptr: 1
  const uint16_t* P;
  const uint16_t* G;
  const uint16_t* base;  // nullptr: 0
  uint16_t* Y;
  uint32_t pitch_p, pitch_b, pitch_y;  // bytes
  int C, R;
};
// Row `row` of a matrix; with a 32-bit pitch that is one instruction.
template <class T>
__device__ __forceinline__ T* row_at(T* p, int row, uint32_t pitch) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + uint64_t(uint32_t(row)) * pitch);
}

// The k index of an MMA step may be dealt to lanes in any order that both
// operands share, and so may its n index: lane t of a quad takes 4 consecutive
// k of a step (8 of a pair of steps), one load a row, and n-tile j of 32
// columns holds columns 8 t + 2 j and the next, so that a lane ends up with 8
// consecutive columns of a row: one 16-byte piece of base and one store.
// What bounds the kernel is the number of bytes under way: each warp copies its
// own columns of base to shared memory two groups of 32 rows ahead of the sums
// ([8192, 16384], R = 16: 91 us, 5.9 TB/s; base read into registers a group ahead
// 112 us; three groups ahead and as many blocks an SM as fit 98 us).
// Where adapters have few rows, what is read is mostly G: a warp then walks along
// the columns (WALK), and reads G and base of the next ones behind the sums.
//   KS: steps of 16 with G in registers (1 or 2); 0: any number, read per 32 rows
template <bool BF16, bool GMN, int KS, int RG, bool WALK>
__global__ void __launch_bounds__(RegShape<RG>::THREADS, RG == 4 ? 2 : KS == 1 ? 4 : 3)
    expand_reg_kernel(const ExpandRegArgs a) {
  using Sh = RegShape<RG>;
  constexpr int kStages = Sh::STAGES;
  constexpr bool kFew = WALK || KS == 0;  // most groups are short: what has no row is left out
  extern __shared__ __align__(128) uint8_t gsm[];
  const int warp = (threadIdx.x >> 5) % Sh::CG, lane = threadIdx.x & 31;
  const int first = 32 * ((threadIdx.x >> 5) / Sh::CG);  // this warp's first rows of the tile
  const int g = lane >> 2, q = lane & 3;
  uint8_t* mine = gsm + (threadIdx.x >> 5) * kStages * 4096;
  int* rowid = reinterpret_cast<int*>(gsm + Sh::WARPS * kStages * 4096) + (threadIdx.x >> 5) * kTile;
  uint8_t* gst = gsm + Sh::BASE;
  griddep_launch_dependents();
  griddep_wait();
  const int4 t = a.plan.tiles[blockIdx.y];
  if (int(blockIdx.y) >= a.plan.hdr[0]) return;
  const int adapter = t.x, pos = t.y, count = t.z;
  if (adapter < 0 && a.base == a.Y) return;
  const int nb = blockIdx.x * Sh::COLS;
  int n0 = nb + warp * kRegCols;
  const bool busy = n0 < a.C && first < count;
  // from a group of 32 rows to the next, and to the next columns behind the last
  auto advance = [&](int& n, int& r0) {
    r0 += 32 * RG;
    if constexpr (WALK) {
      if (r0 >= count) {
        const int stride = gridDim.x * Sh::COLS;
        r0 = first;
        n = a.C - n > stride ? n + stride : a.C;
      }
    }
  };
  // rows of base, 128 bytes each; the halves of odd rows change places, so that
  // eight lanes reading two rows' halves meet no bank twice
  int nf = n0, rf = first;  // what is copied next
  auto copy = [&](int s) {
    if (a.base && rf < count && nf < a.C) {
      const int v = lane & 7, r1 = lane >> 3, r0 = rf;
      const int in = 2 * min(8, max(0, a.C - (nf + 8 * v)));  // bytes inside the row
      const uint16_t* from = a.base + (in ? nf + 8 * v : 0);
      uint8_t* to = mine + s * 4096 + r1 * 128 + ((v ^ ((r1 & 1) << 2)) << 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (kFew && r0 + 4 * i >= count) break;
        const bool ok = r0 + 4 * i + r1 < count;
        cp_async16(to + 512 * i, row_at(from, ok ? rowid[r0 + 4 * i + r1] : rowid[r0], a.pitch_b), ok ? in : 0);
      }
    }
    cp_async_commit();
    advance(nf, rf);
  };
  constexpr int S = KS == 1 ? 1 : 2;  // steps of a fragment
  const uint16_t* G = a.G + int64_t(adapter < 0 ? 0 : adapter) * a.C * a.R;
  // fragments of G for step pair kb (KS == 1: the one step) and half h: b[j][step][2]
  auto load_b = [&](int c, int kb, int h, uint32_t (&b)[4][S][2]) {  // columns from c
    if constexpr (GMN) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          // matrices: k rows 0-7 and 8-15 of tile j, then of tile j + 1
          const uint32_t at = smem_addr(gst + (kb * 32 + s * 16 + (lane & 15)) * Sh::PITCH +
                                        (warp * kRegCols + 32 * h) * 2 + (j + (lane >> 4)) * 16);
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(b[j][s][0]), "=r"(b[j][s][1]), "=r"(b[j + 1][s][0]), "=r"(b[j + 1][s][1])
                       : "r"(at));
        }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int n = c + 32 * h + 8 * (g >> 1) + 2 * j + (g & 1);
        n = n < a.C ? n : a.C - 1;  // a column past the end is not stored
        const uint16_t* from = G + int64_t(n) * a.R;
        if constexpr (KS == 1) {
          const uint2 w = 4 * q < a.R ? *reinterpret_cast<const uint2*>(from + 4 * q) : make_uint2(0u, 0u);
          b[j][0][0] = w.x;
          b[j][0][1] = w.y;
        } else {
          const int k = kb * 32 + 8 * q;
          const uint4 w = k < a.R ? *reinterpret_cast<const uint4*>(from + k) : make_uint4(0u, 0u, 0u, 0u);
          b[j][0][0] = w.x;
          b[j][0][1] = w.y;
          b[j][1][0] = w.z;
          b[j][1][1] = w.w;
        }
      }
    }
  };
  uint32_t held[KS ? 2 : 1][4][S][2], f[2][S][4];
  if (busy) {
    int found[kTile / 32];
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i)
      found[i] = first + 32 * i + lane < count ? a.plan.perm[pos + first + 32 * i + lane] : 0;
    if constexpr (KS > 0 && !GMN) {  // G does not wait for the rows
      load_b(n0, 0, 0, held[0]);
      load_b(n0, 0, 1, held[1]);
    }
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i)
      if (first + 32 * i + lane < count) rowid[first + 32 * i + lane] = found[i];
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kStages; ++s) copy(s);
  }
  // a group of 32 rows: g, g + 8, g + 16, g + 24 are this lane's
  auto find = [&](int r0, int (&rows)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = r0 + 8 * k + g;
      rows[k] = r < count ? rowid[r] : -1;
    }
  };
  auto piece = [&](int s, int h, int k) {
    return a.base ? *reinterpret_cast<const uint4*>(mine + s * 4096 + (8 * k + g) * 128 +
                                                    (((4 * h + q) ^ ((g & 1) << 2)) << 4))
                  : make_uint4(0u, 0u, 0u, 0u);
  };
  auto put = [&](int row, int h, const uint4& v) {
    uint16_t* to = row_at(a.Y + n0 + 8 * q, row, a.pitch_y);
    const int c = n0 + 32 * h + 8 * q;
    if (row < 0) return;
    if (n0 + kRegCols <= a.C) *reinterpret_cast<uint4*>(to + 32 * h) = v;
    else if (c < a.C) store_cols8(to - (n0 + 8 * q), c, a.C, v);
  };
  int rows[4];
  if (adapter < 0) {
    if (!busy) return;
    for (int r0 = first, s = 0; r0 < count && n0 < a.C; advance(n0, r0), s = s + 1 == kStages ? 0 : s + 1) {
      find(r0, rows);
      cp_async_wait<kStages - 1>();
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!kFew || r0 + 8 * k < count) put(rows[k], h, piece(s, h, k));
      __syncwarp();
      copy(s);
    }
    return;
  }
  // fragments of P: rows 16 m .. of the group, step pair kb
  auto load_a = [&](const int (&rows)[4], int kb, int m, uint32_t (&f)[S][4]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rows[2 * m + r];
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (KS == 1) {
        if (row >= 0 && 4 * q < a.R) {
          const uint2 u = *reinterpret_cast<const uint2*>(row_at(a.P + 4 * q, row, a.pitch_p));
          w.x = u.x;
          w.y = u.y;
        }
        f[0][r] = w.x;
        f[0][2 + r] = w.y;
      } else {
        const int k = kb * 32 + 8 * q;
        if (row >= 0 && k < a.R) w = *reinterpret_cast<const uint4*>(row_at(a.P + 8 * q, row, a.pitch_p) + kb * 32);
        f[0][r] = w.x;
        f[0][2 + r] = w.y;
        f[1][r] = w.z;
        f[1][2 + r] = w.w;
      }
    }
  };
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  if constexpr (GMN) {
    // G is [R][C]: its columns of this block to shared memory, rows and columns
    // in the order that the fragments take them; zeros past R and C
    const int krows = KS == 1 ? 16 : (a.R + 31) / 32 * 32;
    for (int i = threadIdx.x; i < krows * (Sh::COLS / 8); i += Sh::THREADS) {
      const int k = i / (Sh::COLS / 8), v = i % (Sh::COLS / 8);
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (k < a.R && nb + 8 * v < a.C) w = *reinterpret_cast<const uint4*>(G + int64_t(k) * a.C + nb + 8 * v);
      const int kp = KS == 1 ? 8 * ((k >> 1) & 1) + 2 * (k >> 2) + (k & 1)
                             : (k & ~31) + 16 * ((k >> 2) & 1) + 8 * ((k >> 1) & 1) + 2 * ((k >> 3) & 3) + (k & 1);
      uint32_t* to = reinterpret_cast<uint32_t*>(gst + kp * Sh::PITCH + (v >> 2) * 64 + (v & 3) * 4);
      to[0] = w.x;
      to[4] = w.y;
      to[8] = w.z;
      to[12] = w.w;
    }
    __syncthreads();
  }
  if (!busy) return;
  find(first, rows);
  if constexpr (KS > 0) {
    if constexpr (GMN) {
      load_b(n0, 0, 0, held[0]);
      load_b(n0, 0, 1, held[1]);
    }
    load_a(rows, 0, 0, f[0]);
    load_a(rows, 0, 1, f[1]);
  }
  for (int r0 = first, s = 0; r0 < count && n0 < a.C; s = s + 1 == kStages ? 0 : s + 1) {
    int next[4], nn = n0, nr = r0;
    advance(nn, nr);
    find(nr, next);
    // the next group's operands, as soon as their registers are free
    auto ahead = [&](int h, int m) {
      if (h == 1 && !(WALK && count <= 32)) load_a(next, 0, m, f[m]);
      if (WALK && m == 1 && nn != n0 && nn < a.C) load_b(nn, 0, h, held[h]);
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (kFew && m == 1 && r0 + 16 >= count) {  // no row in this half: only the next group's reads
          if constexpr (KS > 0) ahead(h, 1);
          break;
        }
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
        auto product = [&](const uint32_t(&fa)[S][4], const uint32_t(&b)[4][S][2]) {
#pragma unroll
          for (int st = 0; st < S; ++st)
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16816<BF16>(acc[j], fa[st], b[j][st][0], b[j][st][1]);
        };
        if constexpr (KS > 0) {
          product(f[m], held[h]);
          ahead(h, m);
        } else {
          for (int kb = 0; kb < (a.R + 31) / 32; ++kb) {
            load_a(rows, kb, m, f[0]);
            load_b(n0, kb, h, held[0]);
            product(f[0], held[0]);
          }
        }
        if (h == 0 && m == 0) {
          cp_async_wait<kStages - 1>();
          __syncwarp();
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (kFew && r0 + 16 * m + 8 * r >= count) break;
          uint4 x = piece(s, h, 2 * m + r);
          uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 b = unpack2<BF16>(w[j]);
            w[j] = pack2<BF16>(fmaf(scale, acc[j][2 * r], b.x), fmaf(scale, acc[j][2 * r + 1], b.y));
          }
          put(rows[2 * m + r], h, x);
        }
      }
    }
    __syncwarp();
    copy(s);
    n0 = nn;
    r0 = nr;
#pragma unroll
    for (int k = 0; k < 4; ++k) rows[k] = next[k];
  }
}

// ---- expand for larger R: the same with tcgen05 ------------------------------------------
// A block takes a tile and `span` blocks of 128 columns.  The product comes from
// MMAs over R in chunks of 64 (with mma.sync the operands' traffic through L1
// grows with R: 142 us for [8192, 16384] at R = 64, 273 us at R = 128; now 117
// and 165; R in one piece leaves room for three blocks an SM: 172 us).  base is
// in registers before it and is added in the same layout, which tcgen05.ld
// 16x256b and a permuted order of G's columns in shared memory give: a lane has
// 8 consecutive columns of a row.  Up to R = 64 P is staged once a block; base of
// the next columns is read as the registers of this one's become free.
struct ExpandTcArgs {
  ExpandRegArgs a;
  int span;
  uint32_t* err;
};
constexpr int kTcCols = 128;

template <bool BF16, bool GMN>
__global__ void __launch_bounds__(128, 4) expand_tc_kernel(const ExpandTcArgs ta) {
  const ExpandRegArgs& a = ta.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int R = a.R, Rn = round16(R), chunks = (Rn + 63) / 64;
  uint8_t* Ps = smem;               // [128 rows][64 of R], K-major
  uint8_t* Gs = Ps + kTile * 128;   // [128 columns][64 of R], K-major, or [64 of R][2 x 64 columns], N-major
  const Ring ring = ring_at(Gs + kTcCols * 128);
  ring_init(ring, kTcCols, warp);
  const uint32_t tmem = *ring.tmem;
  griddep_wait();
  const int4 t = a.plan.tiles[blockIdx.y];
  const int adapter = t.x, pos = t.y, count = t.z;
  const bool none = adapter < 0;
  if (int(blockIdx.y) >= a.plan.hdr[0] || (none && a.base == a.Y)) {
    if (warp == 1) tmem_dealloc(tmem, kTcCols);
    return;
  }
  const int first = blockIdx.x * ta.span * kTcCols;
  const int last = min(a.C, first + ta.span * kTcCols);
  int rows[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 32 * warp + 8 * k + g;
    rows[k] = r < count ? a.plan.perm[pos + r] : -1;
  }
  uint4 x[4][4];
  auto fetch = [&](int n0, int h) {  // this lane's columns 8 q .. of 32 h ..
    const int c = n0 + 32 * h + 8 * q;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[h][k] = make_uint4(0u, 0u, 0u, 0u);
      if (a.base && rows[k] >= 0 && c < last) x[h][k] = load_cols8(row_at(a.base, rows[k], a.pitch_b), c, a.C);
    }
  };
#pragma unroll
  for (int h = 0; h < 4; ++h) fetch(first, h);
  // Operands in 128-byte swizzled rows of 64: piece c of row r sits at c ^ (r % 8).
  // All copies are under way before any is waited for: with loads and stores
  // through registers R = 64 took 182 us.
  const uint16_t* G = a.G + int64_t(none ? 0 : adapter) * a.C * R;
  auto stage_p = [&](int kc) {
    const int pieces = min(64, Rn - 64 * kc) / 8;
    for (int i = threadIdx.x; i < count * pieces; i += 128) {
      const int r = i / pieces, c = i - r * pieces, k = 64 * kc + 8 * c;
      const bool ok = k < R;
      cp_async16(Ps + r * 128 + ((c ^ (r & 7)) << 4), row_at(a.P + (ok ? k : 0), a.plan.perm[pos + r], a.pitch_p),
                 ok ? 16 : 0);
    }
  };
  auto stage_g = [&](int n0, int kc) {
    // column 32 i + 8 j + 2 k + e of the MMA is column 32 i + 8 k + 2 j + e of G
    const int depth = min(64, Rn - 64 * kc);
    if constexpr (GMN) {
      for (int i = threadIdx.x; i < depth * (kTcCols / 2); i += 128) {  // pairs of columns
        const int k = i / (kTcCols / 2), v = i % (kTcCols / 2);
        const int c = 4 * ((v >> 4) & 1) + (v & 3);  // piece of the 64 columns, and 4 bytes of it
        const bool ok = 64 * kc + k < R && n0 + 2 * v < a.C;
        cp_async4(Gs + (v >> 5) * 64 * 128 + k * 128 + ((c ^ (k & 7)) << 4) + ((v >> 2) & 3) * 4,
                  G + (ok ? int64_t(64 * kc + k) * a.C + n0 + 2 * v : 0), ok);
      }
    } else {
      const int pieces = depth / 8;
      for (int i = threadIdx.x; i < kTcCols * pieces; i += 128) {
        const int v = i / pieces, c = i - v * pieces, k = 64 * kc + 8 * c;  // column v of the block, k .. of its row
        // its place: the order is its own inverse
        const int n = (v & ~31) + 8 * ((v >> 1) & 3) + 2 * ((v >> 3) & 3) + (v & 1);
        const bool ok = n0 + v < a.C && k < R;
        cp_async16(Gs + n * 128 + ((c ^ (n & 7)) << 4), G + (ok ? int64_t(n0 + v) * R + k : 0), ok ? 16 : 0);
      }
    }
  };
  if (!none) {
    stage_p(0);
    stage_g(first, 0);
  }
  const float scale = none ? 0.f : a.scale ? a.scale[adapter] : 1.f;
  const uint32_t idesc = instr_desc_major(BF16, kTile, kTcCols, 0, GMN ? 1 : 0);
  uint32_t phase = 0;
  for (int n0 = first; n0 < last; n0 += kTcCols) {
    const bool more = n0 + kTcCols < last;
    for (int kc = 0; kc < chunks && !none; ++kc) {
      cp_async_wait_all();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();  // operands are there, and the accumulators of the last columns have been read
      tc_fence_after();
      if (threadIdx.x == 0) {
        for (int k = 0; k < min(64, Rn - 64 * kc) / 16; ++k) {
          const uint64_t ad = desc_k_major(Ps) + ((32 * k) >> 4);
          const uint64_t bd = GMN ? desc_mn_major(Gs + 2048 * k, 64 * 128) : desc_k_major(Gs) + ((32 * k) >> 4);
          tc_mma(tmem, ad, bd, idesc, (kc | k) != 0);
        }
        tc_commit(ring.done);
      }
      __syncwarp();
      tail_wait(ring.done, phase, ta.err);
      phase ^= 1u;
      __syncwarp();
      tc_fence_after();
      // the product has read its operands: the next ones are copied, the last
      // time behind the sums (a second buffer of G: 159 against 147 us at R = 64)
      const bool last_chunk = kc + 1 == chunks;
      if (!last_chunk || more) {
        if (chunks > 1) stage_p(last_chunk ? 0 : kc + 1);
        last_chunk ? stage_g(n0 + kTcCols, 0) : stage_g(n0, kc + 1);
      }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (!none && 32 * warp < count) {
        uint32_t lo[16], hi[16];  // rows g, g + 8 and g + 16, g + 24
        const uint32_t at = tmem + (uint32_t(32 * warp) << 16) + 32 * h;
        tmem_ld_16x256b_x4(at, lo);
        tmem_ld_16x256b_x4(at + (16u << 16), hi);
        tmem_ld_wait(lo, hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t(&d)[16] = k < 2 ? lo : hi;
          uint32_t* w = reinterpret_cast<uint32_t*>(&x[h][k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 b = unpack2<BF16>(w[j]);
            w[j] = pack2<BF16>(fmaf(scale, __uint_as_float(d[4 * j + 2 * (k & 1)]), b.x),
                               fmaf(scale, __uint_as_float(d[4 * j + 2 * (k & 1) + 1]), b.y));
          }
        }
      }
      const int c = n0 + 32 * h + 8 * q;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (rows[k] >= 0 && c < a.C) store_cols8(row_at(a.Y, rows[k], a.pitch_y), c, a.C, x[h][k]);
      if (more) fetch(n0 + kTcCols, h);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTcCols);
  }
}

// ---- wgrad: dG_l [C][R] = s_l sum over l's rows of T[m][c] P[m][r] ----------------------
// A unit of work is a block of kWgCols columns of T and an adapter.  One block
// takes it, or (parts > 1) all blocks of a cluster split the adapter's rows in
// chunks of 64 and add their sums as shrink_kernel does.
// Both operands are read with the row as the MMA's K index.  Bound by the reading of
// T and the chain of loads, sums and the last join: X [8192, 4096] with four
// adapters 20 us at rank 16, 27 us at rank 64.
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
__device__ __forceinline__ void wgrad_body(uint8_t* smem, const CUtensorMap& tmT, const CUtensorMap& tmT1,
                                           const CUtensorMap& tmP, const CUtensorMap& tmP1, const WgradArgs& a,
                                           int block, int adapter, int cs, int rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = a.R, vecs = R / 8, Rn = round16(R), halves = R > 64 ? 2 : 1;
  const int c0 = block * kWgCols;
  const int cols = min(kWgCols, a.C - c0);
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
  griddep_wait();
  const int start = a.plan.start[adapter], rows = a.plan.start[adapter + 1] - start;
  uint16_t* dG = static_cast<uint16_t*>(a.dG) + int64_t(adapter) * a.C * R;
  if (rows == 0) {  // an adapter without rows: zeros
    if (warp == 1) tmem_dealloc(tmem, tcols);
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
  const int chunks = (rows + 63) / 64;
  const int q0 = int(int64_t(chunks) * rank / cs), n = int(int64_t(chunks) * (rank + 1) / cs) - q0;

  if (warp == 0) {
    const uint32_t tx = subs * 8192 + halves * pbytes;
    int i = 0;
    for (Turn w(a.stages); i < n; ++i, w.next()) {
      const int s = w.s;
      const int at = (q0 + i) * 64;
      const TileRows r = tile_rows(a.plan.perm, start + at, min(64, rows - at), lane, a.M);
      if (!mbar_wait_warp(&ring.empty[s], w.ph ^ 1u, ring.abort_flag, a.err, ERR_WAIT_EMPTY)) break;
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
      const uint64_t ad0 = desc_mn_major(smem, 8192), bd0 = desc_rows(smem + tbytes, a.rowb, pbytes);
      Turn r(a.stages);
      for (int i = 0; i < n; ++i, r.next()) {
        if (!mbar_wait(&ring.full[r.s], r.ph, ring.abort_flag, a.err, ERR_WAIT_FULL)) break;
        tc_fence_after();
        const uint64_t ad = ad0 + ((r.s * stage_bytes) >> 4), bd = bd0 + ((r.s * stage_bytes) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma(tmem, ad + ((2048 * k) >> 4), bd + a.rowb * k, idesc, (i | k) != 0);
        tc_commit(&ring.empty[r.s]);
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
  cs > 1 ? cluster_sync() : __syncthreads();
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
      const uint32_t at = smem_addr(part + c * pitch + r);
      const uint32_t from = cs > 1 ? mapa_shared(at, q) : mapa_shared(at, cluster_ctarank());
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
  if (cs > 1) cluster_sync();
}

template <bool BF16, bool OT>
__global__ void __launch_bounds__(128) wgrad_kernel(const __grid_constant__ CUtensorMap tmT,
                                                    const __grid_constant__ CUtensorMap tmT1,
                                                    const __grid_constant__ CUtensorMap tmP,
                                                    const __grid_constant__ CUtensorMap tmP1, const WgradArgs a,
                                                    int blocks) {
  extern __shared__ uint8_t smem_raw[];
  const int unit = blockIdx.x / cluster_nctarank();
  wgrad_body<BF16, OT>(align1024(smem_raw), tmT, tmT1, tmP, tmP1, a, unit % blocks, unit / blocks, cluster_nctarank(),
                       cluster_ctarank());
}

// ---- both readers of dY: U (shrink) and dB (wgrad) in one launch -------------------------
// The first clusters take the row tiles; all of them are resident at once
// and move along the columns, each rank through its own share of them.  The
// others take the blocks of columns in the order in which the ranks reach them,
// so that whichever reads a part of dY second finds it in L2.  Where there are
// units enough (parts == 1) each block of a cluster has one of its own: split
// over the cluster, [2048, 16384] with 4 adapters took 74 us of 4096 blocks with
// one chunk of rows each.  [8192, 16384]: 79 us at rank 16, 90 us at rank 64, where 390 MB
// come from DRAM (the matrix has 268); DRAM is busy 55 % of that time, L2
// 40 %, and the blocks wait for their loads.
template <bool BF16>
__global__ void __launch_bounds__(128) dual_kernel(const __grid_constant__ CUtensorMap tmT,
                                                   const __grid_constant__ CUtensorMap tmT1,
                                                   const __grid_constant__ CUtensorMap tmG,
                                                   const __grid_constant__ CUtensorMap tmP,
                                                   const __grid_constant__ CUtensorMap tmP1, const ShrinkArgs sa,
                                                   const WgradArgs wa, int tiles, int blocks, int adapters,
                                                   int parts) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const int cs = cluster_nctarank();
  const int unit = blockIdx.x / cs;
  if (unit < tiles) {
    shrink_body<BF16, true>(smem, tmT, tmT1, tmG, sa, unit);
  } else {
    const int rank = cluster_ctarank();
    const int u = parts > 1 ? unit - tiles : (unit - tiles) * cs + rank;
    const int k = u / adapters;  // k-th block of columns in the ranks' order
    const int per = (blocks + cs - 1) / cs;
    const int block = (k % cs) * per + k / cs;
    // some places of the order are past the last block: nothing to do
    if (k < per * cs && block < blocks)
      wgrad_body<BF16, false>(smem, tmT, tmT1, tmP, tmP1, wa, block, u % adapters, parts, parts > 1 ? rank : 0);
  }
}

// ---- host ---------------------------------------------------------------------------
template <class K>
spg_status prepare(K kern, int smem) {
  return allow_smem(reinterpret_cast<const void*>(kern), smem) == cudaSuccess ? SPG_OK : SPG_ERR_CUDA;
}

// Rows of a matrix: boxes of 32 rows, and single rows for gathers, of `rowb` bytes.
bool rows_maps(CUtensorMap* box, CUtensorMap* one, const void* p, int64_t cols, int64_t rows, int64_t ld, int rowb) {
  return make_tmap_2d_swz(box, p, 2, uint64_t(cols), uint64_t(rows), uint64_t(ld) * 2, rowb / 2, 32, rowb) &&
         make_tmap_2d_swz(one, p, 2, uint64_t(cols), uint64_t(rows), uint64_t(ld) * 2, rowb / 2, 1, rowb);
}

int ring_stages(int budget, int stage) {
  const int n = budget / stage;
  return n > kMaxStages ? kMaxStages : n < 2 ? 2 : n;
}

constexpr int kShortRing = 50 * 1024;  // four blocks an SM

// Maps, arguments and launch shape of a shrink; `budget` bytes of ring.
template <bool GMN>
struct ShrinkPlan {
  CUtensorMap tmT, tmT1, tmG;
  ShrinkArgs a;
  int64_t tiles;
  int cs, smem;
  bool ok;
  ShrinkPlan(const void* T, int64_t ldt, const void* G, const float* scale, const Plan& plan, void* P, int64_t ldp,
             int64_t M, int64_t D, int64_t R, int64_t L, int budget, uint32_t* err) {
    const int Rn = round16(int(R)), rowb = row_bytes_of(int(R));
    ok = rows_maps(&tmT, &tmT1, T, D, M, ldt, 128) &&
         (GMN ? make_tmap_3d(&tmG, G, R, D, L, 64, rowb) : make_tmap_3d(&tmG, G, D, R, L, Rn, 128));
    const int gbytes = GMN ? 64 * rowb * (R > 64 ? 2 : 1) : Rn * 128;
    const int trows = M < kTile ? (int(M) + 31) / 32 * 32 : kTile;
    const int stage = trows * 128 + gbytes;
    // blocks of a cluster: as many as let every tile that is expected to have rows
    // be resident at once with two blocks an SM, each with at least two steps of
    // its own (shrink of [8192, 4096], rank 16, alone: 17 us with 4, 20 us with 2 or 8)
    const int64_t nkb = (D + 63) / 64;
    const int64_t busy = M < 64 * L ? (M < L ? M : L) + M / kTile : (M + kTile - 1) / kTile;
    tiles = max_tiles(M, L);
    cs = 1;
    while (cs < 8 && busy * 2 * cs <= 2 * sm_count() && nkb >= 4 * cs) cs *= 2;
    // small stages: twice as many blocks an SM with shorter rings (a row each of 64
    // adapters, K = 4096, rank 16: 19 us with the expand, 26 with long rings)
    if (cs < 8 && budget > kShortRing && trows < kTile && nkb >= 4 * cs && busy * 2 * cs <= 4 * sm_count()) {
      cs *= 2;
      budget = kShortRing;
    }
    // the same where the adapters' last tiles may make them more than two blocks an
    // SM ([8192, 4096], 32 adapters in no order: 31 us, with long rings 42)
    if (budget > kShortRing && M >= 64 * L && (busy + L) * cs > 2 * sm_count()) budget = kShortRing;
    const int stages = ring_stages(budget, stage);
    const int ring = ring_of(stages, stage), part = kTile * (int(R) + 4) * 4;
    smem = block_smem(ring > part ? ring : part, round16(int(R)));
    a = ShrinkArgs{plan, scale, P, ldp, int(M), int(D), int(R), stages, trows, gbytes, rowb, err};
  }
};

template <bool BF16, bool GMN>
spg_status shrink(const void* T, int64_t ldt, const void* G, const float* scale, const Plan& plan, void* P, int64_t ldp,
                  int64_t M, int64_t D, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  const ShrinkPlan<GMN> s(T, ldt, G, scale, plan, P, ldp, M, D, R, L, 100 * 1024, err);
  auto kern = shrink_kernel<BF16, GMN>;
  if (!s.ok || prepare(kern, s.smem) != SPG_OK) return SPG_ERR_CUDA;
  return launch_pdl_cluster(kern, dim3(unsigned(s.tiles * s.cs)), dim3(128), s.smem, s.cs, st, s.tmT, s.tmT1, s.tmG,
                            s.a) == cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

// Y = base + s P G^T.  Up to R = 32 the product is a matter of registers.
// Beyond that tcgen05 does it where there are whole tiles (at least 64 rows
// for each adapter that rows can have); few rows stay with the register kernel.
template <bool BF16, bool GMN>
spg_status expand(const void* P, int64_t ldp, const void* G, const float* scale, const Plan& plan, const void* base,
                  int64_t ldb, void* Y, int64_t ldy, int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err,
                  cudaStream_t st) {
  const ExpandRegArgs a{plan, scale, static_cast<const uint16_t*>(P), static_cast<const uint16_t*>(G),
                        static_cast<const uint16_t*>(base), static_cast<uint16_t*>(Y), uint32_t(ldp * 2),
                        uint32_t(ldb * 2), uint32_t(ldy * 2), int(C), int(R)};
  const unsigned tiles = unsigned(max_tiles(M, L));
  if (R > 32 && M >= 64 * L) {
    const int smem = (kTile + kTcCols) * 128 + kBarBytes + 1024;
    auto kern = expand_tc_kernel<BF16, GMN>;
    if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
    // two blocks of columns a block while there are three rounds of blocks
    // ([8192, 16384], R = 64: 126, 117 and 119 us with 1, 2 and 4; [1024, 4096]: 15, 19 and 26)
    const int64_t blocks = (C + kTcCols - 1) / kTcCols, busy = (M + kTile - 1) / kTile;
    const int span = busy * (blocks / 2) >= 12 * sm_count() ? 2 : 1;
    // Not launched ahead of the shrink's end: an SM that never idles keeps the
    // shrink's large share of shared memory, and the loads of base under way are
    // limited by what that leaves to L1 (R = 64: 144 against 119 us).
    const ExpandTcArgs ta{a, span, err};
    kern<<<dim3(unsigned((blocks + span - 1) / span), tiles), dim3(128), smem, st>>>(ta);
    return launch_status();
  }
  // Few whole tiles: their groups of 32 rows go to warps side by side ([2048, 2048],
  // rank 16, behind a small shrink: 9.3 against 12.5 us); otherwise a warp takes them in turn and
  // keeps G ([2048, 4096] 15.4 against 15.8 us, above that no difference).
  const int64_t busy = M / kTile * ((C + 255) / 256);
  auto go = [&](auto kern, auto shape, int64_t span) -> spg_status {
    using Sh = decltype(shape);
    const int smem = Sh::BASE + (GMN ? (R <= 16 ? 16 : (int(R) + 31) / 32 * 32) * Sh::PITCH : 0);
    if (prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
    const int64_t blocks = (C + Sh::COLS - 1) / Sh::COLS;
    return launch_pdl(kern, dim3(unsigned((blocks + span - 1) / span), tiles), dim3(Sh::THREADS), smem, st, a) ==
                   cudaSuccess
               ? launch_status()
               : SPG_ERR_CUDA;
  };
  if (R > 32) return go(expand_reg_kernel<BF16, GMN, 0, 1, false>, RegShape<1>(), 1);
  if (M >= 64 * L && busy > 0 && busy < 2 * sm_count())
    return go(R <= 16 ? expand_reg_kernel<BF16, GMN, 1, 4, false> : expand_reg_kernel<BF16, GMN, 2, 4, false>,
              RegShape<4>(), 1);
  if constexpr (!GMN) {
    if (M < 64 * L) {
      // a row each of 64 adapters, C 16384, rank 16: 14.0 us with three blocks of columns a
      // block, 14.2 with six, 16.0 with eight, 16.5 with one
      const int64_t groups = M < L ? M : L;
      int64_t span = groups * ((C + 255) / 256) / (8 * sm_count());
      span = span < 1 ? 1 : span > 8 ? 8 : span;
      return go(R <= 16 ? expand_reg_kernel<BF16, GMN, 1, 1, true> : expand_reg_kernel<BF16, GMN, 2, 1, true>,
                RegShape<1>(), span);
    }
  }
  return go(R <= 16 ? expand_reg_kernel<BF16, GMN, 1, 1, false> : expand_reg_kernel<BF16, GMN, 2, 1, false>,
            RegShape<1>(), 1);
}

// Adapters that can have whole tiles of rows.
int64_t row_groups(int64_t M, int64_t L) { return L < M / kTile + 1 ? L : M / kTile + 1; }

// The same for a wgrad.
struct WgradPlan {
  CUtensorMap tmT, tmT1, tmP, tmP1;
  WgradArgs a;
  int64_t blocks;
  int cs, smem;
  bool ok;
  WgradPlan(const void* T, int64_t ldt, const void* P, int64_t ldp, const float* scale, const Plan& plan, void* dG,
            int64_t M, int64_t C, int64_t R, int64_t L, int budget, uint32_t* err) {
    const int rowb = row_bytes_of(int(R));
    ok = rows_maps(&tmT, &tmT1, T, C, M, ldt, 128) && rows_maps(&tmP, &tmP1, P, R, M, ldp, rowb);
    const int stage = (kWgCols / 64) * 8192 + (R > 64 ? 2 : 1) * 64 * rowb;
    const int stages = ring_stages(budget, stage);
    blocks = (C + kWgCols - 1) / kWgCols;
    // blocks of a cluster: up to some three an SM, with a chunk each where the
    // rows are spread evenly
    const int64_t groups = row_groups(M, L);
    cs = 1;
    while (cs < 8 && blocks * groups * cs < 2 * sm_count() && M / groups >= 64 * cs) cs *= 2;
    const int ring = stages * stage, part = kWgCols * (int(R) + 4) * 4;
    smem = block_smem(ring > part ? ring : part, round16(int(R)));
    a = WgradArgs{plan, scale, dG, int(M), int(C), int(R), stages, rowb, err};
  }
};

template <bool BF16, bool OT>
spg_status wgrad(const void* T, int64_t ldt, const void* P, int64_t ldp, const float* scale, const Plan& plan, void* dG,
                 int64_t M, int64_t C, int64_t R, int64_t L, uint32_t* err, cudaStream_t st) {
  // a quarter of an SM's shared memory each: a block's first loads and last sums hide behind three others
  // ([8192, 16384], rank 16, 8 adapters: 60 us; with two blocks an SM 95 us)
  const WgradPlan w(T, ldt, P, ldp, scale, plan, dG, M, C, R, L, 50 * 1024, err);
  auto kern = wgrad_kernel<BF16, OT>;
  if (!w.ok || prepare(kern, w.smem) != SPG_OK) return SPG_ERR_CUDA;
  return launch_pdl_cluster(kern, dim3(unsigned(w.blocks * L * w.cs)), dim3(128), w.smem, w.cs, st, w.tmT, w.tmT1,
                            w.tmP, w.tmP1, w.a, int(w.blocks)) == cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

// U = s dY B_l and dB = s dY^T V, from one reading of dY unless it has few columns:
// then the sums over rows need many more blocks a unit than those over columns,
// and two launches do better (backward of [5692, 144], rank 128: 80 against 169 us;
// with twice as many [1970, 1000], rank 8: 31 against 23 us).
template <bool BF16>
spg_status dual(const void* dY, int64_t lddy, const void* B, const float* scale, const Plan& plan, void* U,
                const void* V, int64_t ldv, void* dB, int64_t M, int64_t N, int64_t R, int64_t L, uint32_t* err,
                cudaStream_t st) {
  const ShrinkPlan<true> s(dY, lddy, B, scale, plan, U, R, M, N, R, L, kShortRing, err);
  const WgradPlan w(dY, lddy, V, ldv, scale, plan, dB, M, N, R, L, 50 * 1024, err);
  if (w.cs >= 4 * s.cs) {
    const spg_status rc = shrink<BF16, true>(dY, lddy, B, scale, plan, U, R, M, N, R, L, err, st);
    return rc != SPG_OK ? rc : wgrad<BF16, false>(dY, lddy, V, ldv, scale, plan, dB, M, N, R, L, err, st);
  }
  auto kern = dual_kernel<BF16>;
  const int smem = s.smem > w.smem ? s.smem : w.smem;
  if (!s.ok || !w.ok || prepare(kern, smem) != SPG_OK) return SPG_ERR_CUDA;
  const int64_t units = (w.blocks + s.cs - 1) / s.cs * s.cs * L;
  // a unit's rows are split over the cluster only where the units do not fill the
  // device and most blocks have rows (backward of 11 rows of 16 adapters, N 13920:
  // 38 us, split 189; [1970, 1000], 5 adapters: split over 8 blocks 23 us, 31 in one)
  const int64_t groups = row_groups(M, L);
  const int parts = w.blocks * groups < sm_count() && M / groups >= 32 * s.cs ? s.cs : 1;
  const int64_t clusters = s.tiles + (parts > 1 ? units : (units + s.cs - 1) / s.cs);
  return launch_pdl_cluster(kern, dim3(unsigned(clusters * s.cs)), dim3(128), smem, s.cs, st, s.tmT, s.tmT1, s.tmG,
                            w.tmP, w.tmP1, s.a, w.a, int(s.tiles), int(w.blocks), int(L), parts) == cudaSuccess
             ? launch_status()
             : SPG_ERR_CUDA;
}

// One of `outs` is the memory of one of `ins`.
bool any_same(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (const void* o : outs)
    for (const void* i : ins)
      if (o && o == i) return true;
  return false;
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
  if (M >= (int64_t(1) << 22) || N >= kMaxPitch - 256 || K >= kMaxPitch - 256 || ldx >= kMaxPitch ||
      ldv >= kMaxPitch)
    return SPG_ERR_UNSUPPORTED_SHAPE;
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
  spg_status rc = dual<BF16>(dY, lddy, B, scale, plan, U, V, ldv, dB, M, N, R, L, err, st);
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
  if (M < 0 || L <= 0) return SPG_ERR_INVALID_ARG;
  if (L > kMaxL || M >= (int64_t(1) << 22)) return SPG_ERR_UNSUPPORTED_SHAPE;
  if (!plan || (M != 0 && !index)) return SPG_ERR_INVALID_ARG;
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
  // the 48 KB that need no leave hold the kernel's static arrays too
  if (smem > 40 * 1024 && prepare(plan_kernel, smem) != SPG_OK) return SPG_ERR_CUDA;
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
  if (ldy >= kMaxPitch || (base && ldbase >= kMaxPitch)) return SPG_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return SPG_OK;
  if (!mat_ok(Y, ldy) || (base && !mat_ok(base, ldbase))) return SPG_ERR_MISALIGNED;
  // V is written while X and A are read, and read while base is replaced by Y
  if (any_same({V}, {X, A, B, base, Y}) || any_same({Y}, {A, B})) return SPG_ERR_INVALID_ARG;
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
  if (lddy >= kMaxPitch || (dX && lddx >= kMaxPitch) || (dX && dbase && lddbase >= kMaxPitch))
    return SPG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(dA, 16) || !aligned(dB, 16)) return SPG_ERR_MISALIGNED;
  auto st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // no rows: the sums over them are zero
    rc = check_device();
    if (rc != SPG_OK) return rc;
    if (taken(cudaMemsetAsync(dA, 0, size_t(L) * R * K * 2, st)) != cudaSuccess ||
        taken(cudaMemsetAsync(dB, 0, size_t(L) * N * R * 2, st)) != cudaSuccess)
      return SPG_ERR_CUDA;
    return SPG_OK;
  }
  if (!dY || !workspace || ws_bytes < lora_bwd_workspace_size(M, N, K, R, L)) return SPG_ERR_INVALID_ARG;
  if (!mat_ok(dY, lddy) || (dX && !mat_ok(dX, lddx)) || (dX && dbase && !mat_ok(dbase, lddbase)) ||
      !aligned(workspace, 16))
    return SPG_ERR_MISALIGNED;
  // dB is written while dY, B and V are read, then dA while X is, and then dX while A is
  if (any_same({dA, dB, workspace}, {dY, X, V, A, B, dbase, dX}) || any_same({dX}, {A, B}) ||
      any_same({dB, workspace}, {dA}) || dB == workspace)
    return SPG_ERR_INVALID_ARG;
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
