// ops_block_tc.cuh -- the FP8 products with block scales on the 5th-generation tensor cores.
//
// tcgen05.mma kind::f8f6f4 multiplies the codes as they are; the four MMAs of a block of 128 of K
// leave its sum in tensor memory (fp32; measured within 2^-21.5 of the sum of the products' magnitudes),
// and eight warps read it back, multiply it by the block's two scales and add it to sums in
// registers while the next block is multiplied.  One side of the product lies along the 128 lanes
// (L), the other along the columns (C) of the tensor memory; either may be K-major or have its rows
// contiguous: shared memory holds a block as 128 rows of 128 codes under the 128-byte swizzle both
// ways, and the instruction descriptor says which.
#pragma once
#include "ops_block.cuh"

namespace emu_ops {

constexpr int kTcThreads8 = 384;                         // warps: loads, MMAs, tensor memory, zeros, eight that read
constexpr int kMaxExperts = 1024;
constexpr int kOutStage = 8 * 2 * 4096;                  // staged outputs: two times 32 rows of 128 bytes a warp

enum class BlockKind { dense, grouped, wgrad };
// how the scales enter: one value for a lane's columns; a vector over the columns, the lanes' one value in it; both vectors
enum ScaleMode { kScaleLane = 0, kScaleColumns = 1, kScaleBoth = 2 };

struct BlockSide {
  const float* scale;
  int shift;                                             // of a row to its scale: 0 or 7
  int64_t rs, ks, gs;                                    // the scales' strides by row, block of K, group
  int rows;
  int mn;                                                // rows contiguous instead of K
};
struct BlockTcParams {
  BlockSide l, c;
  int tiles_l, tiles_c, k_blocks, slices;
  int from, to;                                          // dense: the tiles of this launch
  BlockKind kind;
  const int32_t* offsets; int E, T;                      // groups of tokens (grouped: of rows, wgrad: of K)
  int zero_rest;
  void* out; int out_type, out_map;                      // out_map: its rows are 16-byte aligned, and there is a map of it
  int64_t ldl, ldc, out_group;                           // out[l * ldl + c * ldc], one of them 1
  uint32_t idesc;
};
template <int BN> struct BlockTcShape {
  static constexpr bool PAIR = BN == 256;                // two CTAs on a tile of 256 x 256, each with half of either side
  static constexpr bool SWAP = !PAIR;                    // the output's rows are the columns C, and either four reading
                                                         // warps take every other block, with all columns
  static constexpr int L = PAIR ? 256 : 128, C_ROWS = PAIR ? 128 : BN;       // a tile's lanes; rows of C that a CTA loads
  static constexpr int NS = PAIR ? 4 : BN == 64 ? 6 : 8, STAGE = 128 * 128 + C_ROWS * 128, NB = PAIR ? 2 : 4;
  static constexpr int H = PAIR ? 2 : 1;                 // parts of a tile's columns, each with MMAs and barriers of its own
  static constexpr int OWN = PAIR ? BN / 2 : BN, READ = OWN / H, TMEM = NB * BN;          // a warp's columns, and those of a part
  static constexpr int OUT = NS * STAGE, CS = OUT + (PAIR ? kOutStage : BN * 128 * 4), BARS = CS + 8 * 2 * OWN * 4;
  static constexpr int BAR_COUNT = 3 * NS + 2 * NB * H + 10, TABLE = BARS + 8 * BAR_COUNT + 8 + 2 * 12 * 4;
  static constexpr int smem(int E) { return TABLE + 2 * (E + 1) * 4 + 1024; }
  // Narrow tiles' blocks go in turn to two issuing warps.  A wait for a phase tells it from the one before, not from the one
  // before that: each of a stage's (and each of a buffer's) blocks has to be the same warp's.
  static_assert(PAIR || (NS % 2 == 0 && NB % 2 == 0), "a stage's blocks are one issuing warp's");
};
static_assert(BlockTcShape<256>::smem(kMaxExperts) <= kMaxSmem &&
              BlockTcShape<64>::smem(kMaxExperts) <= kMaxSmem && BlockTcShape<32>::smem(kMaxExperts) <= kMaxSmem, "one CTA an SM");

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}
// shared-memory matrix descriptor: rows of 128 bytes under the 128-byte swizzle, eight of them 1024 bytes apart from
// the next eight; with rows contiguous, 128 of them 16 KB apart from the next 128
__device__ __forceinline__ uint64_t desc8(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
template <bool PAIR> __device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (PAIR)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// the arrival of all MMAs issued before: of a pair, at the barriers of both CTAs
template <bool PAIR> __device__ __forceinline__ void commit8(uint32_t bar, uint32_t both) {
  if constexpr (PAIR)
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)both) : "memory");
  else
    tc_commit(bar);
}
template <bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t slot, int columns) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
  if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
// Arrival at a barrier of the pair's first CTA (an address in the cluster).  What it orders are reads of tensor memory and
// TMA loads that have been waited for, not this thread's own stores: without a cluster-wide release, which waits for all
// that the thread has under way (8192 x 5760 x 1920 170 us with it).
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// `bytes` of this CTA's shared memory to another's of the cluster, counted by a barrier there
__device__ __forceinline__ void send(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src),
               "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
// an address of this CTA's shared memory in that of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t in_cluster(uint32_t at, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(rank));
  return a;
}
// 32 columns of this warp's 32 lanes, asked for, and waited for (whatever was asked for before)
__device__ __forceinline__ void tmem_ask(uint32_t addr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// acc += (x, y) * by, and (x, y) * by, of values asked for from tensor memory: volatile, so that they stay behind the wait
__device__ __forceinline__ void add_scaled(f2& acc, float x, float y, f2 by) {
  asm volatile("{\n .reg .b64 v;\n mov.b64 v, {%1, %2};\n fma.rn.f32x2 %0, v, %3, %0;\n}" : "+l"(acc) : "f"(x), "f"(y), "l"(by));
}
__device__ __forceinline__ f2 scaled(float x, float y, f2 by) {
  f2 r;
  asm volatile("{\n .reg .b64 v;\n mov.b64 v, {%1, %2};\n mul.rn.f32x2 %0, v, %3;\n}" : "=l"(r) : "f"(x), "f"(y), "l"(by));
  return r;
}

// One lane of the warp, in code that the whole warp runs: its values are the warp's then, and the addresses and descriptors
// of loads and MMAs need not be moved from a thread's registers (an MMA's issue took 100 cycles with a branch for lane 0).
__device__ __forceinline__ bool one_of_warp() {
  uint32_t one;
  asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, P;\n}" : "=r"(one) :: "memory");
  return one != 0u;
}

// The groups' first rows (within [0, T], none below the one before it) and, of `tile` rows each, how many tiles come
// before them: a scan by all threads, three entries each.
__device__ __forceinline__ void group_table(const int32_t* offsets, int E, int T, int tile, int* start, int* before, int* part) {
  static_assert(kTcThreads8 * 3 > kMaxExperts, "three entries a thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int v[3];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int i = tid * 3 + j, at = i <= E ? __ldg(offsets + i) : 0;
    v[j] = at < 0 ? 0 : at > T ? T : at;
    if (j > 0) v[j] = v[j] > v[j - 1] ? v[j] : v[j - 1];
  }
  int top = v[2];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int w = __shfl_up_sync(0xFFFFFFFFu, top, o);
    if (lane >= o && w > top) top = w;
  }
  int ahead = __shfl_up_sync(0xFFFFFFFFu, top, 1);
  if (lane == 0) ahead = 0;
  if (lane == 31) part[warp] = top;
  __syncthreads();
  for (int w = 0; w < warp; ++w) ahead = part[w] > ahead ? part[w] : ahead;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (tid * 3 + j <= E) start[tid * 3 + j] = v[j] > ahead ? v[j] : ahead;
  __syncthreads();
  int n[3], sum = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int i = tid * 3 + j;
    n[j] = i < E ? (start[i + 1] - start[i] + tile - 1) / tile : 0;
    sum += n[j];
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int w = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += w;
  }
  if (lane == 31) part[12 + warp] = upto;
  __syncthreads();
  int base = upto - sum;
  for (int w = 0; w < warp; ++w) base += part[12 + w];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    if (tid * 3 + j <= E) before[tid * 3 + j] = base;
    base += n[j];
  }
  __syncthreads();
}

__device__ __forceinline__ float4 four_of(f2 a, f2 b) {
  float4 v;
  halves(a, v.x, v.y);
  halves(b, v.z, v.w);
  return v;
}

struct BlockTile {
  int l0, c0, l_end, c_end, group;
  int kb0, kb1, lo, hi;                                  // blocks of K; wgrad: of them the tokens [lo, hi)
};
// eight rows of tiles at a time, column by column, so that the CTAs at work share both sides' rows
__device__ __forceinline__ void tile_order(int tile, int tiles_l, int tiles_c, int& l, int& c) {
  const int group = tile / (8 * tiles_c), first = group * 8, rows = tiles_l - first < 8 ? tiles_l - first : 8;
  const int in = tile - group * 8 * tiles_c;
  l = first + in % rows;
  c = in / rows;
}
template <int BN> __device__ __forceinline__ int tile_count(const BlockTcParams& p, const int* before) {
  if (p.kind == BlockKind::dense) return (p.to - p.from) * p.slices;
  if (p.kind == BlockKind::wgrad) return p.tiles_l * p.tiles_c * p.E;
  return before[p.E] * (BlockTcShape<BN>::SWAP ? p.tiles_l : p.tiles_c);
}
// (rank: which CTA of a pair)
template <int BN> __device__ __forceinline__ BlockTile tile_at(const BlockTcParams& p, const int* start, const int* before, int tile, int rank) {
  BlockTile t;
  t.group = 0;
  t.kb0 = 0;
  t.kb1 = p.k_blocks;
  t.lo = 0;
  t.hi = 0x7FFFFFFF;
  t.l_end = p.l.rows;
  t.c_end = p.c.rows;
  int l, c;
  if (p.kind == BlockKind::grouped) {
    constexpr bool SWAP = BlockTcShape<BN>::SWAP;
    const int weights = SWAP ? p.tiles_l : p.tiles_c, at = tile / weights;
    int a = 0, b = p.E;                                  // before[a] <= at < before[b]
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (before[m] <= at) a = m;
      else b = m;
    }
    t.group = a;
    const int in = tile - before[a] * weights, n = before[a + 1] - before[a];
    const int token = in % n, weight = in / n;           // an expert's tiles that share weights one after the other
    if (SWAP) {
      l = weight;
      t.c0 = start[a] + token * BN;
      t.c_end = start[a + 1];
      t.l0 = l * 128;
    } else {
      c = weight;
      t.l0 = start[a] + token * 256 + rank * 128;
      t.l_end = start[a + 1];
      t.c0 = c * BN;
    }
    return t;
  }
  if (p.kind == BlockKind::wgrad) {
    t.group = tile / (p.tiles_l * p.tiles_c);
    tile -= t.group * p.tiles_l * p.tiles_c;
    t.lo = start[t.group];
    t.hi = start[t.group + 1];
    t.kb0 = t.lo / kBlock;
    t.kb1 = t.hi > t.lo ? (t.hi + kBlock - 1) / kBlock : t.kb0;
  } else {
    if (p.slices > 1) {
      const int slice = tile % p.slices;
      tile /= p.slices;
      t.kb0 = (int)((int64_t)p.k_blocks * slice / p.slices);
      t.kb1 = (int)((int64_t)p.k_blocks * (slice + 1) / p.slices);
    }
    tile += p.from;
  }
  tile_order(tile, p.tiles_l, p.tiles_c, l, c);
  t.l0 = l * BlockTcShape<BN>::L + rank * 128;
  t.c0 = c * BN;
  return t;
}

// A warp's 32 rows (lanes) x 128 columns of sums to row-major memory, 128 bytes of a row at a time by way of shared
// memory (a row's chunks permuted by its number, as the 128-byte swizzle does): by TMA, which the next tile's
// blocks do not wait for, or, of a group's last rows and where rows are not 16-byte aligned, by the warp.  (A bulk
// copy for each row instead takes the TMA unit as long as the loads of a tile.)
template <class T>
__device__ __forceinline__ void write_rows(const BlockTcParams& p, const CUtensorMap* map, const f2 (&acc)[64], unsigned char* stage,
                                           int row0, int rows, int n0, int group, int lane) {
  constexpr int COLS = 128 / sizeof(T), VEC = 16 / sizeof(T);
  const int cols = p.c.rows - n0;                        // may be none
  // TMA leaves out what is behind the last row and column of the output, not of a group
  const bool whole = p.out_map && rows > 0 && (rows >= 32 || p.kind != BlockKind::grouped);
  const bool vec = p.out_map;                            // 16-byte aligned rows
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += 2 * COLS) {           // two pieces at a time
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // those before have been read
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2 * COLS; i += VEC) {
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; j += 2) halves(acc[(c0 + i + j) / 2], v[j], v[j + 1]);
      store_f<T, VEC>(reinterpret_cast<T*>(stage + i / COLS * 4096 + lane * 128 + (((i % COLS / VEC) ^ (lane & 7)) * 16)), v);
    }
    if (whole) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (c0 + i * COLS < cols)
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                         ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(stage) + i * 4096), "r"(n0 + c0 + i * COLS), "r"(row0), "r"(group)
                         : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      continue;
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + k * COLS;
      const unsigned char* const buf = stage + k * 4096;
      T* const out = static_cast<T*>(p.out) + group * p.out_group + (int64_t)row0 * p.ldl + n0 + c;
      if (vec) {
        const int n = (lane & 7) * VEC;
        if (c + n < cols) {
#pragma unroll
          for (int r = lane >> 3; r < 32; r += 4)
            if (r < rows)
              *reinterpret_cast<uint4*>(out + r * p.ldl + n) = *reinterpret_cast<const uint4*>(buf + r * 128 + (((lane & 7) ^ (r & 7)) * 16));
        }
      } else {
#pragma unroll 4
        for (int r = 0; r < rows; ++r)
#pragma unroll
          for (int i = lane; i < COLS; i += 32)
            if (c + i < cols) out[r * p.ldl + i] = *reinterpret_cast<const T*>(buf + r * 128 + (((i / VEC) ^ (r & 7)) * 16) + (i % VEC) * sizeof(T));
      }
    }
  }
}

// Persistent: one CTA an SM, tiles in turn.  Warp 0 loads the blocks by TMA, warp 1 issues the MMAs, warp 2 owns the
// tensor memory, warp 3 clears the tokens of other experts in a weights' gradient's first and last block (and
// tells the pair's first CTA that its blocks are there), warps 4 to 11 scale and add: each holds 32 lanes x BN / 2
// columns of sums in registers.  BN = 256: pairs of CTAs, whose MMAs the first one issues for both (an SM takes
// in 64 bytes a cycle: a block of 128 x 256 outputs would need 48 KB every 512 cycles, of the pair each 32).
// Several slices of K (dense): the CTAs of a cluster, of which each adds up some of the columns at the end.  All
// waits are bounded; a role that gives up sets the status and takes the others along.
template <int BN, int MODE>
__global__ void __launch_bounds__(kTcThreads8, 1)
block_tc_kernel(const __grid_constant__ BlockTcParams p, const __grid_constant__ CUtensorMap map_l,
                const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_out) {
  using SH = BlockTcShape<BN>;
  constexpr bool PAIR = SH::PAIR;
  constexpr int NS = SH::NS, NB = SH::NB, H = SH::H, OWN = SH::OWN, READ = SH::READ;
  extern __shared__ unsigned char raw[];
  unsigned char* const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  const uint32_t full = base + SH::BARS, empty = full + 8 * NS, fixed = empty + 8 * NS, tfull = fixed + 8 * NS, tempty = tfull + 8 * NB * H,
                 joined = tempty + 8 * NB * H, parted = joined + 32, drained = parted + 32, met_all = drained + 8;
  uint32_t* const slot = reinterpret_cast<uint32_t*>(smem + SH::BARS + 8 * SH::BAR_COUNT);
  volatile int* const given_up = reinterpret_cast<volatile int*>(slot + 1);
  int* const part = reinterpret_cast<int*>(slot + 2);
  int* const start = reinterpret_cast<int*>(smem + SH::TABLE);
  int* const before = start + p.E + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // the same for all, and known to be
  const int rank = PAIR ? blockIdx.x & 1 : 0, first_tile = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;
  const int lead = PAIR && p.slices > 1 ? blockIdx.x & 2 : 0;             // the pair's first CTA in the cluster
  const uint32_t both = 3u << lead;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, H);
      bar_init(fixed + 8 * i, PAIR ? 2 : 1);
    }
    for (int i = 0; i < NB * H; ++i) {
      bar_init(tfull + 8 * i, 1);
      bar_init(tempty + 8 * i, PAIR ? 16 : 4);            // one arrival a reading warp
    }
    for (int i = 0; i < 8; ++i) bar_init(joined + 8 * i, 1);
    bar_init(drained, 2);
    bar_init(met_all, 1);
    if (p.slices > 1) bar_expect(met_all, OWN * 128 * 4); // what the slices send of this one's columns
    *given_up = 0;
    bar_init_fence();
  }
  if (warp == 2) tmem_alloc<PAIR>(smem_addr(slot), SH::TMEM);
  if (p.kind != BlockKind::dense) group_table(p.offsets, p.E, p.T, PAIR ? 256 : BN, start, before, part);
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                              // the other's barriers are there
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int tiles = tile_count<BN>(p, before);

  if (warp < 4) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");       // the operands are laid out
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first_tile; tile < tiles && ok; tile += step) {
        const BlockTile t = tile_at<BN>(p, start, before, tile, rank);
        const int gl = p.kind == BlockKind::grouped && SH::SWAP ? t.group : 0, gc = p.kind == BlockKind::grouped && !SH::SWAP ? t.group : 0;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const uint32_t s = it % NS, bar = full + 8 * s, dst = base + s * SH::STAGE;
          if (it >= NS && !bar_wait_all(empty + 8 * s, (it / NS - 1) & 1, given_up)) {
            ok = false;
            break;
          }
          if (one_of_warp()) {
            bar_expect(bar, SH::STAGE);
            tma_load3(dst, &map_l, p.l.mn ? t.l0 : kb * kBlock, p.l.mn ? kb * kBlock : t.l0, gl, bar);
            const int c = PAIR ? t.c0 + rank * 128 : t.c0;
            tma_load3(dst + 16384, &map_c, p.c.mn ? c : kb * kBlock, p.c.mn ? kb * kBlock : c, gc, bar);
          }
        }
      }
      // The barriers outlive what arrives at them: the loads issued last, one stage each at most, or the MMAs of those (of a pair,
      // the first CTA's at the second's barriers).
      for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i)
        (void)(ok ? bar_wait_all(empty + 8 * (i % NS), (i / NS) & 1, given_up) : bar_wait(full + 8 * (i % NS), (i / NS) & 1));
    } else if (warp <= 2) {                              // two warps: of a pair one for either part of the columns, else for every other block
      if (rank == 0) {
        uint32_t it = 0;
        bool ok = true;
        const int mine = warp - 1, h = PAIR ? mine : 0;
        // a step of 32 of K, in 16 bytes; the parts' rows of C within each CTA's 128
        const uint32_t step_l = p.l.mn ? 256 : 2, step_c = p.c.mn ? 256 : 2, part_c = h * (p.c.mn ? 4 : 512);
        for (int tile = first_tile; tile < tiles && ok; tile += step) {
          const BlockTile t = tile_at<BN>(p, start, before, tile, rank);
          for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
            const uint32_t s = it % NS, buf = it % NB;
            if (!PAIR && (int)(it & 1) != mine) continue;
            ok = bar_wait_all((PAIR || p.kind == BlockKind::wgrad ? fixed : full) + 8 * s, (it / NS) & 1, given_up) &&
                 (it < NB || bar_wait_all(tempty + 8 * (buf * H + h), (it / NB - 1) & 1, given_up));
            if (!ok) break;
            tc_fence_after();
            if (one_of_warp()) {
              const uint64_t dl = desc8(base + s * SH::STAGE), dc = desc8(base + s * SH::STAGE + 16384) + part_c;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma8<PAIR>(tmem + buf * BN + h * (BN / H), dl + k * step_l, dc + k * step_c, p.idesc, k > 0);
              commit8<PAIR>(tfull + 8 * (buf * H + h), both);
              commit8<PAIR>(empty + 8 * s, both);
            }
          }
        }
        if (one_of_warp()) commit8<PAIR>(drained, both);
      }
      (void)bar_wait(drained, 0);                        // the MMAs are done, before the tensor memory goes back, at both CTAs of a pair
    } else if (warp == 3 && (PAIR || p.kind == BlockKind::wgrad)) {
      uint32_t it = 0;
      bool ok = true;
      const uint32_t ready = PAIR ? in_cluster(fixed, lead) : fixed;
      for (int tile = first_tile; tile < tiles && ok; tile += step) {
        const BlockTile t = tile_at<BN>(p, start, before, tile, rank);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const uint32_t s = it % NS;
          ok = __all_sync(0xFFFFFFFFu, bar_wait_all(full + 8 * s, (it / NS) & 1, given_up));
          if (!ok) break;
          const int first = t.lo - kb * kBlock, last = t.hi - kb * kBlock;   // of the block's rows, [first, last) count
          if (p.kind == BlockKind::wgrad && (first > 0 || last < kBlock)) {
            uint4* const rows = reinterpret_cast<uint4*>(smem + s * SH::STAGE);
            for (int i = lane; i < SH::STAGE / 16; i += 32) {
              const int r = (i >> 3) & 127;              // a token's codes of 128 rows are 128 bytes
              if (r < first || r >= last) rows[i] = make_uint4(0u, 0u, 0u, 0u);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            if (PAIR) fence_cluster();
          }
          __syncwarp();
          if (lane == 0) {
            if (PAIR) bar_arrive_cluster(ready + 8 * s);
            else bar_arrive(ready + 8 * s);
          }
        }
      }
    }
    __syncwarp();
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quad = warp & 3, half = (warp - 4) >> 2, mine = quad * 32 + lane;
    const uint32_t released = PAIR ? in_cluster(tempty, lead) : tempty;
    float* const cs = reinterpret_cast<float*>(smem + SH::CS) + (warp - 4) * 2 * OWN;   // this warp's columns' scales, twice
    constexpr int STEP = PAIR ? 1 : 2, NC = MODE == kScaleLane ? 1 : OWN / 32;            // a lane's scales of columns
    uint32_t it = 0;
    bool ok = true, met = false;
    // the scales of a block, asked for two of this warp's blocks ahead, by addresses that step from block to block; those of
    // a tile's first before the outputs of the tile before are written
    BlockTile t;
    const float *pl = nullptr, *pc = nullptr;
    bool r_in = false;
    int left = 0, c_at = 0;                              // blocks whose scales have not been asked for; a lane's first column
    // from one of a lane's columns to the next (a pair's 128 of a warp are within one block)
    const int64_t next_c = p.c.shift == 0 ? 32 * p.c.rs : 0;
    float rl0 = 0.0f, rl1 = 0.0f, rc0[NC] = {}, rc1[NC] = {};
    auto ask = [&](float& rl, float (&rc)[NC]) {
      rl = r_in && left > 0 ? __ldg(pl) : 0.0f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        rc[j] = left > 0 && c_at + 32 * j < t.c_end ? __ldg(PAIR ? pc + j * next_c : pc + ((c_at + 32 * j) >> p.c.shift) * p.c.rs) : 0.0f;
      pl += STEP * p.l.ks;
      pc += STEP * p.c.ks;
      left -= STEP;
    };
    auto begin = [&](int tile) {
      if (tile >= tiles) return;
      t = tile_at<BN>(p, start, before, tile, rank);
      const int gl = p.kind == BlockKind::grouped && SH::SWAP ? t.group : 0, gc = p.kind == BlockKind::grouped && !SH::SWAP ? t.group : 0;
      const int l_at = MODE == kScaleColumns ? t.l0 : t.l0 + mine, kb = t.kb0 + (PAIR ? 0 : (int)(it ^ half) & 1);
      r_in = l_at < t.l_end;
      c_at = t.c0 + (PAIR ? half * OWN : 0) + (MODE == kScaleLane ? 0 : lane);
      pl = p.l.scale + gl * p.l.gs + (l_at >> p.l.shift) * p.l.rs + kb * p.l.ks;
      pc = p.c.scale + gc * p.c.gs + kb * p.c.ks + (PAIR ? (c_at >> p.c.shift) * p.c.rs : 0);
      left = t.kb1 - kb;
      ask(rl0, rc0);
      ask(rl1, rc1);
    };
    begin(first_tile);
    uint32_t done = 0;                                   // tiles
    for (int tile = first_tile; tile < tiles && ok; tile += step, ++done) {
      const int l0 = t.l0, l_end = t.l_end, c = t.c0 + (PAIR ? half * OWN : 0), c_end = t.c_end, group = p.kind == BlockKind::wgrad ? t.group : 0;
      const int l = l0 + mine;
      const bool l_in = l < l_end;
      const int blocks = t.kb1 - t.kb0;
      f2 acc[OWN / 2];
#pragma unroll
      for (int i = 0; i < OWN / 2; ++i) acc[i] = 0ull;
      // Pieces of 32 columns.  Pairs: the next one is asked for before (of another part of the columns or block: while) one's
      // values are used, so that neither the barriers' latency nor the tensor memory's adds to the multiplications'
      // time (5760 x 1920 x 8192 with scales for squares 94 -> 88 us).  Narrow tiles: a block's all at once.
      constexpr int PIECES = OWN / 32, OF_PART = READ / 32;
      float r[2][32];
      auto full_of = [&](uint32_t unit, int h) { return tfull + 8 * (unit % NB * H + h); };
      auto ask_piece = [&](uint32_t unit, int k) {
        const int h = k / OF_PART;
        tmem_ask(tmem + ((uint32_t)(quad * 32) << 16) + unit % NB * BN + h * (BN / H) + (PAIR ? half * READ : 0) + k % OF_PART * 32,
                 r[k & 1]);
      };
      const int first = PAIR ? 0 : (int)(it ^ half) & 1;
      if (PAIR && first < blocks) {
        ok = __all_sync(0xFFFFFFFFu, bar_wait_all(full_of(it + first, 0), ((it + first) / NB) & 1, given_up));
        if (!ok) break;
        tc_fence_after();
        ask_piece(it + first, 0);
      }
      for (int kb = first; kb < blocks; kb += STEP) {
        const uint32_t unit = it + kb;
        const float rl = rl0;
        float rc[NC];
        rl0 = rl1;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          rc[j] = rc0[j];
          rc0[j] = rc1[j];
        }
        ask(rl1, rc1);
        float* const cv = cs + (unit / STEP & 1) * OWN;
        if (MODE != kScaleLane) {
#pragma unroll
          for (int j = 0; j < NC; ++j) cv[32 * j + lane] = MODE == kScaleColumns ? rl * rc[j] : rc[j];
          __syncwarp();
        }
        const float one = MODE == kScaleLane ? rl * rc[0] : rl;
        const f2 by = pair(one, one);
        auto use = [&](int k, int from, int to) {
          const float* const v = r[k & 1];
#pragma unroll
          for (int i = from; i < to; i += 4) {
            f2& a0 = acc[(k * 32 + i) / 2];
            f2& a1 = acc[(k * 32 + i) / 2 + 1];
            if (MODE == kScaleLane) {
              add_scaled(a0, v[i], v[i + 1], by);
              add_scaled(a1, v[i + 2], v[i + 3], by);
            } else {
              const float4 s = *reinterpret_cast<const float4*>(cv + k * 32 + i);
              if (MODE == kScaleColumns) {               // both: one scale after the other (their product first: 152 us instead of 139)
                add_scaled(a0, v[i], v[i + 1], pair(s.x, s.y));
                add_scaled(a1, v[i + 2], v[i + 3], pair(s.z, s.w));
              } else {
                a0 = fma2(scaled(v[i], v[i + 1], by), pair(s.x, s.y), a0);
                a1 = fma2(scaled(v[i + 2], v[i + 3], by), pair(s.z, s.w), a1);
              }
            }
          }
        };
        auto release = [&](int h) {                      // the part has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR) bar_arrive_cluster(released + 8 * (unit % NB * H + h));
            else bar_arrive(released + 8 * (unit % NB * H + h));
          }
        };
        if constexpr (PAIR) {
#pragma unroll
          for (int k = 0; k < PIECES; ++k) {
            tmem_wait();
            if ((k + 1) % OF_PART != 0) {
              ask_piece(unit, k + 1);
              use(k, 0, 32);
              continue;
            }
            release(k / OF_PART);
            const bool last = k + 1 == PIECES, more = !last || kb + STEP < blocks;
            const uint32_t next = last ? unit + STEP : unit, bar = full_of(next, last ? 0 : (k + 1) / OF_PART), parity = (next / NB) & 1;
            const bool there = more && bar_try(bar, parity);
            use(k, 0, 16);
            if (more) {
              ok = __all_sync(0xFFFFFFFFu, there || bar_wait_all(bar, parity, given_up));
              if (!ok) break;
              tc_fence_after();
              ask_piece(next, last ? 0 : k + 1);
            }
            use(k, 16, 32);
          }
        } else {
          ok = __all_sync(0xFFFFFFFFu, bar_wait_all(full_of(unit, 0), (unit / NB) & 1, given_up));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < PIECES; ++k) ask_piece(unit, k);
          tmem_wait();
          release(0);
#pragma unroll
          for (int k = 0; k < PIECES; ++k) use(k, 0, 32);
        }
        if (!ok) break;
      }
      if (!ok) break;
      it += blocks;
      begin(tile + step);
      if constexpr (!SH::SWAP) {
        unsigned char* const stage = smem + SH::OUT + (warp - 4) * (kOutStage / 8);
        if (p.slices > 1) {
          // two slices: each adds up one half of the columns.  The other half's sums go to its place, behind where they are
          // written here, once all are past their last MMA.
          cluster_sync();
          met = true;
          float4* const sums = reinterpret_cast<float4*>(smem) + mine;   // [32][128][4]
          if (half != (lead >> 1)) {
#pragma unroll
            for (int i = 0; i < OWN / 4; ++i) sums[i * 128] = four_of(acc[2 * i], acc[2 * i + 1]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            const uint32_t at = (lane * 128 + quad * 32) * 16, other = (lead ^ 2) + rank;
            send(in_cluster(base + OWN * 128 * 4 + at, other), base + at, 32 * 16, in_cluster(met_all, other));
            continue;
          }
          ok = __all_sync(0xFFFFFFFFu, bar_wait_all(met_all, 0, given_up));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < OWN / 4; ++i) {
            const float4 v = sums[(OWN / 4 + i) * 128];
            acc[2 * i] = add2(acc[2 * i], pair(v.x, v.y));
            acc[2 * i + 1] = add2(acc[2 * i + 1], pair(v.z, v.w));
          }
        }
        const int row0 = l0 + quad * 32, rows = l_end - row0 < 32 ? l_end - row0 : 32;
        if (p.out_type == EMU_OUT_F32) write_rows<float>(p, &map_out, acc, stage, row0, rows, c, group, lane);
        else if (p.out_type == EMU_OUT_BF16) write_rows<__nv_bfloat16>(p, &map_out, acc, stage, row0, rows, c, group, lane);
        else write_rows<__half>(p, &map_out, acc, stage, row0, rows, c, group, lane);
      } else {
        {                                                // the second four warps' sums join the first four's
          float4* const sums = reinterpret_cast<float4*>(smem + SH::OUT) + mine;
          if (half == 1) {
            ok = __all_sync(0xFFFFFFFFu, done == 0 || bar_wait_all(parted + 8 * quad, (done - 1) & 1, given_up));
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < OWN / 4; ++i) sums[i * 128] = four_of(acc[2 * i], acc[2 * i + 1]);
            __syncwarp();
            if (lane == 0) bar_arrive(joined + 8 * quad);
            continue;
          }
          ok = __all_sync(0xFFFFFFFFu, bar_wait_all(joined + 8 * quad, done & 1, given_up));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < OWN / 4; ++i) {
            const float4 v = sums[i * 128];
            acc[2 * i] = add2(acc[2 * i], pair(v.x, v.y));
            acc[2 * i + 1] = add2(acc[2 * i + 1], pair(v.z, v.w));
          }
          __syncwarp();
          if (lane == 0) bar_arrive(parted + 8 * quad);
          if (p.slices > 1) {
            // slice s adds up columns s BN / S on: every slice sends its sums of them there, in the place of that CTA's operands,
            // [S][BN / S / 4][128][4], once all are past their last MMA
            __syncwarp();
#pragma unroll
            for (int i = 0; i < OWN / 4; ++i) sums[i * 128] = four_of(acc[2 * i], acc[2 * i + 1]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            cluster_sync();
            met = true;
            const int per = OWN / 4 / p.slices, slice = tile % p.slices;        // groups of four columns
            if (lane < OWN / 4)
              send(in_cluster(base + ((slice * per + lane % per) * 128 + quad * 32) * 16, lane / per),
                   smem_addr(smem + SH::OUT) + (lane * 128 + quad * 32) * 16, 32 * 16, in_cluster(met_all, lane / per));
            continue;
          }
        }
        auto write = [&](auto* out) {
          using T = std::remove_pointer_t<decltype(out)>;
          T* const to = out + group * p.out_group + l * p.ldl;
#pragma unroll
          for (int i = 0; i < OWN; i += 2) {
            float a, b;
            halves(acc[i / 2], a, b);
            if (l_in && c + i < c_end) to[(c + i) * p.ldc] = from_f<T>(a);
            if (l_in && c + i + 1 < c_end) to[(c + i + 1) * p.ldc] = from_f<T>(b);
          }
        };
        if (p.out_type == EMU_OUT_F32) write(static_cast<float*>(p.out));
        else if (p.out_type == EMU_OUT_BF16) write(static_cast<__nv_bfloat16*>(p.out));
        else write(static_cast<__half*>(p.out));
      }
    }
    if (p.kind == BlockKind::grouped && p.zero_rest) {
      const int64_t N = SH::SWAP ? p.l.rows : p.c.rows, who = (int64_t)blockIdx.x * 256 + tid - 128, count = (int64_t)gridDim.x * 256;
      put_zeros(p.out, p.out_type, 0, start[0] * N, who, count);
      put_zeros(p.out, p.out_type, start[p.E] * N, (int64_t)p.T * N, who, count);
    }
    if (PAIR && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // before the memory is gone
    __syncwarp();
    if (p.slices > 1 && !met) cluster_sync();   // a warp that gave up goes past the first barrier too
  }
  if (p.slices > 1 && warp < 4) cluster_sync();
  if constexpr (SH::SWAP) {
    if (p.slices > 1) {                                  // one tile a CTA
      const BlockTile t = tile_at<BN>(p, start, before, blockIdx.x, 0);
      const int per = OWN / 4 / p.slices, slice = (int)blockIdx.x % p.slices;
      const float4* const sums = reinterpret_cast<const float4*>(smem);
      if (bar_wait_all(met_all, 0, given_up))
        for (int i = tid; i < per * 128; i += kTcThreads8) {
          float4 v = sums[i];
          for (int s = 1; s < p.slices; ++s) {
            const float4 w = sums[s * per * 128 + i];
            v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
          }
          const int l = t.l0 + i % 128, c = t.c0 + (slice * per + i / 128) * 4;
          const float each[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (l < t.l_end && c + j < t.c_end) put(p.out, p.out_type, l * p.ldl + (c + j) * p.ldc, each[j]);
        }
      __syncwarp();
      cluster_sync();                                    // what was sent has been read
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();                              // the first CTA's MMAs and the other's arrivals are over
  tc_fence_after();
  if (tid == 0 && *given_up) atomicExch(&g_block_status, 1);
  if (warp == 2) tmem_free<PAIR>(tmem, SH::TMEM);
}

}  // namespace emu_ops
