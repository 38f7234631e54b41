// ops_int8_tc.cuh -- the int8 product on the 5th-generation tensor cores.
//
// sm_103a's tcgen05 has no int8 kind (and mma.sync on int8 runs at the rate of the dp4a
// instruction, 75 TMAC/s measured), but a code is exact in fp16, a product of two is at most
// 2^14 in magnitude, and 1024 of them sum exactly in the fp32 accumulator: every partial sum is
// a whole number of at most 2^24.  So the codes are multiplied as fp16 by tcgen05.mma
// kind::f16, and after every 1024 of K the accumulator is read back and added up in 32-bit
// integers.  Two kernels: for many tokens, operands laid out as fp16 by a kernel before and
// loaded by TMA; for few, codes converted on the way into shared memory, and K in slices.
#pragma once
#include "ops_common.cuh"

namespace emu_ops {

constexpr int kTcBM = 128, kTcBN = 256, kTcBK = 64, kTcNS = 4;
constexpr int kTcChunk = 1024 / kTcBK;                       // K blocks that one accumulator takes
constexpr int kTcStage = (kTcBM + kTcBN) * kTcBK * 2;        // 48 KB
constexpr int kTcStageRow = 128;                             // bytes of a staged output row
constexpr int kTcOut = kTcNS * kTcStage;                     // eight warps' staging, 32 rows each
constexpr int kTcBars = kTcOut + 8 * 32 * kTcStageRow;
constexpr int kTcSmem = kTcBars + 128 + 1024;                // and what aligning to 1024 may take
static_assert(kTcSmem <= 227 * 1024, "one CTA an SM");
constexpr int kTcThreads = 384;

struct TcTiles {
  int tiles_m, tiles_n, k_blocks;
  // eight rows of tiles at a time, column by column, so that the CTAs at work share both operands' rows
  // (4096^3: 107 us with all rows at a time, 103 with eight)
  __device__ __forceinline__ void at(int tile, int& m, int& n) const {
    const int group = tile / (8 * tiles_n), first = group * 8, rows = tiles_m - first < 8 ? tiles_m - first : 8;
    const int in = tile - group * 8 * tiles_n;
    m = first + in % rows;
    n = in / rows;
  }
};

// ---- TMA and tcgen05 (inline PTX)
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
// shared-memory matrix descriptor: K-major rows of 128 bytes under the 128-byte swizzle, groups of
// eight rows 1024 bytes apart
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// instruction descriptor of kind::f16: fp16 operands, both K-major, fp32 accumulator
__device__ __forceinline__ uint32_t tc_idesc(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tc_read32(uint32_t addr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr)
      : "memory");
}

// ---------------------------------------------------------------------------------------
// Up to a few hundred tokens, where reading B and the latency of each step count.  A CTA takes 128
// columns of B (the M side of the MMA) by BT tokens (its N side) and one of S slices of K.  Eight
// warps load codes straight into registers, some stages of 128 of K ahead, convert them and store
// them as K-major fp16 rows under the 128-byte swizzle in one of two buffers; a ninth issues the
// eight MMAs of a stage (issuing them takes as long as they run, about 740 cycles at 64 tokens, so
// a converting warp would hold the others up).  The S slices are the CTAs of a cluster and
// share out the tile's tokens: each sends the others its integer sums of theirs.
// (The same on mma.sync, each warp converting its own fragments, took 13.4 us for
// 64 x 5760 x 1920: six times the instructions, as fragments are converted again by each warp.)
constexpr int kMaxSlices = 8, kFixedStages = 4;
template <int BT> struct FewShape {
  static constexpr int ROWS = 128 + BT, ATOM = ROWS * 128, STAGE = 2 * ATOM;   // an atom: 64 of K
  static constexpr int PIECES = (ROWS * 8 + 255) / 256;                        // of 16 codes, a thread
  static constexpr int SMEM = 2 * STAGE + 1024;
  static constexpr int RESIDENT = 228 * 1024 / (SMEM + 2048) < 2 ? 1 : 2;      // CTAs an SM
  static constexpr int COLS = BT < 32 ? 32 : BT;                               // of tensor memory
  static constexpr int OWN = BT < 32 ? 16 : BT / 2;                            // tokens a thread reads back
  static constexpr int AHEAD = BT < 64 ? 3 : 2;                                // stages in registers
  static_assert(BT * 128 * 4 <= 2 * STAGE, "the sums take the buffers' place");
};

template <int N> __device__ __forceinline__ void tc_read(uint32_t addr, float (&r)[N]) {
  if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\ntcgen05.wait::ld.sync.aligned;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(addr)
        : "memory");
  } else {
    tc_read32(addr, r);
  }
}

// LONG: slices of more than eight stages, whose sums are taken out of the tensor memory every 1024 of K
constexpr int kFewThreads = 288;
template <int BT, bool LONG, bool VEC>
__global__ void __launch_bounds__(kFewThreads, FewShape<BT>::RESIDENT)
int8_few_kernel(const Int8Params p, int S) {
  using SH = FewShape<BT>;
  constexpr int PP = SH::PIECES, AHEAD = VEC ? SH::AHEAD : 1, STEP = SH::OWN < 32 ? 16 : 32;
  extern __shared__ unsigned char raw_smem[];
  __shared__ __align__(8) uint64_t bars[5];                 // full[2], empty[2], read (sums taken)
  __shared__ uint32_t slot;
  __shared__ int gave_up;
  unsigned char* const smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem), full = smem_addr(bars), empty = full + 16, taken = full + 32;
  volatile int* const given_up = &gave_up;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t slice = blockIdx.x % (uint32_t)S;
  const int64_t n0 = (int64_t)(blockIdx.x / (uint32_t)S) * 128, m0 = (int64_t)blockIdx.y * BT;
  const uint32_t all = (uint32_t)(p.K + 127) / 128, first = all * slice / (uint32_t)S;
  const int count = (int)(all * (slice + 1) / (uint32_t)S - first);     // stages of 128 codes
  // piece i of a thread: codes 16 c8 to 16 c8 + 15 of a stage, of row r8 + 32 i (B's 128 rows, then tokens)
  const int c8 = tid & 7, r8 = (tid & 255) >> 3;
  const int8_t* at[PP];
  Codes<VEC> w[AHEAD][PP];
  auto first_of = [&](int st) { return (int)(first + st) * 128 + c8 * 16; };
  auto load = [&](int st, Codes<VEC> (&v)[PP]) {
    const int k = first_of(st);
    const bool in = st < count && k < p.K;
#pragma unroll
    for (int i = 0; i < PP; ++i) v[i].ask(at[i], k, in && at[i], i < 4 ? p.b : p.a, i < 4 ? p.b_end : p.a_end);
  };
  if (warp < 8) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int64_t r = i < 4 ? n0 + r8 + 32 * i : m0 + r8 + 32 * (i - 4);
      const bool in = r < (i < 4 ? p.N : p.M) && (i < 4 || r8 + 32 * (i - 4) < BT);
      at[i] = in ? (i < 4 ? p.b + r * p.ldb : p.a + r * p.lda) : nullptr;
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(u, w[u]);
  } else {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        bar_init(full + 8 * i, 8);                          // one arrival a converting warp
        bar_init(empty + 8 * i, 1);                         // a stage's MMAs
      }
      bar_init(taken, 8);
      gave_up = 0;
      bar_init_fence();
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&slot)), "r"(SH::COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = slot;
  // the tokens of a lane (a column of B): half of them for each four warps; of 16, warps 4 to 7 read none
  const int quad = warp & 3, t0 = BT < 32 ? 0 : (warp >> 2) * SH::OWN;
  const bool reads = warp < (BT >= 32 ? 8 : 4);
  int sum[SH::OWN];
  if (LONG) {
#pragma unroll
    for (int i = 0; i < SH::OWN; ++i) sum[i] = 0;
  }
  bool ok = true;
  if (warp == 8) {
    if (lane == 0) {
      int st = 0;
      for (; st < count && ok; ++st) {
        if (LONG && (st & 7) == 0 && st > 0) ok = bar_wait_all(taken, ((st >> 3) - 1) & 1, given_up);   // 1024 products a sum
        ok = ok && bar_wait_all(full + 8 * (st & 1), (st >> 1) & 1, given_up);
        if (!ok) break;
        tc_fence_after();
        const uint32_t buf = base + (st & 1) * SH::STAGE;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t atom = buf + (k >> 2) * SH::ATOM;
          tc_mma(tmem, tc_desc(atom) + 2 * (k & 3), tc_desc(atom + 128 * 128) + 2 * (k & 3), tc_idesc(128, BT),
                 k > 0 || (LONG ? (st & 7) != 0 : st > 0));
        }
        tc_commit(empty + 8 * (st & 1));
      }
      if (!ok)                                              // the MMAs issued end before their memory is given back
        for (int i = st > 2 ? st - 2 : 0; i < st; ++i) (void)bar_wait(empty + 8 * (i & 1), (i >> 1) & 1);
    }
    __syncwarp();
  } else {
    auto take = [&](int st) {                               // stage st and all before it are multiplied: their sums
      ok = __all_sync(0xFFFFFFFFu, bar_wait_all(empty + 8 * (st & 1), (st >> 1) & 1, given_up));
      if (!ok) return;
      tc_fence_after();
      if (reads) {
#pragma unroll
        for (int c = 0; c < SH::OWN; c += STEP) {
          float r[STEP];
          tc_read<STEP>(tmem + ((uint32_t)(quad * 32) << 16) + t0 + c, r);
#pragma unroll
          for (int i = 0; i < STEP; ++i) sum[c + i] = (LONG ? sum[c + i] : 0) + __float2int_rn(r[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (LONG && lane == 0) bar_arrive(taken);
    };
    for (int s0 = 0; s0 < count && ok; s0 += AHEAD) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int st = s0 + u;
        if (st >= count || !ok) break;
        if (st >= 2) {                                      // its buffer has been read
          ok = __all_sync(0xFFFFFFFFu, bar_wait_all(empty + 8 * (st & 1), ((st >> 1) - 1) & 1, given_up));
          if (!ok) break;
        }
        unsigned char* const buf = smem + (st & 1) * SH::STAGE + (c8 >> 2) * SH::ATOM;
#pragma unroll
        for (int i = 0; i < PP; ++i) {
          const int row = r8 + 32 * i;
          if (PP * 32 != SH::ROWS && row >= SH::ROWS) break;
          const uint4 q = w[u][i].get(at[i], first_of(st), p.K, first_of(st) < p.K && at[i], i < 4 ? p.b : p.a,
                                      i < 4 ? p.b_end : p.a_end);
          uint32_t h[8];
          codes_to_f16(q.x, h[0], h[1]);
          codes_to_f16(q.y, h[2], h[3]);
          codes_to_f16(q.z, h[4], h[5]);
          codes_to_f16(q.w, h[6], h[7]);
          const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
          // the two atoms' chunks share banks: their threads store odd and even chunks in turn
          const int odd = c8 >> 2, chunk = (c8 & 3) * 2;
          *reinterpret_cast<uint4*>(buf + row * 128 + (((chunk + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(buf + row * 128 + (((chunk + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(full + 8 * (st & 1));
        load(st + AHEAD, w[u]);
        if (LONG && (st & 7) == 7 && st + 1 < count) take(st);
      }
    }
    if (ok && count > 0) take(count - 1);
  }
  __syncthreads();
  if (S > 1) cluster_arrive();
  if (tid == 0 && *given_up) atomicExch(&g_ops_status, 1);
  tc_fence_after();
  if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(SH::COLS) : "memory");

  const int nl = quad * 32 + lane;
  if (S == 1) {
    const int64_t n = n0 + nl;
    if (!reads) return;                                     // whole warps
    const float sb = n < p.N ? scale_b(p, n) : 0.0f;
    float sa[(SH::OWN + 31) / 32];                            // of token lane, lane + 32: asked for at once
#pragma unroll
    for (int i = 0; i < SH::OWN; i += 32) {
      const int64_t m = m0 + t0 + i + lane;
      sa[i / 32] = i + lane < SH::OWN && m < p.M ? scale_a(p, m) : 0.0f;
    }
    auto write = [&](auto* out) {
      using T = std::remove_pointer_t<decltype(out)>;
#pragma unroll
      for (int i = 0; i < SH::OWN; ++i) {
        const int64_t m = m0 + t0 + i;
        const float v = ((float)sum[i] * __shfl_sync(0xFFFFFFFFu, sa[i / 32], i % 32)) * sb;
        if (m < p.M && n < p.N) out[m * p.N + n] = from_f<T>(v);
      }
    };
    if (p.out_type == EMU_OUT_F32) write(static_cast<float*>(p.out));
    else if (p.out_type == EMU_OUT_BF16) write(static_cast<__nv_bfloat16*>(p.out));
    else write(static_cast<__half*>(p.out));
    return;
  }
  // slice s adds up the tokens s, s + S, ...: every slice writes its sums of them there, once that CTA is
  // past its last MMA, and each then finds all it needs in its own shared memory, [S][slots][128]
  int* const sums = reinterpret_cast<int*>(smem);
  const int slots = (BT + S - 1) / S;
  const bool together = stores_together<4>(p);
  const int64_t n = n0 + (tid * 4) % 128;                   // a thread's four columns
  float sb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sb[j] = n + j < p.N ? scale_b(p, n + j) : 0.0f;
  float sa[BT < 64 ? 1 : 2];                                // of its lane-th token, its lane + 32-th
#pragma unroll
  for (int i = 0; i < (BT < 64 ? 1 : 2); ++i) {
    const int q = i * 32 + lane;
    const int64_t m = m0 + (int64_t)q * S + slice;
    sa[i] = q < slots && m < p.M ? scale_a(p, m) : 0.0f;
  }
  cluster_wait();
  if (reads) {
    int owner = t0 % S, slot_of = t0 / S;
#pragma unroll
    for (int i = 0; i < SH::OWN; ++i) {
      asm volatile("st.shared::cluster.s32 [%0], %1;"
                   ::"r"(in_cluster(sums + ((int)slice * slots + slot_of) * 128 + nl, owner)), "r"(sum[i]) : "memory");
      if (++owner == S) {
        owner = 0;
        ++slot_of;
      }
    }
  }
  cluster_sync();
  for (int q = tid / 32; tid < 256 && q * S + (int)slice < BT; q += 8) {
    const int64_t m = m0 + q * S + slice;
    if (m >= p.M) break;
    const float of_token = __shfl_sync(0xFFFFFFFFu, BT >= 64 && q >= 32 ? sa[BT >= 64] : sa[0], q % 32);
    int v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < kMaxSlices; ++r)
      if (r < S) {
        const int4 x = *reinterpret_cast<const int4*>(sums + (r * slots + q) * 128 + lane * 4);
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
      }
    store_row<4>(p, m, n, v, of_token, sb, together);
  }
}

// ---------------------------------------------------------------------------------------
// For many tokens.  Codes to fp16 rows of 16 `chunks` values, zeros after the K-th: rows_a rows of A from row
// m on, then rows_b of B from row n on.  A thread takes 16 codes.
template <bool VEC>
__global__ void __launch_bounds__(256)
int8_to_f16_kernel(const Int8Params p, int64_t m, uint32_t rows_a, uint16_t* a16, int64_t n, uint32_t rows_b, uint16_t* b16,
                   uint32_t chunks) {
  const uint32_t total = (rows_a + rows_b) * chunks;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product waits for this kernel's end
  for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < total; i += gridDim.x * 256u) {
    const uint32_t row = i / chunks, c = i - row * chunks;
    const bool is_a = row < rows_a;
    const uint32_t r = is_a ? row : row - rows_a;
    const int k = (int)c * 16;
    const int8_t* const row_at = is_a ? p.a + (m + r) * p.lda : p.b + (n + r) * p.ldb;
    const int8_t* const from = is_a ? p.a : p.b;
    const uintptr_t end = is_a ? p.a_end : p.b_end;
    Codes<VEC> codes;
    codes.ask(row_at, k, k < p.K, from, end);
    const uint4 q = codes.get(row_at, k, p.K, k < p.K, from, end);
    uint4* dst = reinterpret_cast<uint4*>((is_a ? a16 : b16) + (size_t)r * chunks * 16 + (size_t)c * 16);
    uint32_t h[8];
    codes_to_f16(q.x, h[0], h[1]);
    codes_to_f16(q.y, h[2], h[3]);
    codes_to_f16(q.z, h[4], h[5]);
    codes_to_f16(q.w, h[6], h[7]);
    dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
    dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// A warp's 32 rows x 128 columns of sums, a row a lane, scaled and written out: 128 bytes of each row at a
// time go through shared memory (16 bytes a lane, a row's chunks permuted by its number: no two lanes of a
// phase meet in a bank), so that whole lines are stored, or, where rows are not 16-byte aligned, elements.
// sb: scale_b of columns lane, lane + 32, ...
template <class T>
__device__ __forceinline__ void write_tile(const Int8Params& p, const int (&sum)[128], const float (&sb)[4], float sa,
                                           unsigned char* stage, int64_t m0, int64_t n0, int lane) {
  constexpr int COLS = 128 / sizeof(T), VEC = 16 / sizeof(T);
  const int rows = p.M - m0 < 32 ? (int)(p.M - m0) : 32;
  T* const out = static_cast<T*>(p.out);
  const bool vec = p.N % VEC == 0 && p.cols % VEC == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll
  for (int c = 0; c < 128; c += COLS) {
    const int64_t nc = n0 + c;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < COLS; i += VEC) {
      float v[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int n = c + i + j;
        v[j] = ((float)sum[n] * sa) * __shfl_sync(0xFFFFFFFFu, sb[n / 32], n % 32);
      }
      store_f<T, VEC>(reinterpret_cast<T*>(stage + lane * kTcStageRow + (((i / VEC) ^ (lane & 7)) * 16)), v);
    }
    __syncwarp();
    if (vec) {
      const int64_t n = nc + (lane & 7) * VEC;
      if (n < p.cols) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = k * 4 + (lane >> 3);
          if (r < rows)
            *reinterpret_cast<uint4*>(out + (m0 + r) * p.N + n) =
                *reinterpret_cast<const uint4*>(stage + r * kTcStageRow + (((lane & 7) ^ (r & 7)) * 16));
        }
      }
    } else {
      const unsigned char* from = stage + (lane % VEC) * sizeof(T);
      const int chunk = lane / VEC * 16;
      T* to = out + m0 * p.N + nc + lane;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8, from += 8 * kTcStageRow) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {                   // four rows' values asked for at once
          T v[4][COLS / 32];
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < COLS / 32; ++i)
              v[r][i] = *reinterpret_cast<const T*>(from + (h + r) * kTcStageRow + (chunk ^ ((i * 32 / VEC ^ (h + r)) * 16)));
#pragma unroll
          for (int r = 0; r < 4; ++r, to += p.N)
#pragma unroll
            for (int i = 0; i < COLS / 32; ++i)
              if (r0 + h + r < rows && nc + i * 32 + lane < p.cols) to[i * 32] = v[r][i];
        }
      }
    }
  }
}

// Persistent: one CTA an SM, tiles of 128 x 256 outputs in turn.  Warp 0 loads the stages by TMA,
// warp 1 issues the MMAs, warp 2 owns the tensor memory, warps 4 to 11 read the accumulators
// back: each holds 32 rows x 128 columns of sums in registers.  All waits are bounded; a role that
// gives up sets the status and takes the others along.  8192 x 5760 x 1920 in 109 us, 85% of the
// measured bf16 rate of the library's product; the tensor pipe is active 69% of the time.
__global__ void __launch_bounds__(kTcThreads, 1)
int8_tc_kernel(const Int8Params p, const TcTiles tl, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b) {
  extern __shared__ unsigned char raw[];
  unsigned char* const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_addr(smem);
  const uint32_t full = base + kTcBars, empty = full + 8 * kTcNS, tfull = empty + 8 * kTcNS, tempty = tfull + 16,
                 drained = tempty + 16;
  uint32_t* const slot = reinterpret_cast<uint32_t*>(smem + kTcBars + 8 * (2 * kTcNS + 5));
  volatile int* const given_up = reinterpret_cast<volatile int*>(slot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < kTcNS; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(tfull + 8 * i, 1);
      bar_init(tempty + 8 * i, 8);                // one arrival a reading warp
    }
    bar_init(drained, 1);
    *given_up = 0;
    bar_init_fence();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const int tiles = tl.tiles_m * tl.tiles_n;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");       // the operands are laid out
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        int tm, tn;
        tl.at(tile, tm, tn);
        const int m0 = tm * kTcBM, n0 = tn * kTcBN;
        for (int kb = 0; kb < tl.k_blocks; ++kb, ++it) {
          const uint32_t s = it % kTcNS, bar = full + 8 * s, dst = base + s * kTcStage;
          if (it >= kTcNS && !bar_wait_all(empty + 8 * s, (it / kTcNS - 1) & 1, given_up)) {
            ok = false;
            break;
          }
          bar_expect(bar, kTcStage);
          tma_load(dst, &map_a, kb * kTcBK, m0, bar);
          tma_load(dst + kTcBM * kTcBK * 2, &map_b, kb * kTcBK, n0, bar);
        }
      }
      if (!ok)                                    // the loads issued last, one a stage at most
        for (uint32_t i = it > kTcNS ? it - kTcNS : 0; i < it; ++i) (void)bar_wait(full + 8 * (i % kTcNS), (i / kTcNS) & 1);
    } else if (warp == 1 && lane == 0) {
      const uint32_t idesc = tc_idesc(kTcBM, kTcBN);
      uint32_t it = 0, unit = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        for (int k0 = 0; k0 < tl.k_blocks && ok; k0 += kTcChunk, ++unit) {
          const uint32_t buf = unit & 1;
          if (unit >= 2 && !bar_wait_all(tempty + 8 * buf, ((unit >> 1) - 1) & 1, given_up)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int k1 = k0 + kTcChunk < tl.k_blocks ? k0 + kTcChunk : tl.k_blocks;
          for (int kb = k0; kb < k1; ++kb, ++it) {
            const uint32_t s = it % kTcNS;
            if (!bar_wait_all(full + 8 * s, (it / kTcNS) & 1, given_up)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = tc_desc(base + s * kTcStage), db = tc_desc(base + s * kTcStage + kTcBM * kTcBK * 2);
#pragma unroll
            for (int k = 0; k < kTcBK / 16; ++k)
              tc_mma(tmem + buf * 256, da + 2 * k, db + 2 * k, idesc, kb > k0 || k > 0);
            tc_commit(empty + 8 * s);
          }
          if (ok) tc_commit(tfull + 8 * buf);
        }
      }
      tc_commit(drained);                         // the MMAs are done before the tensor memory goes back
      (void)bar_wait(drained, 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quad = warp & 3, half = (warp - 4) >> 2;
    unsigned char* const stage = smem + kTcOut + (warp - 4) * 32 * kTcStageRow;
    uint32_t unit = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
      int tm, tn;
      tl.at(tile, tm, tn);
      const int64_t m0 = (int64_t)tm * kTcBM + quad * 32;
      const int64_t n0 = (int64_t)tn * kTcBN + half * 128;
      const float sa = m0 + lane < p.M ? scale_a(p, m0 + lane) : 0.0f;
      float sb[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) sb[c] = n0 + c * 32 + lane < p.cols ? scale_b(p, n0 + c * 32 + lane) : 0.0f;
      int sum[128];
      for (int k0 = 0; k0 < tl.k_blocks; k0 += kTcChunk, ++unit) {
        const uint32_t buf = unit & 1;
        ok = __all_sync(0xFFFFFFFFu, bar_wait_all(tfull + 8 * buf, (unit >> 1) & 1, given_up));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float r[32];
          tc_read32(tmem + ((uint32_t)(quad * 32) << 16) + buf * 256 + half * 128 + c * 32, r);
          if (k0 == 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c * 32 + i] = __float2int_rn(r[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c * 32 + i] += __float2int_rn(r[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(tempty + 8 * buf);
      }
      if (!ok) break;
      if (p.out_type == EMU_OUT_F32) write_tile<float>(p, sum, sb, sa, stage, m0, n0, lane);
      else if (p.out_type == EMU_OUT_BF16) write_tile<__nv_bfloat16>(p, sum, sb, sa, stage, m0, n0, lane);
      else write_tile<__half>(p, sum, sb, sa, stage, m0, n0, lane);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *given_up) atomicExch(&g_ops_status, 1);
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace emu_ops
