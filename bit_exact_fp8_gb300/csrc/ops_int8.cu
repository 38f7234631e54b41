// ops_int8.cu -- the product of 8-bit integers with a scale for each token (row of A) and
// each channel (column of B), declared in include/emu_fp8.h:
//   out[m, n] = (fp32(sum_k A[m, k] B[k, n]) * scale_a[m]) * scale_b[n]
// The sum is exact in 32-bit integers, so the result does not depend on the order or the
// kernel that took it.
#include "ops_common.cuh"

#include <cuda.h>             // CUtensorMap (the type only; the driver is called through an entry point)
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#include <type_traits>

namespace emu_ops {

// 1 once a bounded wait of the pipeline gave up (the outputs of that call are not valid)
__device__ int g_ops_status = 0;

constexpr int64_t kInt8MaxK = 131071;             // K * 128 * 128 < 2^31

struct Int8Params {
  const int8_t* a; int64_t lda;                   // [M, K]
  const int8_t* b; int64_t ldb;                   // [N, K]
  uintptr_t a_end, b_end;                         // where their memory ends
  int64_t M, N;                                   // N: also the output's row stride
  int64_t cols;                                   // columns of B here (a slab of the N)
  int K;
  const float* scale_a; int sa_step;              // 0: one scale for all
  const float* scale_b; int sb_step;
  void* out; int out_type;                        // [M, N] contiguous
};

// the scales by the read-only path, so that their loads need not wait for the stores before them
__device__ __forceinline__ float scale_a(const Int8Params& p, int64_t m) { return __ldg(p.scale_a + m * p.sa_step); }
__device__ __forceinline__ float scale_b(const Int8Params& p, int64_t n) { return __ldg(p.scale_b + n * p.sb_step); }
__device__ __forceinline__ void store_out(const Int8Params& p, int64_t m, int64_t n, int acc, float sa, float sb) {
  const float v = ((float)acc * sa) * sb;
  const int64_t i = m * p.N + n;
  if (p.out_type == EMU_OUT_F32) static_cast<float*>(p.out)[i] = v;
  else if (p.out_type == EMU_OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p.out)[i] = __float2half_rn(v);
}
// outputs (m, n) to (m, n + N - 1), of which the matrix may have fewer; `together`: it has all or none of
// them, and they can be stored at once
template <int N>
__device__ __forceinline__ void store_row(const Int8Params& p, int64_t m, int64_t n, const int (&acc)[N], float sa,
                                          const float (&sb)[N], bool together) {
  if (m >= p.M || n >= p.N) return;
  if (together) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ((float)acc[i] * sa) * sb[i];
    const int64_t at = m * p.N + n;
    if (p.out_type == EMU_OUT_F32) store_f<float, N>(static_cast<float*>(p.out) + at, v);
    else if (p.out_type == EMU_OUT_BF16) store_f<__nv_bfloat16, N>(static_cast<__nv_bfloat16*>(p.out) + at, v);
    else store_f<__half, N>(static_cast<__half*>(p.out) + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (n + i < p.N) store_out(p, m, n + i, acc[i], sa, sb[i]);
  }
}
template <int N> __device__ __forceinline__ bool stores_together(const Int8Params& p) {
  const uintptr_t es = p.out_type == EMU_OUT_F32 ? 4 : 2;
  return p.N % N == 0 && (reinterpret_cast<uintptr_t>(p.out) & (N * es - 1)) == 0;
}

// 16 bytes of the 32 in a and b, from the at-th on (0 to 16)
__device__ __forceinline__ uint4 bytes_from(const uint4& a, const uint4& b, int at) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t x[6], y[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = at & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) y[i] = at & 4 ? x[i + 1] : x[i];
  const uint32_t shift = (uint32_t)(at & 3) * 8;
  if (at == 16) return b;
  return make_uint4(__funnelshift_r(y[0], y[1], shift), __funnelshift_r(y[1], y[2], shift),
                    __funnelshift_r(y[2], y[3], shift), __funnelshift_r(y[3], y[4], shift));
}

// 16 codes of a row from the k-th on, zeros after the K-th, in two steps, so that a thread's loads are all
// asked for before the first is waited for.  Rows that are 16-byte aligned (VEC): one load.  Else the two
// 16-byte words that the codes touch, as far as these lie within the operand's memory (`from` to `end`),
// shifted into place; at its very ends code by code.
template <bool VEC> struct Codes;
template <> struct Codes<true> {
  uint4 w;
  __device__ __forceinline__ void ask(const int8_t* row, int k, bool in, const int8_t*, uintptr_t) {
    w = make_uint4(0u, 0u, 0u, 0u);
    if (in) w = *reinterpret_cast<const uint4*>(row + k);
  }
  __device__ __forceinline__ uint4 get(const int8_t*, int, int, bool, const int8_t*, uintptr_t) const { return w; }
};
template <> struct Codes<false> {
  uint4 a, b;
  __device__ __forceinline__ void ask(const int8_t* row, int k, bool in, const int8_t* from, uintptr_t end) {
    const uintptr_t word = reinterpret_cast<uintptr_t>(row + k) & ~(uintptr_t)15;
    a = b = make_uint4(0u, 0u, 0u, 0u);
    if (in && word >= reinterpret_cast<uintptr_t>(from) && word + 16 <= end) a = *reinterpret_cast<const uint4*>(word);
    if (in && word + 32 <= end) b = *reinterpret_cast<const uint4*>(word + 16);
  }
  __device__ __forceinline__ uint4 get(const int8_t* row, int k, int K, bool in, const int8_t* from, uintptr_t end) const {
    if (!in) return make_uint4(0u, 0u, 0u, 0u);
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k), word = at & ~(uintptr_t)15;
    const int n = K - k;
    uint32_t r[4];
    if (word >= reinterpret_cast<uintptr_t>(from) && word + 32 <= end) {
      const uint4 q = bytes_from(a, b, (int)(at & 15));
      r[0] = q.x; r[1] = q.y; r[2] = q.z; r[3] = q.w;
    } else {
      r[0] = r[1] = r[2] = r[3] = 0u;
      for (int j = 0; j < 16 && j < n; ++j) {
        const uint32_t c = (uint32_t)(uint8_t)row[k + j] << (8 * (j & 3));
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] |= j >> 2 == i ? c : 0u;
      }
    }
    if (n < 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int left = n - 4 * i;
        if (left < 4) r[i] = left <= 0 ? 0u : r[i] & ((1u << (8 * left)) - 1u);
      }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
};

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// One token, or a few: MT rows by NT columns for a warp, its lanes 16 codes of K each in turn, or for the
// four warps of a CTA (SHARED), which share out K.  Bound by reading B once, and by how many of its bytes
// are asked for at a time: 1 x 5760 x 1920 in 3.1 us shared, 3.6 by warps.
template <int MT, int NT, bool VEC, bool SHARED>
__global__ void __launch_bounds__(128)
int8_dot_kernel(const Int8Params p) {
  __shared__ int part[SHARED ? 4 : 1][MT * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n0 = (SHARED ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp) * NT;
  if (n0 >= p.N) return;
  for (int64_t m0 = 0; m0 < p.M; m0 += MT) {
    int acc[MT][NT] = {};
    for (int k = (SHARED ? (int)threadIdx.x : lane) * 16; k < p.K; k += SHARED ? 2048 : 512) {
      Codes<VEC> a[MT], b[NT];
      const int8_t *row_a[MT], *row_b[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        row_b[j] = p.b + (n0 + j < p.N ? n0 + j : p.N - 1) * p.ldb;
        b[j].ask(row_b[j], k, true, p.b, p.b_end);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        row_a[i] = p.a + (m0 + i < p.M ? m0 + i : p.M - 1) * p.lda;
        a[i].ask(row_a[i], k, true, p.a, p.a_end);
      }
      uint4 cb[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) cb[j] = b[j].get(row_b[j], k, p.K, true, p.b, p.b_end);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const uint4 ca = a[i].get(row_a[i], k, p.K, true, p.a, p.a_end);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = dot16(ca, cb[j], acc[i][j]);
      }
    }
    const int mine = lane;                                // lane i NT + j: output (m0 + i, n0 + j)
    const int64_t m = m0 + mine / NT, n = n0 + mine % NT;
    const bool out = (!SHARED || warp == 0) && mine < MT * NT && m < p.M && n < p.N;
    const float sa = out ? scale_a(p, m) : 0.0f, sb = out ? scale_b(p, n) : 0.0f;
    int s = 0;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int all = __reduce_add_sync(0xFFFFFFFFu, acc[i][j]);
        if (lane == i * NT + j) s = all;
      }
    if constexpr (SHARED) {
      if (mine < MT * NT) part[warp][mine] = s;
      __syncthreads();
      if (out) s = part[0][mine] + part[1][mine] + part[2][mine] + part[3][mine];
      if (m0 + MT < p.M) __syncthreads();
    }
    if (out) store_out(p, m, n, s, sa, sb);
  }
}

template <int MT> int launch_dot(const Int8Params& p, bool vec, cudaStream_t st) {
  constexpr int NT = 4;
  static_assert(MT * NT <= 32, "an output a lane");
  const int64_t groups = (p.N + NT - 1) / NT;
  // Shared where there is something to share, K > 512; but 16 sums of four unaligned tokens, with their
  // registers, only where there are few columns (4 x 60 x 20000 5.8 us, 18.4 by warps, and unaligned 4 x 5760 x
  // 1921 13.2, 9.0 by warps).
  const bool shared = p.K > 512 && (MT == 1 || vec || groups <= 2 * emu_ops_sm_count());
  auto kernel = vec ? shared ? int8_dot_kernel<MT, NT, true, true> : int8_dot_kernel<MT, NT, true, false>
                    : shared ? int8_dot_kernel<MT, NT, false, true> : int8_dot_kernel<MT, NT, false, false>;
  kernel<<<(unsigned)(shared ? groups : (groups + 3) / 4), 128, 0, st>>>(p);
  return EMU_OK;
}

// Four codes as fp16 (exact: |code| <= 128 has at most eight significant bits).  With the sign
// bit flipped a code is u = code + 128 in 0..255; the fp16 word 0x6400 | u is 1024 + u.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));          // 1152
  uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&a), bias), y = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

}  // namespace emu_ops

#include "ops_int8_tc.cuh"

namespace emu_ops {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// fp16 rows of Kp values, boxes of 64 values by `box` rows under the 128-byte swizzle
int f16_map(CUtensorMap* map, const uint16_t* at, int64_t rows, int64_t Kp, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[2] = {(cuuint64_t)Kp, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)Kp * 2};
  const cuuint32_t boxes[2] = {64u, (cuuint32_t)box}, step[2] = {1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<uint16_t*>(at), dims, strides, boxes, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EMU_OK : emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

inline size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }
inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How a product is computed, by its sizes alone.
enum class Int8Kind { dot, few, tensor };
struct Plan {
  Int8Kind kind;
  int64_t Kp;                    // tensor: operands laid out in rows of Kp values,
  int64_t rows_a, rows_b;        // so many rows at a time,
  size_t a_bytes, b_bytes;       // in the workspace: A's part, then B's
};
constexpr int64_t kSms = 152;                      // of the GPU that the rule was measured on
constexpr size_t kSlabBytes = (size_t)128 << 20;   // fp16 rows at a time, so that the workspace stays small

// The few-token kernel's slices of K: the rounds of CTAs (`room` of them live at once) times the stages of a
// slice and, in stages, a CTA's fixed time are to be few.
struct Slices { int S; int64_t rounds, stages; };
Slices few_slices(int64_t tiles, int64_t room, int stages) {
  Slices best = {1, (tiles + room - 1) / room, stages};
  for (int n = 2; n <= kMaxSlices && n <= stages; ++n) {
    const Slices s = {n, (tiles * n + room - 1) / room, (stages + n - 1) / n};
    if (s.rounds * (s.stages + kFixedStages) < best.rounds * (best.stages + kFixedStages)) best = s;
  }
  return best;
}

Plan plan_for(int64_t M, int64_t N, int64_t K) {
  Plan pl = {};
  pl.kind = M <= 4 || K == 0 ? Int8Kind::dot : Int8Kind::few;
  if (pl.kind == Int8Kind::few && M > 128) {
    // For many tokens both are open.  Measured, in us: the few-token kernel takes 3, and a round 4.5 and 0.8 a
    // stage, 2.1 where rows are not 16-byte aligned; laying out 5.5 and 0.43 a million codes, and then a round
    // of 128 x 256 tiles 2 and 0.27 for 64 of K.  As few and laid out: 1637 x 188 x 32 8.4 and 8.9, 300 x 5760
    // x 301 13.9 and 9.6, 2000 x 1000 x 1000 23.1 and 13.0, 400 x 5760 x 1920 35.4 and 21.0, 130 x 2000 x
    // 8000 20.5 and 48.7.
    const Slices f = few_slices(((M + 127) / 128) * ((N + 127) / 128), kSms, (int)((K + 127) / 128));
    const double few = 3.0 + (double)f.rounds * (4.5 + (K % 16 == 0 ? 0.8 : 2.1) * (double)f.stages);
    const double rounds = (double)((((M + 127) / 128) * ((N + 255) / 256) + kSms - 1) / kSms);
    const double laid_out = 5.5 + (double)(M + N) * (double)K * 0.43e-6 + rounds * (2.0 + 0.27 * (double)((K + 63) / 64));
    if (laid_out < few) pl.kind = Int8Kind::tensor;
  }
  if (pl.kind == Int8Kind::tensor) {
    pl.Kp = round_up(K, kTcBK);
    const int64_t most = (int64_t)(kSlabBytes / (2 * (size_t)pl.Kp)) / kTcBN * kTcBN;   // K < 2^17: 512 rows at least
    pl.rows_a = M < most ? M : most;
    pl.rows_b = N < most ? N : most;
    pl.a_bytes = round256((size_t)pl.rows_a * (size_t)pl.Kp * 2);
    pl.b_bytes = round256((size_t)pl.rows_b * (size_t)pl.Kp * 2);
  }
  return pl;
}

int launch_tc(const Int8Params& p, const Plan& pl, bool vec, unsigned char* ws, cudaStream_t st) {
  static std::atomic<bool> done[64];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(int8_tc_kernel), kTcSmem, done)) return emu_ops_launched("cudaFuncSetAttribute");
  uint16_t* a16 = reinterpret_cast<uint16_t*>(ws);
  uint16_t* b16 = reinterpret_cast<uint16_t*>(ws + pl.a_bytes);
  const int sms = emu_ops_sm_count();
  const size_t es = elem_bytes((emu_out_t)p.out_type);
  const uint32_t chunks = (uint32_t)(pl.Kp / 16);
  for (int64_t m = 0; m < p.M; m += pl.rows_a) {
    const int64_t rows_a = p.M - m < pl.rows_a ? p.M - m : pl.rows_a;
    for (int64_t n = 0; n < p.N; n += pl.rows_b) {
      const int64_t rows_b = p.N - n < pl.rows_b ? p.N - n : pl.rows_b;
      const uint32_t lay_a = n == 0 ? (uint32_t)rows_a : 0u;
      const bool lay_b = m == 0 || pl.rows_b < p.N;
      const uint64_t work = ((uint64_t)lay_a + (lay_b ? (uint64_t)rows_b : 0u)) * chunks;
      if (work > 0) {
        const uint64_t blocks = (work + 255) / 256;
        auto lay_out = vec ? int8_to_f16_kernel<true> : int8_to_f16_kernel<false>;
        lay_out<<<(unsigned)(blocks < 16384 ? blocks : 16384), 256, 0, st>>>(
            p, m, lay_a, a16, n, lay_b ? (uint32_t)rows_b : 0u, b16, chunks);
      }
      CUtensorMap map_a, map_b;
      int rc = f16_map(&map_a, a16, rows_a, pl.Kp, kTcBM);
      if (rc == EMU_OK) rc = f16_map(&map_b, b16, rows_b, pl.Kp, kTcBN);
      if (rc != EMU_OK) return rc;
      Int8Params q = p;
      q.M = rows_a;
      q.cols = rows_b;
      q.scale_a += m * p.sa_step;
      q.scale_b += n * p.sb_step;
      q.out = static_cast<unsigned char*>(p.out) + (size_t)(m * p.N + n) * es;
      const TcTiles tl = {(int)((rows_a + kTcBM - 1) / kTcBM), (int)((rows_b + kTcBN - 1) / kTcBN), (int)(pl.Kp / kTcBK)};
      const int tiles = tl.tiles_m * tl.tiles_n;
      // launched while the operands are still laid out, if they are: it waits for them itself
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(tiles < sms ? tiles : sms));
      cfg.blockDim = dim3(kTcThreads);
      cfg.dynamicSmemBytes = kTcSmem;
      cfg.stream = st;
      cudaLaunchAttribute early;
      early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      early.val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = &early;
      cfg.numAttrs = work > 0 ? 1 : 0;
      if (cudaLaunchKernelEx(&cfg, int8_tc_kernel, q, tl, map_a, map_b) != cudaSuccess)
        return emu_ops_launched("emu_int8_scaled_mm");
    }
  }
  return EMU_OK;
}

template <int BT> int launch_few(const Int8Params& p, bool vec, cudaStream_t st) {
  using SH = FewShape<BT>;
  const int64_t tn = (p.N + 127) / 128, tiles = tn * ((p.M + BT - 1) / BT), room = (int64_t)emu_ops_sm_count() * SH::RESIDENT;
  const int stages = (p.K + 127) / 128;
  const int S = few_slices(tiles, room, stages).S;
  const bool is_long = (stages + S - 1) / S > 8;
  auto kernel = vec ? is_long ? int8_few_kernel<BT, true, true> : int8_few_kernel<BT, false, true>
                    : is_long ? int8_few_kernel<BT, true, false> : int8_few_kernel<BT, false, false>;
  static std::atomic<bool> done[4][64];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(kernel), SH::SMEM, done[2 * vec + is_long]))
    return emu_ops_launched("cudaFuncSetAttribute");
  // rows of tiles on grid.y, at most 65535 a launch
  for (int64_t m = 0; m < p.M; m += (int64_t)65535 * BT) {
    Int8Params q = p;
    q.M = p.M - m < (int64_t)65535 * BT ? p.M - m : (int64_t)65535 * BT;
    q.a += m * p.lda;
    q.scale_a += m * p.sa_step;
    q.out = static_cast<unsigned char*>(p.out) + (size_t)(m * p.N) * elem_bytes((emu_out_t)p.out_type);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tn * S), (unsigned)((q.M + BT - 1) / BT));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = SH::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)S;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = S > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, q, S) != cudaSuccess) return emu_ops_launched("emu_int8_scaled_mm");
  }
  return EMU_OK;
}

int run_plan(const Int8Params& p, bool vec, void* workspace, cudaStream_t st) {
  const Plan pl = plan_for(p.M, p.N, p.K);
  int rc;
  if (pl.kind == Int8Kind::tensor) rc = launch_tc(p, pl, vec, static_cast<unsigned char*>(workspace), st);
  else if (pl.kind == Int8Kind::dot) rc = p.M == 1 ? launch_dot<1>(p, vec, st) : launch_dot<4>(p, vec, st);
  else if (p.M <= 16) rc = launch_few<16>(p, vec, st);
  else if (p.M <= 32) rc = launch_few<32>(p, vec, st);
  else if (p.M <= 64) rc = launch_few<64>(p, vec, st);
  else rc = launch_few<128>(p, vec, st);
  return rc == EMU_OK ? emu_ops_launched("emu_int8_scaled_mm") : rc;
}

}  // namespace emu_ops

using namespace emu_ops;

int emu_ops_int8_status(int* status, bool reset) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_ops_status, sizeof v);
  if (e != cudaSuccess) return emu_ops_fail(EMU_ECUDA, "reading the device status failed: %s", cudaGetErrorString(e));
  *status = v;
  if (reset) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_ops_status, &zero, sizeof zero);
    if (e != cudaSuccess) return emu_ops_fail(EMU_ECUDA, "clearing the device status failed: %s", cudaGetErrorString(e));
  }
  return EMU_OK;
}

extern "C" {

size_t emu_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1 || K > kInt8MaxK || M >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 31)) return 0;
  const Plan plan = plan_for(M, N, K);
  return plan.a_bytes + plan.b_bytes;
}

int emu_int8_scaled_mm(const int8_t* A, int64_t lda, const int8_t* B, int64_t ldb, int64_t M, int64_t N, int64_t K,
                       const float* scale_a, int64_t scale_a_count, const float* scale_b, int64_t scale_b_count,
                       void* out, emu_out_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  emu_ops_begin();
  if (!is_float_type(out_dtype)) return emu_ops_fail(EMU_EINVAL, "the output is fp32, bf16 or fp16 (got %d)", (int)out_dtype);
  if (M < 0 || N < 0 || K < 0)
    return emu_ops_fail(EMU_EINVAL, "negative size (%lld, %lld, %lld)", (long long)M, (long long)N, (long long)K);
  if (M >= ((int64_t)1 << 31) || N >= ((int64_t)1 << 31)) return emu_ops_fail(EMU_EUNSUPPORTED, "sizes must be below 2^31");
  if (K > kInt8MaxK)
    return emu_ops_fail(EMU_EUNSUPPORTED, "K = %lld: the 32-bit sums are exact up to K = %lld", (long long)K, (long long)kInt8MaxK);
  if ((scale_a_count != 1 && scale_a_count != M) || (scale_b_count != 1 && scale_b_count != N))
    return emu_ops_fail(EMU_EINVAL, "one scale, or one for each of the %lld rows and %lld columns (got %lld, %lld)",
                        (long long)M, (long long)N, (long long)scale_a_count, (long long)scale_b_count);
  if (M == 0 || N == 0) return EMU_OK;
  if (!out || !scale_a || !scale_b || (K > 0 && (!A || !B))) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (lda < K || ldb < K) return emu_ops_fail(EMU_EINVAL, "a row stride is below K = %lld", (long long)K);
  const size_t es = elem_bytes(out_dtype);
  if (!aligned(out, es) || !aligned(scale_a, 4) || !aligned(scale_b, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  const bool vec = K % 16 == 0 && lda % 16 == 0 && ldb % 16 == 0 && aligned(A, 16) && aligned(B, 16);
  const size_t need = emu_int8_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return emu_ops_fail(EMU_EINVAL, "workspace of %zu bytes needed, 256-byte aligned (got %zu)", need, workspace_bytes);
  if (!apart({Span(out, M, N, N, es), Span(need ? workspace : nullptr, 1, 1, 1, need)},
             {Span(A, M, lda, K, 1), Span(B, N, ldb, K, 1), Span(scale_a, 1, scale_a_count, scale_a_count, 4),
              Span(scale_b, 1, scale_b_count, scale_b_count, 4)}))
    return emu_ops_fail(EMU_EINVAL, "the output or the workspace overlaps an input, or the other");
  Int8Params p;
  p.a = A; p.lda = lda; p.b = B; p.ldb = ldb;
  p.a_end = reinterpret_cast<uintptr_t>(A) + (size_t)(M - 1) * (size_t)lda + (size_t)K;
  p.b_end = reinterpret_cast<uintptr_t>(B) + (size_t)(N - 1) * (size_t)ldb + (size_t)K;
  p.M = M; p.N = N; p.cols = N; p.K = (int)K;
  p.scale_a = scale_a; p.sa_step = scale_a_count == 1 ? 0 : 1;
  p.scale_b = scale_b; p.sb_step = scale_b_count == 1 ? 0 : 1;
  p.out = out; p.out_type = (int)out_dtype;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return run_plan(p, vec, workspace, st);
}

}  // extern "C"
