// ops_int8.cu -- the product of 8-bit integers with a scale for each token (row of A) and
// each channel (column of B), declared in include/emu_fp8.h:
//   out[m, n] = (fp32(sum_k A[m, k] B[k, n]) * scale_a[m]) * scale_b[n]
// The sum is exact in 32-bit integers, so the result does not depend on the order or the
// kernel that took it.
#include "ops_common.cuh"

namespace emu_ops {

constexpr int64_t kInt8MaxK = 131071;             // K * 128 * 128 < 2^31

struct Int8Params {
  const int8_t* a; int64_t lda;                   // [M, K]
  const int8_t* b; int64_t ldb;                   // [N, K]
  int64_t M, N;
  int K;
  const float* scale_a; int sa_step;              // 0: one scale for all
  const float* scale_b; int sb_step;
  void* out; int out_type;                        // [M, N] contiguous
};

__device__ __forceinline__ void store_out(const Int8Params& p, int64_t m, int64_t n, int acc) {
  const float v = ((float)acc * p.scale_a[m * p.sa_step]) * p.scale_b[n * p.sb_step];
  const int64_t i = m * p.N + n;
  if (p.out_type == EMU_OUT_F32) static_cast<float*>(p.out)[i] = v;
  else if (p.out_type == EMU_OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p.out)[i] = __float2half_rn(v);
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a((int)a.x, (int)b.x, acc);
  acc = __dp4a((int)a.y, (int)b.y, acc);
  acc = __dp4a((int)a.z, (int)b.z, acc);
  return __dp4a((int)a.w, (int)b.w, acc);
}

// A warp takes MT rows by NT columns, its lanes 16 codes of K each in turn (one code where
// rows are not 16-byte aligned), and adds the lanes' sums up.
template <int MT, int NT, bool VEC>
__global__ void __launch_bounds__(128)
int8_dot_kernel(const Int8Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * NT;
  if (n0 >= p.N) return;
  for (int64_t m0 = (int64_t)blockIdx.y * MT; m0 < p.M; m0 += (int64_t)gridDim.y * MT) {
    int acc[MT][NT] = {};
    if constexpr (VEC) {
      for (int k = lane * 16; k < p.K; k += 512) {
        uint4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          b[j] = *reinterpret_cast<const uint4*>(p.b + (n0 + j < p.N ? n0 + j : p.N - 1) * p.ldb + k);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint4 a = *reinterpret_cast<const uint4*>(p.a + (m0 + i < p.M ? m0 + i : p.M - 1) * p.lda + k);
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = dot16(a, b[j], acc[i][j]);
        }
      }
    } else {
      for (int k = lane; k < p.K; k += 32) {
        int b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = p.b[(n0 + j < p.N ? n0 + j : p.N - 1) * p.ldb + k];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int a = p.a[(m0 + i < p.M ? m0 + i : p.M - 1) * p.lda + k];
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] += a * b[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int s = __reduce_add_sync(0xFFFFFFFFu, acc[i][j]);
        if (lane == (i * NT + j) % 32 && m0 + i < p.M && n0 + j < p.N) store_out(p, m0 + i, n0 + j, s);
      }
  }
}

template <bool VEC> void launch_dot(const Int8Params& p, cudaStream_t st) {
  constexpr int NT = 4;
  const unsigned gx = (unsigned)((p.N + 4 * NT - 1) / (4 * NT));
  const int64_t tiles = (p.M + 7) / 8;
  const unsigned gy = (unsigned)(tiles < 65535 ? tiles : 65535);
  if (p.M == 1) int8_dot_kernel<1, NT, VEC><<<dim3(gx, 1), 128, 0, st>>>(p);
  else int8_dot_kernel<8, NT, VEC><<<dim3(gx, gy), 128, 0, st>>>(p);
}

}  // namespace emu_ops

using namespace emu_ops;

int emu_ops_device_status_int8(int* status, bool) {
  *status = 0;
  return EMU_OK;
}

extern "C" {

size_t emu_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  (void)M; (void)N; (void)K;
  return 0;
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
  const size_t need = emu_int8_workspace_bytes(M, N, K);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return emu_ops_fail(EMU_EINVAL, "workspace of %zu bytes needed, 256-byte aligned (got %zu)", need, workspace_bytes);
  Int8Params p;
  p.a = A; p.lda = lda; p.b = B; p.ldb = ldb; p.M = M; p.N = N; p.K = (int)K;
  p.scale_a = scale_a; p.sa_step = scale_a_count == 1 ? 0 : 1;
  p.scale_b = scale_b; p.sb_step = scale_b_count == 1 ? 0 : 1;
  p.out = out; p.out_type = (int)out_dtype;
  const bool vec = K % 16 == 0 && lda % 16 == 0 && ldb % 16 == 0 && aligned(A, 16) && aligned(B, 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (vec) launch_dot<true>(p, st);
  else launch_dot<false>(p, st);
  return emu_ops_launched("emu_int8_scaled_mm");
}

}  // extern "C"
