// ops_block_mm.cu -- FP8 products with a scale for each block of 128 of K, dense, by expert over
// ragged groups of rows, and the experts' weights' gradients (declared in include/emu_fp8.h):
//   out[m, n] = sum over blocks kb of (sum over k in kb of a[m, k] b[n, k]) * (sa[m, kb] * sb[n, kb])
#include "ops_block.cuh"

#include <type_traits>

namespace emu_ops {

constexpr int64_t kMaxExperts = 1024;

enum class BlockKind { dense, grouped, wgrad };
struct BlockMm {
  emu_block_operand_t a, b;                              // M and N rows; wgrad: rows by tokens
  BlockKind kind;
  int64_t M, N, K;                                       // grouped: M tokens; wgrad: K tokens
  const int32_t* offsets; int E;
  bool zero_rest;
  void* out; int out_type;                               // [M, N], wgrad [E, M, N]
};

// rows [lo, hi) of expert e: the offsets within [0, T], none below the one before it
__device__ __forceinline__ void group_of(const BlockMm& p, int e, int64_t T, int64_t& lo, int64_t& hi) {
  lo = 0;
  for (int i = 0; i <= e + 1; ++i) {
    int64_t at = p.offsets[i];
    at = at < 0 ? 0 : at > T ? T : at;
    if (i == e + 1) hi = at > lo ? at : lo;
    else lo = at > lo ? at : lo;
  }
}
__device__ __forceinline__ float scale_at(const emu_block_operand_t& o, int64_t row, int64_t kb, int64_t group) {
  return __ldg(o.scale + group * o.scale_group_stride + (o.scale_rows == 1 ? row : row / kBlock) * o.scale_row_stride +
               kb * o.scale_k_stride);
}
__device__ __forceinline__ void store_out(void* out, int type, int64_t i, float v) {
  if (type == EMU_OUT_F32) static_cast<float*>(out)[i] = v;
  else if (type == EMU_OUT_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

// one output a thread
__global__ void __launch_bounds__(256) block_mm_kernel(const BlockMm p) {
  const int64_t per = p.M * p.N, total = per * (p.kind == BlockKind::wgrad ? p.E : 1);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    int64_t group = i / per, m = i % per / p.N, n = i % p.N, k0 = 0, k1 = p.K;
    if (p.kind == BlockKind::wgrad) {
      group_of(p, (int)group, p.K, k0, k1);
    } else if (p.kind == BlockKind::grouped) {
      int64_t lo = 0, hi = 0;
      int e = 0;
      for (; e < p.E; ++e) {
        group_of(p, e, p.M, lo, hi);
        if (m >= lo && m < hi) break;
      }
      if (e == p.E) {
        if (p.zero_rest) store_out(p.out, p.out_type, i, 0.0f);
        continue;
      }
      group = e;
    }
    const int64_t gb = p.kind == BlockKind::grouped ? group : 0;
    const uint8_t* a = static_cast<const uint8_t*>(p.a.codes) + m * p.a.row_stride;
    const uint8_t* b = static_cast<const uint8_t*>(p.b.codes) + gb * p.b.group_stride + n * p.b.row_stride;
    float sum = 0.0f;
    while (k0 < k1) {
      const int64_t kb = k0 / kBlock, end = (kb + 1) * kBlock < k1 ? (kb + 1) * kBlock : k1;
      float part = 0.0f;
      for (; k0 < end; ++k0)
        part = fmaf(code_value(a[k0 * p.a.k_stride], p.a.format), code_value(b[k0 * p.b.k_stride], p.b.format), part);
      sum = fmaf(part, scale_at(p.a, m, kb, 0) * scale_at(p.b, n, kb, gb), sum);
    }
    store_out(p.out, p.out_type, i, sum);
  }
}

int run_block_mm(const BlockMm& p, cudaStream_t st) {
  const int64_t total = p.M * p.N * (p.kind == BlockKind::wgrad ? p.E : 1), ctas = (total + 255) / 256;
  block_mm_kernel<<<(unsigned)(ctas < 1 << 20 ? ctas : 1 << 20), 256, 0, st>>>(p);
  return emu_ops_launched("emu_block_scaled_mm");
}

// ------------------------------------------------------------------------------- checks
struct Sizes { int64_t rows, K, groups; };
// the memory that an operand's codes and scales span
Span codes_span(const emu_block_operand_t& o, const Sizes& s) {
  const int64_t r = s.rows > 0 && s.K > 0 ? (s.rows - 1) * o.row_stride + (s.K - 1) * o.k_stride + 1 : 0;
  return Span(o.codes, s.groups, o.group_stride, r, 1);
}
Span scale_span(const emu_block_operand_t& o, const Sizes& s) {
  const int64_t rb = (s.rows + o.scale_rows - 1) / o.scale_rows, kb = (s.K + kBlock - 1) / kBlock;
  const int64_t r = rb > 0 && kb > 0 ? (rb - 1) * o.scale_row_stride + (kb - 1) * o.scale_k_stride + 1 : 0;
  return Span(o.scale, s.groups, o.scale_group_stride, r, 4);
}
int check_operand(const char* name, const emu_block_operand_t* o, const Sizes& s) {
  if (!o) return emu_ops_fail(EMU_EINVAL, "%s: null operand", name);
  if (o->format != EMU_E4M3FN && o->format != EMU_E5M2) return emu_ops_fail(EMU_EINVAL, "%s: unknown FP8 format %d", name, (int)o->format);
  if (o->scale_rows != 1 && o->scale_rows != kBlock)
    return emu_ops_fail(EMU_EINVAL, "%s: a scale is for 1 row or %d (got %d)", name, kBlock, (int)o->scale_rows);
  if (s.rows == 0 || s.K == 0 || s.groups == 0) return EMU_OK;
  if (!o->codes || !o->scale) return emu_ops_fail(EMU_EINVAL, "%s: null tensor", name);
  const bool by_k = o->k_stride == 1 && (s.rows == 1 || o->row_stride >= s.K);
  const bool by_row = o->row_stride == 1 && (s.K == 1 || o->k_stride >= s.rows);
  if (!by_k && !by_row)
    return emu_ops_fail(EMU_EINVAL, "%s: a row's codes or a K position's are contiguous and apart from the next (strides %lld, %lld)",
                        name, (long long)o->row_stride, (long long)o->k_stride);
  if (o->scale_row_stride < 0 || o->scale_k_stride < 0 || o->group_stride < 0 || o->scale_group_stride < 0)
    return emu_ops_fail(EMU_EINVAL, "%s: negative stride", name);
  if (s.groups > 1 && o->group_stride < (by_k ? (s.rows - 1) * o->row_stride + s.K : (s.K - 1) * o->k_stride + s.rows))
    return emu_ops_fail(EMU_EINVAL, "%s: the groups overlap (stride %lld)", name, (long long)o->group_stride);
  if (!aligned(o->scale, 4)) return emu_ops_fail(EMU_EINVAL, "%s: the scales are not aligned to their elements", name);
  return EMU_OK;
}
int check_sizes(emu_out_t type, int64_t M, int64_t N, int64_t K, int64_t E) {
  if (!is_float_type(type)) return emu_ops_fail(EMU_EINVAL, "the output is fp32, bf16 or fp16 (got %d)", (int)type);
  if (M < 0 || N < 0 || K < 0 || E < 0)
    return emu_ops_fail(EMU_EINVAL, "negative size (%lld, %lld, %lld, %lld)", (long long)M, (long long)N, (long long)K, (long long)E);
  const int64_t most = (int64_t)1 << 31;
  if (M >= most || N >= most || K >= most) return emu_ops_fail(EMU_EUNSUPPORTED, "sizes must be below 2^31");
  if (E > kMaxExperts) return emu_ops_fail(EMU_EUNSUPPORTED, "more than %lld experts", (long long)kMaxExperts);
  return EMU_OK;
}
int check_out(void* out, emu_out_t type, int64_t rows, int64_t cols, const int32_t* offsets, int64_t E, void* workspace,
              size_t workspace_bytes, size_t need, const emu_block_operand_t& a, const Sizes& sa, const emu_block_operand_t& b,
              const Sizes& sb) {
  const size_t es = elem_bytes(type);
  if (!out) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (!aligned(out, es) || !aligned(offsets, 4)) return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
    return emu_ops_fail(EMU_EINVAL, "workspace of %zu bytes needed, 256-byte aligned (got %zu)", need, workspace_bytes);
  if (!apart({Span(out, rows, cols, cols, es), Span(need ? workspace : nullptr, 1, 1, 1, need)},
             {codes_span(a, sa), scale_span(a, sa), codes_span(b, sb), scale_span(b, sb), Span(offsets, 1, E + 1, E + 1, 4)}))
    return emu_ops_fail(EMU_EINVAL, "the output or the workspace overlaps an input, or the other");
  return EMU_OK;
}

}  // namespace emu_ops

using namespace emu_ops;

extern "C" {

size_t emu_block_mm_workspace_bytes(const emu_block_operand_t*, const emu_block_operand_t*, int64_t, int64_t, int64_t) { return 0; }
size_t emu_grouped_block_mm_workspace_bytes(const emu_block_operand_t*, const emu_block_operand_t*, int64_t, int64_t, int64_t,
                                            int64_t) {
  return 0;
}
size_t emu_grouped_block_wgrad_workspace_bytes(const emu_block_operand_t*, const emu_block_operand_t*, int64_t, int64_t, int64_t) {
  return 0;
}

int emu_block_scaled_mm(const emu_block_operand_t* a, const emu_block_operand_t* b, int64_t M, int64_t N, int64_t K, void* out,
                        emu_out_t out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  emu_ops_begin();
  int rc = check_sizes(out_dtype, M, N, K, 0);
  if (rc == EMU_OK) rc = check_operand("a", a, {M, K, 1});
  if (rc == EMU_OK) rc = check_operand("b", b, {N, K, 1});
  if (rc != EMU_OK || M == 0 || N == 0) return rc;
  const size_t need = emu_block_mm_workspace_bytes(a, b, M, N, K);
  rc = check_out(out, out_dtype, M, N, nullptr, -1, workspace, workspace_bytes, need, *a, {M, K, 1}, *b, {N, K, 1});
  if (rc != EMU_OK) return rc;
  BlockMm p = {*a, *b, BlockKind::dense, M, N, K, nullptr, 1, false, out, (int)out_dtype};
  return run_block_mm(p, static_cast<cudaStream_t>(stream));
}

int emu_grouped_block_scaled_mm(const emu_block_operand_t* a, const emu_block_operand_t* b, const int32_t* offsets, int64_t E,
                                int64_t T, int64_t N, int64_t K, void* out, emu_out_t out_dtype, int32_t zero_rest,
                                void* workspace, size_t workspace_bytes, void* stream) {
  emu_ops_begin();
  int rc = check_sizes(out_dtype, T, N, K, E);
  if (rc == EMU_OK) rc = check_operand("a", a, {T, K, 1});
  if (rc == EMU_OK) rc = check_operand("b", b, {N, K, E});
  if (rc != EMU_OK || T == 0 || N == 0) return rc;
  if (K > 1 && a->k_stride != 1) return emu_ops_fail(EMU_EINVAL, "a: a row's codes must be contiguous");
  if (!offsets) return emu_ops_fail(EMU_EINVAL, "null tensor");
  const size_t need = emu_grouped_block_mm_workspace_bytes(a, b, T, N, K, E);
  rc = check_out(out, out_dtype, T, N, offsets, E, workspace, workspace_bytes, need, *a, {T, K, 1}, *b, {N, K, E});
  if (rc != EMU_OK) return rc;
  BlockMm p = {*a, *b, BlockKind::grouped, T, N, K, offsets, (int)E, zero_rest != 0, out, (int)out_dtype};
  return run_block_mm(p, static_cast<cudaStream_t>(stream));
}

int emu_grouped_block_scaled_wgrad(const emu_block_operand_t* a, const emu_block_operand_t* b, const int32_t* offsets, int64_t E,
                                   int64_t T, int64_t N, int64_t K, void* out, emu_out_t out_dtype, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  emu_ops_begin();
  int rc = check_sizes(out_dtype, T, N, K, E);
  if (rc == EMU_OK) rc = check_operand("a", a, {N, T, 1});
  if (rc == EMU_OK) rc = check_operand("b", b, {K, T, 1});
  if (rc != EMU_OK || N == 0 || K == 0 || E == 0) return rc;
  if ((N > 1 && T > 0 && a->row_stride != 1) || (K > 1 && T > 0 && b->row_stride != 1))
    return emu_ops_fail(EMU_EINVAL, "the codes of a token must be contiguous");
  if (!offsets) return emu_ops_fail(EMU_EINVAL, "null tensor");
  const size_t need = emu_grouped_block_wgrad_workspace_bytes(a, b, T, N, K);
  rc = check_out(out, out_dtype, E * N, K, offsets, E, workspace, workspace_bytes, need, *a, {N, T, 1}, *b, {K, T, 1});
  if (rc != EMU_OK) return rc;
  BlockMm p = {*a, *b, BlockKind::wgrad, N, K, T, offsets, (int)E, false, out, (int)out_dtype};
  return run_block_mm(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
