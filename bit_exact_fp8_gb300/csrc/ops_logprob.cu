// ops_logprob.cu -- log probabilities of given tokens with the rows' entropies and top
// alternatives, and their gradient (declared in include/emu_fp8.h).
//
// Of a row x of V logits: m = max x, z = sum e^(x - m), u = sum e^(x - m) (x - m);
//   lse = m + log z,  logprob = x[token] - lse,  entropy = log z - u / z.
// A row of nothing but -inf is empty: lse and logprobs -inf, entropy 0, gradient 0.  The
// gradient is given m and log z apart, since m + log z loses log z where |m| is large (a
// mask of large negative numbers that leaves nothing).  A row
// holding NaN or +inf has NaN for all of its floats, and -1 for its top ids.
#include "ops_common.cuh"

namespace emu_ops {

constexpr int kMaxTop = 32;
constexpr float kLog2e = 1.44269504f;

struct LogprobParams {
  const void* x; int64_t ldx;
  const int64_t* tokens;
  int64_t ignore;
  int64_t T; int V; int k;
  float* logprob; float* entropy; float* lse; float* stats;   // stats [T, 3]: m, log z, entropy
  float* top_val; int64_t* top_id;               // [T, k]
};

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// the order of floats as that of unsigned words, above 0 (-0 as +0)
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Running (m, z, u) of a part of a row; m = -inf: nothing above -inf yet.
struct Soft {
  float m, z, u;
};
__device__ __forceinline__ Soft soft_join(const Soft& a, const Soft& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return Soft{m, a.z + b.z, a.u + b.u};      // zeros, or a NaN that is kept
  Soft r{m, 0.0f, 0.0f};
  if (a.m != -INFINITY || a.z != 0.0f) {
    const float d = fmaxf(a.m - m, -1e4f), f = exp2_approx(d * kLog2e);
    r.z += a.z * f;
    r.u += (a.u + a.z * d) * f;
  }
  if (b.m != -INFINITY || b.z != 0.0f) {
    const float d = fmaxf(b.m - m, -1e4f), f = exp2_approx(d * kLog2e);
    r.z += b.z * f;
    r.u += (b.u + b.z * d) * f;
  }
  return r;
}
__device__ __forceinline__ Soft soft_shfl(const Soft& a, int o) {
  return Soft{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.z, o),
              __shfl_xor_sync(0xFFFFFFFFu, a.u, o)};
}

// the row's outputs but its alternatives; x - m is exact where it matters, so logprob is (x - m) - log z
template <class T>
__device__ __forceinline__ void finish_row(const LogprobParams& p, int64_t row, float m, float z, float u, const T* x) {
  const bool empty = m == -INFINITY && z == 0.0f;
  const float logz = logf(z);
  const float entropy = empty ? 0.0f : logz - u / z;
  const int64_t tok = p.tokens[row];
  p.logprob[row] = tok == p.ignore ? 0.0f
                   : tok < 0 || tok >= p.V ? NAN
                   : empty ? -INFINITY : to_f(x[tok]) - m - logz;
  p.entropy[row] = entropy;
  p.lse[row] = empty ? -INFINITY : m + logz;
  float* st = p.stats + row * 3;
  st[0] = m;
  st[1] = logz;
  st[2] = entropy;
}

// One CTA a row; each thread takes every 256th logit.  The alternatives: k times the
// largest (key, lowest index) below the last one found.
template <class T>
__global__ void __launch_bounds__(256)
logprob_kernel(const LogprobParams p) {
  __shared__ Soft sm[8];
  __shared__ unsigned long long best[8];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Soft s{-INFINITY, 0.0f, 0.0f};
  for (int v = tid; v < p.V; v += 256) {
    const float f = to_f(x[v]);
    if (f == -INFINITY) continue;
    s = soft_join(s, f != f || f == INFINITY ? Soft{s.m, NAN, NAN} : Soft{f, 1.0f, 0.0f});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = soft_join(s, soft_shfl(s, o));
  if (lane == 0) sm[warp] = s;
  __syncthreads();
  s = sm[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) s = soft_join(s, sm[w]);
  const bool empty = s.m == -INFINITY && s.z == 0.0f;
  const float logz = logf(s.z);
  if (tid == 0) finish_row(p, row, s.m, s.z, s.u, x);
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.k; ++i) {
    unsigned long long mine = 0ull;
    for (int v = tid; v < p.V; v += 256) {
      const unsigned long long c = ((unsigned long long)order_key(to_f(x[v])) << 32) | (0xFFFFFFFFu - (uint32_t)v);
      if (c < last && c > mine) mine = c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long c = __shfl_xor_sync(0xFFFFFFFFu, mine, o);
      mine = c > mine ? c : mine;
    }
    __syncthreads();
    if (lane == 0) best[warp] = mine;
    __syncthreads();
    last = best[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) last = best[w] > last ? best[w] : last;
    if (tid == 0) {
      const bool bad = logz != logz;
      p.top_val[row * p.k + i] = bad ? NAN : empty ? -INFINITY : key_value((uint32_t)(last >> 32)) - s.m - logz;
      p.top_id[row * p.k + i] = bad ? -1 : (int64_t)(0xFFFFFFFFu - (uint32_t)last);
    }
  }
}

struct LogprobGradParams {
  const void* x; int64_t ldx;
  const int64_t* tokens;
  int64_t ignore;
  int64_t T; int V;
  const float* stats;
  const float* g_logprob; const float* g_entropy;     // either may be null
  void* gx; int64_t ldo;
};

// gx = gl ([v = token] - p) - ge p (log p + H), log p = (x - m) - log z, one CTA a row
template <class T>
__global__ void __launch_bounds__(256)
logprob_grad_kernel(const LogprobGradParams p) {
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  T* gx = static_cast<T*>(p.gx) + row * p.ldo;
  const float m = p.stats[row * 3], logz = p.stats[row * 3 + 1], H = p.stats[row * 3 + 2];
  const int64_t tok = p.tokens[row];
  const bool out_of_range = tok != p.ignore && (tok < 0 || tok >= p.V);
  const float gl = tok == p.ignore || !p.g_logprob ? 0.0f : out_of_range ? NAN : p.g_logprob[row];
  const float ge = p.g_entropy ? p.g_entropy[row] : 0.0f;
  const bool empty = m == -INFINITY && logz == -INFINITY;
  for (int v = threadIdx.x; v < p.V; v += 256) {
    float r = 0.0f;
    if (!empty) {
      const float lp = to_f(x[v]) - m - logz;
      const float pr = exp2_approx(lp * kLog2e);
      r = -pr * fmaf(ge, max_nan(lp, -1e4f) + H, gl);
      if (v == tok) r += gl;
    }
    gx[v] = from_f<T>(r);
  }
}

int check_logits(const char* what, emu_out_t type, const void* x, int64_t ldx, const int64_t* tokens, int64_t T,
                 int64_t V) {
  if (!is_float_type(type)) return emu_ops_fail(EMU_EINVAL, "%s: unknown element type %d", what, (int)type);
  if (T < 0 || V < 1) return emu_ops_fail(EMU_EINVAL, "%s: sizes (%lld, %lld)", what, (long long)T, (long long)V);
  if (T >= ((int64_t)1 << 31) || V > ((int64_t)1 << 30))
    return emu_ops_fail(EMU_EUNSUPPORTED, "%s: at most 2^31 - 1 rows of 2^30 logits", what);
  if (T == 0) return EMU_OK;
  if (!x || !tokens) return emu_ops_fail(EMU_EINVAL, "%s: null logits or tokens", what);
  if (ldx < V) return emu_ops_fail(EMU_EINVAL, "%s: the row stride is below the row's %lld logits", what, (long long)V);
  if (!aligned(x, elem_bytes(type)) || !aligned(tokens, 8))
    return emu_ops_fail(EMU_EINVAL, "%s: a tensor is not aligned to its elements", what);
  return EMU_OK;
}

}  // namespace emu_ops

using namespace emu_ops;

extern "C" {

int emu_token_logprobs(const void* logits, int64_t ldx, emu_out_t type, const int64_t* tokens, int64_t T, int64_t V,
                       int32_t top_k, int64_t ignore_index, float* logprob, float* entropy, float* lse,
                       float* stats, float* top_logprobs, int64_t* top_ids, void* stream) {
  emu_ops_begin();
  int rc = check_logits("emu_token_logprobs", type, logits, ldx, tokens, T, V);
  if (rc != EMU_OK) return rc;
  if (top_k < 0 || top_k > V) return emu_ops_fail(EMU_EINVAL, "top_k %d of %lld logits", top_k, (long long)V);
  if (top_k > kMaxTop) return emu_ops_fail(EMU_EUNSUPPORTED, "top_k above %d is not supported", kMaxTop);
  if (T == 0) return EMU_OK;
  if (!logprob || !entropy || !lse || !stats || (top_k > 0 && (!top_logprobs || !top_ids)))
    return emu_ops_fail(EMU_EINVAL, "null output");
  if (!aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(stats, 4) ||
      !aligned(top_logprobs, 4) ||
      !aligned(top_ids, 8))
    return emu_ops_fail(EMU_EINVAL, "an output is not aligned to its elements");
  LogprobParams p;
  p.x = logits; p.ldx = ldx; p.tokens = tokens; p.ignore = ignore_index;
  p.T = T; p.V = (int)V; p.k = top_k;
  p.logprob = logprob; p.entropy = entropy; p.lse = lse; p.stats = stats; p.top_val = top_logprobs; p.top_id = top_ids;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == EMU_OUT_F32) logprob_kernel<float><<<(unsigned)T, 256, 0, st>>>(p);
  else if (type == EMU_OUT_BF16) logprob_kernel<__nv_bfloat16><<<(unsigned)T, 256, 0, st>>>(p);
  else logprob_kernel<__half><<<(unsigned)T, 256, 0, st>>>(p);
  return emu_ops_launched("emu_token_logprobs");
}

int emu_token_logprobs_backward(const void* logits, int64_t ldx, emu_out_t type, const int64_t* tokens, int64_t T,
                                int64_t V, int64_t ignore_index, const float* stats, const float* grad_logprob,
                                const float* grad_entropy, void* grad_logits, int64_t ldo, void* stream) {
  emu_ops_begin();
  int rc = check_logits("emu_token_logprobs_backward", type, logits, ldx, tokens, T, V);
  if (rc != EMU_OK || T == 0) return rc;
  if (!stats || !grad_logits) return emu_ops_fail(EMU_EINVAL, "null stats or grad_logits");
  if (ldo < V) return emu_ops_fail(EMU_EINVAL, "grad_logits' row stride is below the row's %lld values", (long long)V);
  const size_t es = elem_bytes(type);
  if (!aligned(grad_logits, es) || !aligned(stats, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  if (Span(grad_logits, T, ldo, V, es).meets(Span(logits, T, ldx, V, es)) && !(grad_logits == logits && ldo == ldx))
    return emu_ops_fail(EMU_EINVAL, "grad_logits overlaps the logits without being them");
  LogprobGradParams p;
  p.x = logits; p.ldx = ldx; p.tokens = tokens; p.ignore = ignore_index; p.T = T; p.V = (int)V;
  p.stats = stats; p.g_logprob = grad_logprob; p.g_entropy = grad_entropy;
  p.gx = grad_logits; p.ldo = ldo;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == EMU_OUT_F32) logprob_grad_kernel<float><<<(unsigned)T, 256, 0, st>>>(p);
  else if (type == EMU_OUT_BF16) logprob_grad_kernel<__nv_bfloat16><<<(unsigned)T, 256, 0, st>>>(p);
  else logprob_grad_kernel<__half><<<(unsigned)T, 256, 0, st>>>(p);
  return emu_ops_launched("emu_token_logprobs_backward");
}

}  // extern "C"
