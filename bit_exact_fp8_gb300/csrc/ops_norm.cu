// ops_norm.cu -- RMS norm with the residual's addition and an 8-bit output, and its
// gradient (declared in include/emu_fp8.h); and the host side that the operators share.
#include "ops_common.cuh"

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <string>

namespace {
thread_local std::string g_ops_error;
}

int emu_ops_fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    g_ops_error = buf;
  } catch (...) {                  // out of host memory: no message, the code still goes out
  }
  return code;
}
void emu_ops_begin() {
  g_ops_error.clear();
  cudaGetLastError();
}
int emu_ops_launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? EMU_OK : emu_ops_fail(EMU_ECUDA, "%s: CUDA launch failed: %s", what, cudaGetErrorString(e));
}
bool emu_ops_allow_smem(const void* kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return true;
}
int emu_ops_sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    int n = 0;
    v = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0 ? n : 152;
    cached[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

namespace emu_ops {

// 1 once a bounded wait gave up (the outputs of that call are not valid)
__device__ int g_norm_status = 0;

constexpr float kScaleMin = 1.17549435e-38f;      // 2^-126, the smallest scale of a row

struct NormParams {
  const void* x; int64_t ldx;
  const void* residual; int64_t ldr;              // null: none
  const void* weight; bool weight_f32;            // else of x's type
  int64_t T; int H;
  float eps, qmax;
  const float* scale;                             // one value, or null: one for each row
  int q_format;
  uint8_t* q;
  float* scale_out;
  void* residual_out; int64_t ldo;                // null: not written
  float* rstd;
};

template <class T, int VEC, class P>
__device__ __forceinline__ void load_weight(const P& p, int col, float (&w)[VEC]) {
  if (p.weight_f32) {
    constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
    for (int j = 0; j < VEC; j += V4) {
      float t[V4];
      load_f<float, V4>(static_cast<const float*>(p.weight) + col + j, t);
#pragma unroll
      for (int i = 0; i < V4; ++i) w[j + i] = t[i];
    }
  } else {
    load_f<T, VEC>(static_cast<const T*>(p.weight) + col, w);
  }
}

// the code of each value, rounded to nearest even and saturated (NaN: the formats' NaN, int8 0)
__device__ __forceinline__ uint32_t code_pair(float lo, float hi, int q_format) {
  uint16_t r;
  if (q_format == EMU_Q_E4M3FN) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  if (q_format == EMU_Q_E5M2) {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  int a, b;
  asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(a) : "f"(lo));
  asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(b) : "f"(hi));
  return ((uint32_t)a & 0xFFu) | (((uint32_t)b & 0xFFu) << 8);
}
template <int VEC> __device__ __forceinline__ void store_codes(uint8_t* q, const float (&v)[VEC], int q_format) {
  if constexpr (VEC == 1) {
    q[0] = (uint8_t)code_pair(v[0], 0.0f, q_format);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      w[i] = code_pair(v[4 * i], v[4 * i + 1], q_format) | (code_pair(v[4 * i + 2], v[4 * i + 3], q_format) << 16);
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(q) = w[0];
  }
}

// the sums (and maxima) of the TPR threads of a row: shuffles, then one barrier
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, float& mx, float (*sm)[2]) {
  sum = warp_sum(sum);
  mx = warp_max_nan(mx);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
      sm[warp][0] = sum;
      sm[warp][1] = mx;
    }
    __syncthreads();
    sum = sm[0][0];
    mx = sm[0][1];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) {
      sum += sm[w][0];
      mx = max_nan(mx, sm[w][1]);
    }
  }
}

// One row for each TPR threads (a warp's rows: four to a CTA).  With h = x + residual in
// fp32, both the sum of squares and amax |h w| come from one pass over the row, so a row
// needs one reduction and one barrier: rstd = 1 / sqrt(mean h^2 + eps), and since rstd > 0
// is common to the row, amax |y| = rstd amax |h w|.  IT > 0: the products h w of the row
// stay in registers (IT vectors a thread) and memory is read once.  IT == 0, rows too long
// for that: the row is read again (residual_out is written in that second pass, by the
// thread that read the element, so it may be x or residual itself).
template <class T, int VEC, int TPR, int IT>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR)
norm_quant_kernel(const NormParams p) {
  __shared__ float sm[TPR / 32][2];
  const int t = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (TPR == 32 && row >= p.T) return;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  T* ho = p.residual_out ? static_cast<T*>(p.residual_out) + row * p.ldo : nullptr;
  uint8_t* q = p.q + row * p.H;
  constexpr int N = IT > 0 ? IT : 1;
  float hw[N][VEC];
  float sum = 0.0f, mx = 0.0f;
  auto take = [&](int col, float (&v)[VEC], bool store) {
    load_f<T, VEC>(x + col, v);
    if (r) {
      float a[VEC];
      load_f<T, VEC>(r + col, a);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] += a[j];
    }
    if (store && ho) store_f<T, VEC>(ho + col, v);
    float w[VEC];
    load_weight<T, VEC>(p, col, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if (IT > 0 || !store) sum = fmaf(v[j], v[j], sum);
      v[j] *= w[j];
      if (IT > 0 || !store) mx = max_nan(mx, fabsf(v[j]));
    }
  };
  if constexpr (IT > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int col = (i * TPR + t) * VEC;
      if (col < p.H) take(col, hw[i], true);
    }
  } else {
    for (int col = t * VEC; col < p.H; col += TPR * VEC) take(col, hw[0], false);
  }
  row_reduce<TPR>(sum, mx, sm);
  const float rstd = __frsqrt_rn(__fdiv_rn(sum, (float)p.H) + p.eps);
  // y / scale = ((h w) rstd) (1 / scale): two factors, as rstd / scale can pass fp32's range
  // where y does not
  float scale;
  if (p.scale) {
    scale = __ldg(p.scale);
  } else {
    scale = max_nan(__fdiv_rn(mx * rstd, p.qmax), kScaleMin);
    if (t == 0) p.scale_out[row] = scale;
  }
  const float inv = __fdiv_rn(1.0f, scale);
  if (t == 0) p.rstd[row] = rstd;
  if constexpr (IT > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int col = (i * TPR + t) * VEC;
      if (col < p.H) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) hw[i][j] = hw[i][j] * rstd * inv;
        store_codes<VEC>(q + col, hw[i], p.q_format);
      }
    }
  } else {
    for (int col = t * VEC; col < p.H; col += TPR * VEC) {
      take(col, hw[0], true);
#pragma unroll
      for (int j = 0; j < VEC; ++j) hw[0][j] = hw[0][j] * rstd * inv;
      store_codes<VEC>(q + col, hw[0], p.q_format);
    }
  }
}

template <class T, int VEC, int TPR, int IT> void launch_norm(const NormParams& p, cudaStream_t st) {
  const int64_t blocks = TPR == 32 ? (p.T + 3) / 4 : p.T;
  norm_quant_kernel<T, VEC, TPR, IT><<<(unsigned)blocks, TPR == 32 ? 128 : TPR, 0, st>>>(p);
}

// the fewest threads whose registers hold the row
template <class T> void pick_norm(const NormParams& p, bool vec, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    const int nv = p.H / V;
    if (nv <= 128) return launch_norm<T, V, 32, 4>(p, st);
    if (nv <= 256) return launch_norm<T, V, 128, 2>(p, st);
    if (nv <= 1024) return launch_norm<T, V, 256, 4>(p, st);
    if (nv <= 2048) return launch_norm<T, V, 512, 4>(p, st);
    return launch_norm<T, V, 512, 0>(p, st);
  }
  if (p.H <= 256) return launch_norm<T, 1, 32, 8>(p, st);
  if (p.H <= 2048) return launch_norm<T, 1, 256, 8>(p, st);
  if (p.H <= 8192) return launch_norm<T, 1, 1024, 8>(p, st);
  return launch_norm<T, 1, 1024, 0>(p, st);
}

// ------------------------------------------------------------------------- gradient
constexpr int kGradParts = 304;                   // two CTAs on each of 152 SMs

struct NormGradParams {
  const void* gy; int64_t ldy;
  const void* h; int64_t ldh;
  const void* gh; int64_t ldg;                    // null: none
  const void* weight; bool weight_f32;
  const float* rstd;
  int64_t T; int H;
  void* gx;                                       // [T, H] contiguous
  float* part;                                    // [gridDim.x, H]
};

// The gradient in one pass.  A CTA takes rows blockIdx.x, + gridDim.x, ...; a thread has IT vectors of
// columns, and keeps their weights and their sums of gy h rstd in registers over all its rows.  A
// row's sum of g h (g = gy w) has to be known before its first output, so a row is looked at twice:
// both times in shared memory, where a ring of S rows is filled ahead by bulk copies, so that HBM
// is read once and without a pause between rows.  (Rows that are not 16-byte aligned: `ring` false,
// read from memory twice.)  At the end the eight CTAs of a cluster add their column sums up
// through distributed shared memory, so that only gridDim / 8 parts of H sums go through memory to
// the joining kernel.  Bound by HBM: four tensors of T H values.
constexpr int kGradCluster = 8, kGradStages = 8;
template <class T, int VEC, int IT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
norm_grad_kernel(const NormGradParams p, int S) {
  constexpr bool RING = VEC > 1;
  extern __shared__ __align__(16) unsigned char dyn[];      // the ring; then the column sums, [H] fp32
  __shared__ float sm[2][32];
  __shared__ __align__(8) uint64_t full[kGradStages];
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5, warps = nt >> 5;
  const uint32_t row_bytes = (uint32_t)p.H * sizeof(T), inputs = p.gh ? 3u : 2u, stage_bytes = inputs * row_bytes;
  const int64_t rows = p.T > blockIdx.x ? (p.T - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  auto fill = [&](int64_t i, int s) {                       // one thread: row i of this CTA into stage s
    const int64_t row = blockIdx.x + i * gridDim.x;
    const uint32_t bar = smem_addr(&full[s]), dst = smem_addr(dyn) + s * stage_bytes;
    bar_expect(bar, stage_bytes);
    bulk_load(dst, static_cast<const T*>(p.gy) + row * p.ldy, row_bytes, bar);
    bulk_load(dst + row_bytes, static_cast<const T*>(p.h) + row * p.ldh, row_bytes, bar);
    if (p.gh) bulk_load(dst + 2 * row_bytes, static_cast<const T*>(p.gh) + row * p.ldg, row_bytes, bar);
  };
  if (RING) {
    if (t == 0) {
      for (int i = 0; i < S; ++i) bar_init(smem_addr(&full[i]), 1);
      bar_init_fence();
      for (int i = 0; i < S && i < rows; ++i) fill(i, i);
    }
    __syncthreads();
  }
  float w[IT][VEC], dw[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int col = (i * nt + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.0f;
    if (col < p.H) load_weight<T, VEC>(p, col, w[i]);
  }
  bool ok = true;
  int s = 0, before = S - 1;                                // row k's stage and row k - 1's
  uint32_t phase = 0;
  for (int64_t k = 0; k < rows; ++k) {
    const int64_t row = blockIdx.x + k * gridDim.x;
    const float rstd = p.rstd[row];
    const T *gy, *h, *gh = nullptr;
    if (RING) {
      ok = bar_wait(smem_addr(&full[s]), phase);
      gy = reinterpret_cast<const T*>(dyn + s * stage_bytes);
      h = gy + p.H;
      if (p.gh) gh = h + p.H;
    } else {
      gy = static_cast<const T*>(p.gy) + row * p.ldy;
      h = static_cast<const T*>(p.h) + row * p.ldh;
      if (p.gh) gh = static_cast<const T*>(p.gh) + row * p.ldg;
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int col = (i * nt + t) * VEC;
      if (col < p.H) {
        float y[VEC], x[VEC];
        load_f<T, VEC>(gy + col, y);
        load_f<T, VEC>(h + col, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum = fmaf(y[j] * w[i][j], x[j], sum);
      }
    }
    sum = warp_sum(sum);
    if (lane == 0) sm[k & 1][warp] = sum;                   // the other half of sm is the row before's
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    if (RING) {                                             // all are past the row before
      if (t == 0 && k >= 1 && k - 1 + S < rows) fill(k - 1 + S, before);
      before = s;
      if (++s == S) {
        s = 0;
        phase ^= 1u;
      }
    }
    sum = 0.0f;
    for (int i = 0; i < warps; ++i) sum += sm[k & 1][i];
    const float coef = __fdiv_rn(sum, (float)p.H) * rstd * rstd;
    T* gx = static_cast<T*>(p.gx) + row * p.H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int col = (i * nt + t) * VEC;
      if (col < p.H) {
        float y[VEC], x[VEC];
        load_f<T, VEC>(gy + col, y);
        load_f<T, VEC>(h + col, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          dw[i][j] = fmaf(y[j], x[j] * rstd, dw[i][j]);
          y[j] = rstd * (y[j] * w[i][j] - x[j] * coef);
        }
        if (gh) {
          load_f<T, VEC>(gh + col, x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) y[j] += x[j];
        }
        store_f<T, VEC>(gx + col, y);
      }
    }
  }
  if (!ok && t == 0) {                                      // a copy that never came: wait for the others, then end
    atomicExch(&g_norm_status, 1);
    for (int s = 0; s < S; ++s) {
      (void)bar_wait(smem_addr(&full[s]), 0);
      (void)bar_wait(smem_addr(&full[s]), 1);
    }
  }
  __syncthreads();
  float* const column_sums = reinterpret_cast<float*>(dyn);
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int col = (i * nt + t) * VEC + j;
      if (col < p.H) column_sums[col] = dw[i][j];
    }
  cluster_sync();
  const int rank = blockIdx.x % kGradCluster;
  for (int col = rank * nt + t; col < p.H; col += kGradCluster * nt) {
    float v[kGradCluster];
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r)
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(in_cluster(column_sums + col, r)) : "memory");
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r) s += v[r];
    p.part[(int64_t)(blockIdx.x / kGradCluster) * p.H + col] = s;
  }
  cluster_sync();
}

// Rows too long for a CTA's registers, in two passes over them.
//
// Row t: g = gy w, c = rstd^2 mean(g h), gx = rstd (g - h c) + gh.  One element a thread and
// step, the row read twice.
template <class T>
__global__ void __launch_bounds__(256)
norm_grad_rows_kernel(const NormGradParams p) {
  __shared__ float sm[8][2];
  const int64_t row = blockIdx.x;
  const T* gy = static_cast<const T*>(p.gy) + row * p.ldy;
  const T* h = static_cast<const T*>(p.h) + row * p.ldh;
  const T* gh = p.gh ? static_cast<const T*>(p.gh) + row * p.ldg : nullptr;
  T* gx = static_cast<T*>(p.gx) + row * p.H;
  auto weight = [&](int c) {
    return p.weight_f32 ? static_cast<const float*>(p.weight)[c] : to_f(static_cast<const T*>(p.weight)[c]);
  };
  float sum = 0.0f, none = 0.0f;
  for (int c = threadIdx.x; c < p.H; c += 256) sum = fmaf(to_f(gy[c]) * weight(c), to_f(h[c]), sum);
  row_reduce<256>(sum, none, sm);
  const float rstd = p.rstd[row];
  const float coef = __fdiv_rn(sum, (float)p.H) * rstd * rstd;
  for (int c = threadIdx.x; c < p.H; c += 256) {
    float v = rstd * (to_f(gy[c]) * weight(c) - to_f(h[c]) * coef);
    if (gh) v += to_f(gh[c]);
    gx[c] = from_f<T>(v);
  }
}
// part[b, c] = sum over the rows b, b + parts, ... of gy h rstd
template <class T>
__global__ void __launch_bounds__(256)
norm_grad_weight_kernel(const NormGradParams p) {
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= p.H) return;
  float acc = 0.0f;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x)
    acc = fmaf(to_f(static_cast<const T*>(p.gy)[row * p.ldy + c]),
               to_f(static_cast<const T*>(p.h)[row * p.ldh + c]) * p.rstd[row], acc);
  p.part[(int64_t)blockIdx.x * p.H + c] = acc;
}
// gw[c] = sum of the parts, in order: 32 columns a CTA, eight threads a column
__global__ void __launch_bounds__(256)
norm_grad_join_kernel(const float* part, int parts, int H, float* gw) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.0f;
  if (c < H)
    for (int b = g; b < parts; b += 8) acc += part[(int64_t)b * H + c];
  sm[g][lane] = acc;
  __syncthreads();
  if (g == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += sm[i][lane];
    gw[c] = acc;
  }
}

// Launches the kernel; the parts that it leaves for the joining kernel, 0 if it failed.
template <class T, int VEC, int IT, int MAXT, int MINB>
int launch_grad(const NormGradParams& p, int threads, cudaStream_t st) {
  auto kernel = norm_grad_kernel<T, VEC, IT, MAXT, MINB>;
  static std::atomic<bool> done[64];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(kernel), kMaxSmem - 1024, done)) return 0;
  // CTAs an SM by threads and registers (MAXT * MINB threads have theirs), and a ring that lets that many
  // share its memory: two rows at least, kGradStages at most
  int resident = MAXT * MINB / threads < 16 ? MAXT * MINB / threads : 16, S = 0;
  size_t bytes = (size_t)p.H * 4;
  if (VEC > 1) {
    const size_t stage = (size_t)p.H * sizeof(T) * (p.gh ? 3 : 2);
    while (resident > 1 && (kMaxSmem / resident - 2048) / stage < 3) --resident;
    S = (int)((kMaxSmem / resident - 2048) / stage);
    if (S > kGradStages) S = kGradStages;
    if (bytes < S * stage) bytes = S * stage;
  } else {
    while (resident > 1 && kMaxSmem / resident - 2048 < (int)bytes) --resident;
  }
  const int64_t most = (int64_t)emu_ops_sm_count() * resident;
  int64_t clusters = ((p.T < most ? p.T : most) + kGradCluster - 1) / kGradCluster;
  if (clusters > kGradParts) clusters = kGradParts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * kGradCluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kGradCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, S) == cudaSuccess ? (int)clusters : 0;
}

// The fewest vectors a thread that leave a CTA within its threads; 0: a launch failed.
template <class T> int pick_norm_grad(const NormGradParams& p, bool vec, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  auto threads = [](int n, int it) { return ((n + it - 1) / it + 31) / 32 * 32; };
  if (vec) {
    const int nv = p.H / V;
    if (nv <= 256) return launch_grad<T, V, 1, 256, 5>(p, threads(nv, 1), st);
    if (nv <= 1024) return launch_grad<T, V, 2, 512, 2>(p, threads(nv, 2), st);
    if (nv <= 2048) return launch_grad<T, V, 4, 512, 1>(p, threads(nv, 4), st);
  } else if (p.H <= 8192) {
    return p.H <= 2048 ? launch_grad<T, 1, 8, 256, 4>(p, threads(p.H, 8), st)
                       : launch_grad<T, 1, 8, 1024, 1>(p, threads(p.H, 8), st);
  }
  const int parts = (int)(p.T < kGradParts ? p.T : kGradParts);
  norm_grad_rows_kernel<T><<<(unsigned)p.T, 256, 0, st>>>(p);
  norm_grad_weight_kernel<T><<<dim3((unsigned)parts, (unsigned)((p.H + 255) / 256)), 256, 0, st>>>(p);
  return parts;
}

int check_rows(const char* what, int64_t T, int64_t H) {
  if (T < 0 || H < 1) return emu_ops_fail(EMU_EINVAL, "%s: sizes (%lld, %lld)", what, (long long)T, (long long)H);
  if (T >= ((int64_t)1 << 31) || H > (1 << 22))
    return emu_ops_fail(EMU_EUNSUPPORTED, "%s: at most 2^31 - 1 rows of 2^22 values", what);
  return EMU_OK;
}

}  // namespace emu_ops

using namespace emu_ops;

extern "C" {

const char* emu_ops_last_error(void) { return g_ops_error.c_str(); }

int emu_ops_device_status(int32_t* status, int32_t reset) {
  emu_ops_begin();
  if (!status) return emu_ops_fail(EMU_EINVAL, "status is null");
  int v = 0;
  const int rc = emu_ops_int8_status(&v, reset != 0);
  if (rc != EMU_OK) return rc;
  int n = 0;
  if (cudaMemcpyFromSymbol(&n, g_norm_status, sizeof n) != cudaSuccess) return emu_ops_launched("emu_ops_device_status");
  const int zero = 0;
  if (reset && cudaMemcpyToSymbol(g_norm_status, &zero, sizeof zero) != cudaSuccess)
    return emu_ops_launched("emu_ops_device_status");
  *status = v | n;
  return EMU_OK;
}

int emu_rms_norm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                       const void* weight, emu_out_t weight_type, emu_out_t type, int64_t T, int64_t H,
                       float eps, const float* scale, emu_q_t q_format, void* q, float* scale_out,
                       void* residual_out, int64_t ldo, float* rstd, void* stream) {
  emu_ops_begin();
  int rc = check_rows("emu_rms_norm_quant", T, H);
  if (rc != EMU_OK) return rc;
  if (!is_float_type(type)) return emu_ops_fail(EMU_EINVAL, "unknown element type %d", (int)type);
  if (weight_type != type && weight_type != EMU_OUT_F32)
    return emu_ops_fail(EMU_EINVAL, "the weight is of x's type or fp32 (got %d)", (int)weight_type);
  if ((int)q_format < 0 || (int)q_format > 2) return emu_ops_fail(EMU_EINVAL, "unknown 8-bit format %d", (int)q_format);
  if (!(eps >= 0.0f)) return emu_ops_fail(EMU_EINVAL, "eps must be at least 0");
  if (T == 0) return EMU_OK;
  if (!x || !weight || !q || !rstd) return emu_ops_fail(EMU_EINVAL, "null x, weight, q or rstd");
  if (!scale && !scale_out) return emu_ops_fail(EMU_EINVAL, "neither a scale nor a place for the rows' scales");
  if (ldx < H || (residual && ldr < H) || (residual_out && ldo < H))
    return emu_ops_fail(EMU_EINVAL, "a row stride is below the row's %lld values", (long long)H);
  const size_t es = elem_bytes(type);
  const void* bases[3] = {x, residual, residual_out};
  for (const void* b : bases)
    if (!aligned(b, es)) return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  if (!aligned(weight, elem_bytes(weight_type)) || !aligned(rstd, 4) || !aligned(scale, 4) || !aligned(scale_out, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  if (residual_out) {
    // an output row may replace its input row, and may not meet any other
    const Span o(residual_out, T, ldo, H, es);
    if ((o.meets(Span(x, T, ldx, H, es)) && !(residual_out == x && ldo == ldx)) ||
        (residual && o.meets(Span(residual, T, ldr, H, es)) && !(residual_out == residual && ldo == ldr)))
      return emu_ops_fail(EMU_EINVAL, "residual_out overlaps an input without being that input");
  }
  NormParams p;
  p.x = x; p.ldx = ldx;
  p.residual = residual; p.ldr = ldr;
  p.weight = weight; p.weight_f32 = weight_type == EMU_OUT_F32;
  p.T = T; p.H = (int)H; p.eps = eps;
  p.qmax = q_format == EMU_Q_E4M3FN ? 448.0f : q_format == EMU_Q_E5M2 ? 57344.0f : 127.0f;
  p.scale = scale; p.q_format = (int)q_format;
  p.q = static_cast<uint8_t*>(q); p.scale_out = scale_out;
  p.residual_out = residual_out; p.ldo = ldo; p.rstd = rstd;
  const int64_t v = 16 / (int64_t)es;
  const bool vec = H % v == 0 && ldx % v == 0 && (!residual || ldr % v == 0) && (!residual_out || ldo % v == 0) &&
                   aligned(x, 16) && aligned(residual, 16) && aligned(residual_out, 16) && aligned(weight, 16) &&
                   aligned(q, (size_t)v);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == EMU_OUT_F32) pick_norm<float>(p, vec, st);
  else if (type == EMU_OUT_BF16) pick_norm<__nv_bfloat16>(p, vec, st);
  else pick_norm<__half>(p, vec, st);
  return emu_ops_launched("emu_rms_norm_quant");
}

size_t emu_rms_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T < 1 || H < 1 || H > (1 << 22)) return 0;
  return (size_t)(T < kGradParts ? T : kGradParts) * (size_t)H * sizeof(float);
}

int emu_rms_norm_backward(const void* grad_y, int64_t ldy, const void* hidden, int64_t ldh,
                          const float* rstd, const void* weight, emu_out_t weight_type,
                          const void* grad_residual, int64_t ldg, emu_out_t type, int64_t T, int64_t H,
                          void* grad_x, float* grad_weight, void* workspace, size_t workspace_bytes,
                          void* stream) {
  emu_ops_begin();
  int rc = check_rows("emu_rms_norm_backward", T, H);
  if (rc != EMU_OK) return rc;
  if (!is_float_type(type)) return emu_ops_fail(EMU_EINVAL, "unknown element type %d", (int)type);
  if (weight_type != type && weight_type != EMU_OUT_F32)
    return emu_ops_fail(EMU_EINVAL, "the weight is of grad_y's type or fp32 (got %d)", (int)weight_type);
  if (!grad_weight || !aligned(grad_weight, 4)) return emu_ops_fail(EMU_EINVAL, "null or misaligned grad_weight");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {                                    // the sum over no rows
    if (cudaMemsetAsync(grad_weight, 0, (size_t)H * 4, st) != cudaSuccess) return emu_ops_launched("emu_rms_norm_backward");
    return EMU_OK;
  }
  if (!grad_y || !hidden || !rstd || !weight || !grad_x) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (ldy < H || ldh < H || (grad_residual && ldg < H))
    return emu_ops_fail(EMU_EINVAL, "a row stride is below the row's %lld values", (long long)H);
  const size_t es = elem_bytes(type);
  if (!aligned(grad_y, es) || !aligned(hidden, es) || !aligned(grad_residual, es) || !aligned(grad_x, es) ||
      !aligned(weight, elem_bytes(weight_type)) || !aligned(rstd, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  const Span o(grad_x, T, H, H, es);
  if (o.meets(Span(grad_y, T, ldy, H, es)) || o.meets(Span(hidden, T, ldh, H, es)) ||
      (grad_residual && o.meets(Span(grad_residual, T, ldg, H, es))))
    return emu_ops_fail(EMU_EINVAL, "grad_x overlaps an input");
  const size_t need = emu_rms_norm_backward_workspace_bytes(T, H);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return emu_ops_fail(EMU_EINVAL, "workspace of %zu bytes needed, 16-byte aligned (got %zu)", need, workspace_bytes);
  NormGradParams p;
  p.gy = grad_y; p.ldy = ldy; p.h = hidden; p.ldh = ldh; p.gh = grad_residual; p.ldg = ldg;
  p.weight = weight; p.weight_f32 = weight_type == EMU_OUT_F32; p.rstd = rstd;
  p.T = T; p.H = (int)H; p.gx = grad_x; p.part = static_cast<float*>(workspace);
  const int64_t v = 16 / (int64_t)es;
  const bool vec = H % v == 0 && ldy % v == 0 && ldh % v == 0 && (!grad_residual || ldg % v == 0) && aligned(grad_y, 16) &&
                   aligned(hidden, 16) && aligned(grad_residual, 16) && aligned(grad_x, 16) && aligned(weight, 16);
  const int parts = type == EMU_OUT_F32    ? pick_norm_grad<float>(p, vec, st)
                    : type == EMU_OUT_BF16 ? pick_norm_grad<__nv_bfloat16>(p, vec, st)
                                           : pick_norm_grad<__half>(p, vec, st);
  if (parts == 0) return emu_ops_launched("emu_rms_norm_backward");
  norm_grad_join_kernel<<<(unsigned)((H + 31) / 32), 256, 0, st>>>(p.part, parts, p.H, grad_weight);
  return emu_ops_launched("emu_rms_norm_backward");
}

}  // extern "C"
