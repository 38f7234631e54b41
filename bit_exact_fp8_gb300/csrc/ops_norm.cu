// ops_norm.cu -- RMS norm with the residual's addition and an 8-bit output, and its
// gradient (declared in include/emu_fp8.h); and the host side that the operators share.
#include "ops_common.cuh"

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <string>
#include <type_traits>

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

// A row's rstd, scale and the two factors of its codes, given its sum of squares and its largest |h w|: the same
// roundings in every kernel.  H and qmax divide as factors (their quotients, and a correctly rounded root, are on
// every row's way from its last load to its first code: 8192 x 5760 bf16 57.2 us a call with them, 54.9 with
// factors).  A code is the rounding of ((h w) a) b, where a b = num / den is
//   a row's own scale: qmax / max|h w|, which is rstd / scale without the roundings of either;
//   a given scale, or a row's at its least: rstd / scale.
// a is the power of two that brings den to [1, 2), so that b is in range whatever the two are ((h w) a passes
// fp32's only where y / scale is far above every code, or far below).
struct RowRule {
  float inv_h, inv_qmax, qmax, eps;
  // NaN where the sum is none: rstd = 0 would make a row past fp32's range look like one of zeros
  __device__ __forceinline__ float rstd(float sum) const { return sum < INFINITY ? rsqrtf(fmaf(sum, inv_h, eps)) : NAN; }
  __device__ __forceinline__ float scale(float mx, float rstd) const { return max_nan(mx * rstd * inv_qmax, kScaleMin); }
  __device__ __forceinline__ void factors(float mx, float rstd, float scale, bool given, float& a, float& b) const {
    const bool own = !given && scale > kScaleMin;            // not at its least, nor NaN
    const float den = own ? mx : scale;
    const uint32_t e = (__float_as_uint(den) >> 23) & 0xFFu;
    a = __uint_as_float((254u - min(max(e, 1u), 253u)) << 23);
    b = __fdiv_rn(own ? qmax : rstd, den * a);
  }
};
__device__ __forceinline__ RowRule rule_of(const NormParams& p) {
  return RowRule{__fdiv_rn(1.0f, (float)p.H), __fdiv_rn(1.0f, p.qmax), p.qmax, p.eps};
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

// ---- rows through shared memory.  A row of a tensor is held as the 16-byte vectors that it touches:
// vector v has the values of columns v * VEC - off + j, `off` values of the row before it in its
// first one.  Tensors whose rows lie alike about 16-byte addresses share off, and the rows
// of one CTA (a multiple of 8 apart) do too, so a thread's columns, weights and sums of columns
// stay its own over all its rows, whatever the row's length.
constexpr int kStages = 8;
struct Ring {
  int S;                        // rows held at once
  uint32_t pitch;               // bytes of one row's vectors
  bool q_vec;                   // codes can be stored a vector at a time
};
// EDGES: rows that begin or end inside a vector
template <class T, bool EDGES> struct Columns {
  static constexpr int VEC = 16 / sizeof(T);
  int first, lo, hi;            // of a thread's vector: the column of value 0, its valid values [lo, hi)
  __device__ __forceinline__ Columns(int v, int off, int H) : first(v * VEC - (EDGES ? off : 0)) {
    lo = EDGES && first < 0 ? -first : 0;
    hi = !EDGES ? (first < H ? VEC : 0) : H - first < VEC ? H - first : VEC;
  }
  __device__ __forceinline__ bool any() const { return hi > lo; }
  __device__ __forceinline__ bool whole() const { return !EDGES || (lo == 0 && hi == VEC); }
};
// One thread: row `row` of a [rows, H] tensor into shared memory at dst, by a bulk copy of the vectors
// that lie within the tensor; values of others (the tensor's very ends) one by one.
template <class T>
__device__ __forceinline__ void fill_row(unsigned char* dst, const T* base, int64_t ld, int64_t row, int64_t rows, int H,
                                         uint32_t bar) {
  const uintptr_t start = reinterpret_cast<uintptr_t>(base + row * ld), end = start + (size_t)H * sizeof(T);
  const uintptr_t tensor_end = reinterpret_cast<uintptr_t>(base + (rows - 1) * ld) + (size_t)H * sizeof(T);
  const uintptr_t from = start & ~(uintptr_t)15;
  uintptr_t lo = from, hi = (end + 15) & ~(uintptr_t)15;
  if (lo < reinterpret_cast<uintptr_t>(base)) lo += 16;
  if (hi > tensor_end) hi -= 16;
  if (lo > start || hi < end) {
    for (uintptr_t a = start; a < end && a < lo; a += sizeof(T))
      *reinterpret_cast<T*>(dst + (a - from)) = *reinterpret_cast<const T*>(a);
    for (uintptr_t a = hi > start ? hi : start; a < end; a += sizeof(T))
      if (a >= lo) *reinterpret_cast<T*>(dst + (a - from)) = *reinterpret_cast<const T*>(a);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before a later row's copy takes their place
  }
  const uint32_t bytes = hi > lo ? (uint32_t)(hi - lo) : 0u;
  bar_expect(bar, bytes);
  if (bytes) bulk_load(smem_addr(dst + (lo - from)), reinterpret_cast<const void*>(lo), bytes, bar);
}
template <class T> __device__ __forceinline__ int offset_of(const void* base, int64_t ld, int64_t row) {
  return (int)((reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld) & 15u) / sizeof(T));
}
// a thread's vector from shared memory as pairs; values outside the row as 0
template <class T, bool EDGES>
__device__ __forceinline__ void read_pairs(const unsigned char* at, const Columns<T, EDGES>& c, f2 (&f)[8 / sizeof(T)]) {
  constexpr int VEC = Columns<T, EDGES>::VEC;
  float v[VEC];
  load_f<T, VEC>(reinterpret_cast<const T*>(at), v);
  if (!c.whole()) {
    asm volatile("");           // a branch for the two vectors of a row, not selects for all
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = j >= c.lo && j < c.hi ? v[j] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < VEC; j += 2) f[j / 2] = pair(v[j], v[j + 1]);
}
template <class T, bool EDGES>
__device__ __forceinline__ void write_pairs(T* row, const Columns<T, EDGES>& c, const f2 (&f)[8 / sizeof(T)]) {
  constexpr int VEC = Columns<T, EDGES>::VEC;
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; j += 2) halves(f[j / 2], v[j], v[j + 1]);
  if (c.whole()) {
    store_f<T, VEC>(row + c.first, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (j >= c.lo && j < c.hi) row[c.first + j] = from_f<T>(v[j]);
  }
}
template <class T, bool EDGES, class P>
__device__ __forceinline__ void weight_pairs(const P& p, const Columns<T, EDGES>& c, f2 (&w)[8 / sizeof(T)]) {
  constexpr int VEC = Columns<T, EDGES>::VEC;
  float v[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    v[j] = 0.0f;
    if (j >= c.lo && j < c.hi)
      v[j] = p.weight_f32 ? static_cast<const float*>(p.weight)[c.first + j]
                          : to_f(static_cast<const T*>(p.weight)[c.first + j]);
  }
#pragma unroll
  for (int j = 0; j < VEC; j += 2) w[j / 2] = pair(v[j], v[j + 1]);
}
// the sum of what the first `warps` warps left in part (16 places, zeros after theirs)
__device__ __forceinline__ float sum16(const float* part) {
  const float4* q = reinterpret_cast<const float4*>(part);
  const float4 a = q[0], b = q[1], c = q[2], d = q[3];
  return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w)) + (((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w)));
}

__device__ __forceinline__ float max16(const float* part) {
  const float4* q = reinterpret_cast<const float4*>(part);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_nan(m, max_nan(max_nan(q[i].x, q[i].y), max_nan(q[i].z, q[i].w)));
  return m;
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

// ---- the order of a row's sum of squares, the same in every kernel and at every address, so that a row's
// rstd, scale and codes are its own wherever it stands.  The columns are taken in blocks of VEC, and block b
// belongs to thread b % N (N: split_of() below, by the row's length alone).  A block's squares are added from its
// last column to its first, even and odd columns apart (the halves of a pair), a thread's blocks in rising
// order, then the halves, the lanes by shuffles and the warps by sum16.
template <int NP> __device__ __forceinline__ f2 add_squares(const f2 (&q)[NP], f2 s) {
#pragma unroll
  for (int j = NP - 1; j >= 0; --j) s = fma2(q[j], q[j], s);
  return s;
}
struct Split {
  int it, threads;              // blocks a thread (0: as many as it takes) and threads a row
};
int threads_for(int n, int it) { return ((n + it - 1) / it + 31) / 32 * 32; }
template <class T> Split split_of(int H) {
  const int V = 16 / (int)sizeof(T), n = (H + V - 1) / V;
  return n <= 256 ? Split{2, threads_for(n, 2)} : n <= 2048 ? Split{4, threads_for(n, 4)} : Split{0, 512};
}

// A row a warp (TPR 32, four rows to a CTA) or a CTA of up to TPR threads, straight from memory.  With
// h = x + residual in fp32, both the sum of squares and max|h w| come from one pass over the row, so a row needs
// one reduction and one barrier.  IT > 0: the products h w of the row stay in registers (IT blocks a thread) and
// memory is read once.  IT == 0, rows too long for that: the row is read again (residual_out is written in that
// second pass, by the thread that read the element, so it may be x or residual itself).  VECS: a thread
// loads its blocks as vectors.  Else, where rows are not aligned, a warp loads its 32 blocks element by
// element, 32 neighbours at a time, and turns them round in shared memory for the sum.
template <class T, bool VECS, int TPR, int IT, int J>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR)
norm_quant_kernel(const NormParams p) {
  constexpr int VEC = 16 / sizeof(T), NP = VEC / 2, WARPS = TPR == 32 ? 4 : TPR / 32;
  __shared__ __align__(16) float sums[16], tops[16];
  __shared__ __align__(16) float turn_all[VECS ? 1 : WARPS][VECS ? 4 : 32 * VEC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = TPR == 32 ? lane : threadIdx.x, n = TPR == 32 ? 32 : IT == 0 ? TPR : blockDim.x;
  const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 4 + warp : (int64_t)blockIdx.x;
  if (TPR == 32 && row >= p.T) return;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  T* ho = p.residual_out ? static_cast<T*>(p.residual_out) + row * p.ldo : nullptr;
  uint8_t* q = p.q + row * p.H;
  float* turn = turn_all[VECS ? 0 : warp];
  // slot i: this thread's first column, and how far apart its J columns are (J < VEC: rows that end within so many)
  auto first_of = [&](int i) { return VECS ? (i * n + t) * VEC : (i * n + (t & ~31)) * VEC + lane; };
  constexpr int APART = VECS ? 1 : 32;
  constexpr int N = IT > 0 ? IT : 1;
  float hw[N][J];
  float mx = 0.0f;
  f2 sq[2] = {0ull, 0ull};                                  // [1]: a warp's rows of 64 threads' blocks, the second 32's
  // slot i of h into v (columns past the row: 0)
  auto load = [&](int i, float (&v)[J]) {
    const int col = first_of(i);
    if constexpr (VECS) {
      if (col >= p.H) return;
      load_f<T, VEC>(x + col, v);
      if (r) {
        float a[VEC];
        load_f<T, VEC>(r + col, a);
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] += a[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = col + j * APART;
        v[j] = c < p.H ? to_f(x[c]) : 0.0f;
        if (r && c < p.H) v[j] += to_f(r[c]);
      }
    }
  };
  auto keep = [&](int i, const float (&v)[J]) {           // to residual_out
    const int col = first_of(i);
    if constexpr (VECS) {
      if (col < p.H) store_f<T, VEC>(ho + col, v);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (col + j * APART < p.H) ho[col + j * APART] = from_f<T>(v[j]);
    }
  };
  // h w in the place of h; in the summing pass h counts in the sum, and h w in the maximum
  auto weigh = [&](int i, float (&v)[J], bool sum) {
    const int col = first_of(i);
    if (VECS && col >= p.H) return;
    if (sum) {
      f2 h[NP];
      if constexpr (!VECS) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j) turn[j * 32 + lane] = v[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < VEC; j += 2)
          h[j / 2] = lane * VEC < J * 32 ? pair(turn[lane * VEC + j], turn[lane * VEC + j + 1]) : 0ull;
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) h[j / 2] = pair(v[j], v[j + 1]);
      }
      sq[IT == 3 ? i & 1 : 0] = add2(sq[IT == 3 ? i & 1 : 0], add_squares(h, 0ull));
    }
    float w[J];
    if constexpr (VECS) {
      load_weight<T, VEC>(p, col, w);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = col + j * APART;
        w[j] = c >= p.H ? 0.0f : p.weight_f32 ? static_cast<const float*>(p.weight)[c] : to_f(static_cast<const T*>(p.weight)[c]);
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      v[j] *= w[j];
      if (sum) mx = max_nan(mx, fabsf(v[j]));
    }
  };
  auto live = [&](int i) { return (VECS ? first_of(i) : (i * n + (t & ~31)) * VEC) < p.H; };   // by elements: the warp's
  if constexpr (IT > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (live(i)) load(i, hw[i]);
    if (ho)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (live(i)) keep(i, hw[i]);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (live(i)) weigh(i, hw[i], true);
  } else {
#pragma unroll 4
    for (int i = 0; live(i); ++i) {
      load(i, hw[0]);
      weigh(i, hw[0], true);
    }
  }
  float s0, s1;
  halves(sq[0], s0, s1);
  float sum = warp_sum(s0 + s1);
  if constexpr (IT == 3) {
    halves(sq[1], s0, s1);
    sum += warp_sum(s0 + s1);
  }
  mx = warp_max_nan(mx);
  if constexpr (TPR > 32) {
    if (lane == 0) {
      sums[warp] = sum;
      tops[warp] = mx;
    }
    if (t < 16 && t >= n / 32) sums[t] = tops[t] = 0.0f;
    __syncthreads();
    sum = sum16(sums);
    mx = max16(tops);
  }
  const RowRule rule = rule_of(p);
  const float rstd = rule.rstd(sum);
  const float scale = p.scale ? __ldg(p.scale) : rule.scale(mx, rstd);
  if (t == 0 && !p.scale) p.scale_out[row] = scale;
  float fa, fb;
  rule.factors(mx, rstd, scale, p.scale != nullptr, fa, fb);
  if (t == 0) p.rstd[row] = rstd;
  auto put = [&](int i, float (&v)[J]) {
    const int col = first_of(i);
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = v[j] * fa * fb;
    if constexpr (VECS) {
      if (col < p.H) store_codes<VEC>(q + col, v, p.q_format);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (col + j * APART < p.H) q[col + j * APART] = (uint8_t)code_pair(v[j], 0.0f, p.q_format);
    }
  };
  if constexpr (IT > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (live(i)) put(i, hw[i]);
  } else {
    for (int i = 0; live(i); ++i) {
      load(i, hw[0]);
      if (ho) keep(i, hw[0]);
      weigh(i, hw[0], false);
      put(i, hw[0]);
    }
  }
}

template <class T, bool VECS, int TPR, int IT, int J = 16 / (int)sizeof(T)> void launch_norm(const NormParams& p, cudaStream_t st) {
  const int64_t blocks = TPR == 32 ? (p.T + 3) / 4 : p.T;
  norm_quant_kernel<T, VECS, TPR, IT, J><<<(unsigned)blocks, TPR == 32 ? 128 : split_of<T>(p.H).threads, 0, st>>>(p);
}

// Many rows: a CTA takes rows blockIdx.x, + gridDim.x, ..., staged ahead in a ring in shared memory by
// bulk copies, so that HBM is read without a pause between rows; a thread keeps the weights of its
// IT vectors of columns in registers.  The rest is as above.  Bound by HBM: x, residual, h and q.
template <class T, int IT, int MAXT, int MINB, bool EDGES>
__global__ void __launch_bounds__(MAXT, MINB)
norm_quant_ring_kernel(const NormParams p, const Ring ring) {
  constexpr int VEC = 16 / sizeof(T), NP = VEC / 2;
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ __align__(16) float sums[2][16], tops[2][16];
  __shared__ __align__(8) uint64_t full[kStages];
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
  const int inputs = p.residual ? 2 : 1;
  const uint32_t stage_bytes = (uint32_t)inputs * ring.pitch;
  const int rows = (int)(p.T > blockIdx.x ? (p.T - blockIdx.x + gridDim.x - 1) / gridDim.x : 0);
  const int second = nt > 32 ? 32 : 1;                      // the thread that fetches the residual
  auto fill = [&](int i, int s) {
    const int64_t row = blockIdx.x + (int64_t)i * gridDim.x;
    unsigned char* dst = dyn + s * stage_bytes;
    if (t == 0) fill_row(dst, static_cast<const T*>(p.x), p.ldx, row, p.T, p.H, smem_addr(&full[s]));
    else fill_row(dst + ring.pitch, static_cast<const T*>(p.residual), p.ldr, row, p.T, p.H, smem_addr(&full[s]));
  };
  const bool fetches = t == 0 || (t == second && inputs == 2);
  if (t < 16) sums[0][t] = sums[1][t] = tops[0][t] = tops[1][t] = 0.0f;
  if (t == 0) {
    for (int i = 0; i < ring.S; ++i) bar_init(smem_addr(&full[i]), inputs);
    bar_init_fence();
  }
  __syncthreads();
  if (fetches)
    for (int i = 0; i < ring.S && i < rows; ++i) fill(i, i);
  const int off = offset_of<T>(p.x, p.ldx, blockIdx.x);
  f2 w[IT][NP];
#pragma unroll
  for (int i = 0; i < IT; ++i) weight_pairs(p, Columns<T, EDGES>(i * nt + t, off, p.H), w[i]);
  f2 tail[NP];                                              // 1 for a vector's first off values, else 0
#pragma unroll
  for (int j = 0; j < NP; ++j) tail[j] = pair(2 * j < off ? 1.0f : 0.0f, 2 * j + 1 < off ? 1.0f : 0.0f);
  // a row that begins inside its first vector may end in one past the threads': its few columns, one a thread
  const int late = IT * nt * VEC - off + t;
  const bool has_late = EDGES && late < p.H;
  const float late_w = !has_late ? 0.0f : p.weight_f32 ? static_cast<const float*>(p.weight)[late]
                                                      : to_f(static_cast<const T*>(p.weight)[late]);
  const RowRule rule = rule_of(p);
  const float given = p.scale ? __ldg(p.scale) : 0.0f;
  bool ok = true;
  int s = 0, before = ring.S - 1;
  uint32_t phase = 0;
  for (int k = 0; k < rows; ++k) {
    const int64_t row = blockIdx.x + (int64_t)k * gridDim.x;
    ok = bar_wait(smem_addr(&full[s]), phase);
    const unsigned char* in = dyn + s * stage_bytes;
    T* ho = p.residual_out ? static_cast<T*>(p.residual_out) + row * p.ldo : nullptr;
    f2 hw[IT][NP], sq = 0ull;
    float mx = 0.0f, late_hw = 0.0f;
    // vector v of the row as h = x + residual
    auto read_h = [&](int v, const Columns<T, EDGES>& c, f2 (&h)[NP]) {
      read_pairs(in + v * 16, c, h);
      if (inputs == 2) {
        f2 r[NP];
        read_pairs(in + ring.pitch + v * 16, c, r);
#pragma unroll
        for (int j = 0; j < NP; ++j) h[j] = add2(h[j], r[j]);
      }
    };
    // of the vectors after the warp's last ones, a slot a lane: the sums of the columns of the blocks before them
    f2 next = 0ull;
    if (EDGES && off != 0 && lane < IT) {
      const int v = lane * nt + (t & ~31) + 32;
      const Columns<T, EDGES> c(v, off, p.H);
      if (c.any()) {
        const int most = off < c.hi ? off : c.hi;
        float x[VEC], r[VEC];
        load_f<T, VEC>(reinterpret_cast<const T*>(in + v * 16), x);
        if (inputs == 2) load_f<T, VEC>(reinterpret_cast<const T*>(in + ring.pitch + v * 16), r);
        f2 h[NP];
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          if (inputs == 2) {
            x[j] += r[j];
            x[j + 1] += r[j + 1];
          }
          h[j / 2] = pair(j < most ? x[j] : 0.0f, j + 1 < most ? x[j + 1] : 0.0f);
        }
        next = add_squares(h, 0ull);
      }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int v = i * nt + t;
      const Columns<T, EDGES> c(v, off, p.H);
      if (!EDGES && !c.any()) continue;
      // none of the warp's (asked in the last slot of four, which is often so: 8192 x 4097 bf16 64 us, 74 without;
      // asked in each slot it costs more than it spares where there are columns)
      if (EDGES && IT > 2 && i == IT - 1 && (v - lane) * VEC - off >= p.H) continue;
      if (c.any()) read_h(v, c, hw[i]);
      if constexpr (EDGES) {
        if (!c.any()) {
#pragma unroll
          for (int j = 0; j < NP; ++j) hw[i][j] = 0ull;
        }
      }
      if (!EDGES || off == 0) {
        sq = add2(sq, add_squares(hw[i], 0ull));
      } else {
        // This vector holds the last off columns of the block before and the first ones of its own: the former's
        // sum goes to the lane before, which goes on with it.
        f2 mine[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) mine[j] = mul2(hw[i][j], tail[j]);
        f2 after = __shfl_down_sync(0xFFFFFFFFu, add_squares(mine, 0ull), 1);
        const f2 from_next = __shfl_sync(0xFFFFFFFFu, next, i);
        if (lane == 31) after = from_next;
#pragma unroll
        for (int j = 0; j < NP; ++j) mine[j] = fma2(mine[j], pair(-1.0f, -1.0f), hw[i][j]);
        sq = add2(sq, add_squares(mine, after));
        if (!c.any()) continue;
      }
      if (ho && c.any()) write_pairs(ho, c, hw[i]);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        hw[i][j] = mul2(hw[i][j], w[i][j]);
        float a, b;
        halves(hw[i][j], a, b);
        mx = max_nan(mx, max_nan(fabsf(a), fabsf(b)));
      }
    }
    if (has_late) {
      const T* from = reinterpret_cast<const T*>(in + IT * nt * 16) + t;
      float h = to_f(*from);
      if (inputs == 2) h += to_f(*reinterpret_cast<const T*>(reinterpret_cast<const unsigned char*>(from) + ring.pitch));
      if (ho) ho[late] = from_f<T>(h);
      late_hw = h * late_w;
      mx = max_nan(mx, fabsf(late_hw));
    }
    float s0, s1;
    halves(sq, s0, s1);
    const float part = warp_sum(s0 + s1);
    mx = warp_max_nan(mx);
    if (lane == 0) {                                        // the other halves are the row before's
      sums[k & 1][warp] = part;
      tops[k & 1][warp] = mx;
    }
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    if (fetches && k >= 1 && k - 1 + ring.S < rows) fill(k - 1 + ring.S, before);   // all are past the row before
    before = s;
    if (++s == ring.S) {
      s = 0;
      phase ^= 1u;
    }
    const float rstd = rule.rstd(sum16(sums[k & 1]));
    const float top = max16(tops[k & 1]), scale = p.scale ? given : rule.scale(top, rstd);
    if (t == 0 && !p.scale) p.scale_out[row] = scale;
    float fa, fb;
    rule.factors(top, rstd, scale, p.scale != nullptr, fa, fb);
    if (t == 0) p.rstd[row] = rstd;
    uint8_t* q = p.q + row * p.H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Columns<T, EDGES> c(i * nt + t, off, p.H);
      if (!c.any()) continue;
      float v[VEC];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        float a, b;
        halves(hw[i][j], a, b);
        v[2 * j] = a * fa * fb;
        v[2 * j + 1] = b * fa * fb;
      }
      if (ring.q_vec && c.whole()) {
        store_codes<VEC>(q + c.first, v, p.q_format);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (j >= c.lo && j < c.hi) q[c.first + j] = (uint8_t)code_pair(v[j], 0.0f, p.q_format);
      }
    }
    if (has_late) q[late] = (uint8_t)code_pair(late_hw * fa * fb, 0.0f, p.q_format);
  }
  if (!ok && t == 0) {                                      // a copy that never came: wait for the others, then end
    atomicExch(&g_norm_status, 1);
    for (int i = 0; i < ring.S; ++i) {
      (void)bar_wait(smem_addr(&full[i]), 0);
      (void)bar_wait(smem_addr(&full[i]), 1);
    }
  }
}

// The ring for rows of `inputs` tensors in CTAs of `threads` threads, of which registers let `most` live
// on an SM: CTAs an SM (at least three rows in each, if that leaves one) and rows a CTA.
Ring ring_for(int64_t H, size_t es, bool aligned16, int inputs, int most, int* resident) {
  Ring r = {};
  r.pitch = (uint32_t)((size_t)H * es);
  if (!aligned16) r.pitch = (r.pitch + 30u) & ~15u;
  const size_t stage = (size_t)inputs * r.pitch;
  int n = most < 16 ? most : 16;
  while (n > 1 && (size_t)(kMaxSmem / n - 2048) / stage < 3) --n;
  const size_t S = (size_t)(kMaxSmem / n - 2048) / stage;
  r.S = S < kStages ? (int)S : kStages;
  *resident = n;
  return r;
}

// MINB and EDGEB: the CTAs of MAXT threads that registers let live on an SM, of aligned rows and of others
template <class T, int IT, int MAXT, int MINB, int EDGEB>
int launch_norm_ring(const NormParams& p, int threads, bool aligned16, bool q_vec, cudaStream_t st) {
  auto kernel = aligned16 ? norm_quant_ring_kernel<T, IT, MAXT, MINB, false> : norm_quant_ring_kernel<T, IT, MAXT, EDGEB, true>;
  static std::atomic<bool> flags[2][64];
  std::atomic<bool>* done = flags[aligned16];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(kernel), kMaxSmem - 1024, done))
    return emu_ops_launched("cudaFuncSetAttribute");
  int resident;
  Ring ring = ring_for(p.H, sizeof(T), aligned16, p.residual ? 2 : 1, MAXT * (aligned16 ? MINB : EDGEB) / threads, &resident);
  ring.q_vec = q_vec;
  const int64_t most = (int64_t)emu_ops_sm_count() * resident;
  int64_t ctas = p.T < most ? p.T : most;
  if (!aligned16) ctas = (ctas + 7) / 8 * 8;               // a CTA's rows lie alike
  kernel<<<(unsigned)ctas, threads, (size_t)ring.S * (p.residual ? 2 : 1) * ring.pitch, st>>>(p, ring);
  return EMU_OK;
}

// A row's step has a fixed part for each warp (reduction, barrier, scale), so rows take few threads of
// many vectors: 8192 x 5760 bf16 in 52.7 us with four vectors a thread, 54.5 with two.  (Few rows would be
// done a little sooner by more threads, 64 x 5760 in 3.6 us with two vectors, 4.0 with four; but the
// split goes by the row's length alone, so that a row's codes do not depend on the rows beside it.)
template <class T> int pick_norm(const NormParams& p, bool alike, bool aligned16, bool q_vec, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int nv = (p.H + V - 1) / V;
  const Split sp = split_of<T>(p.H);
  // Short rows: a warp a row, straight from memory, by vectors or by elements; a ring's barriers and copies
  // would cost more than such a row.  So, and by the ring, bf16 with a residual: 100000 x 64 32 us and 62,
  // 100000 x 512 61 and 78, 50000 x 768 47 and 59, but 50000 x 1024 63 and 61; 100000 x 91 28 and 90,
  // 100000 x 255 50 and 108 (the ring's when it added unaligned rows by address, which was faster than now).
  if (aligned16 && nv <= 96) {
    if (nv <= 32) launch_norm<T, true, 32, 1>(p, st);
    else if (nv <= 64) launch_norm<T, true, 32, 2>(p, st);
    else launch_norm<T, true, 32, 3>(p, st);                // split_of: 64 threads of two blocks; see sq above
    return EMU_OK;
  }
  if (!aligned16 && p.H <= 256) {
    if (p.H <= 128) launch_norm<T, false, 32, 1, 4>(p, st);
    else launch_norm<T, false, 32, (V < 8 ? 2 : 1)>(p, st);
    return EMU_OK;
  }
  // By columns' blocks instead of by address, unaligned rows take longer: 8192 x 1111 bf16 24 us and 22,
  // 8192 x 3001 44 and 36, 8192 x 5761 84 and 66 (aligned 5760 53).
  if (alike && sp.it > 0) {
    if (nv <= 256) return launch_norm_ring<T, 2, 128, 8, 6>(p, sp.threads, aligned16, q_vec, st);
    if (nv <= 1024) return launch_norm_ring<T, 4, 256, 2, 2>(p, sp.threads, aligned16, q_vec, st);
    return launch_norm_ring<T, 4, 512, 1, 1>(p, sp.threads, aligned16, q_vec, st);
  }
  if (sp.it > 0) launch_norm<T, false, 512, 4>(p, st);
  else if (aligned16) launch_norm<T, true, 512, 0>(p, st);
  else launch_norm<T, false, 512, 0>(p, st);
  return EMU_OK;
}

// ------------------------------------------------------------------------- gradient
// The parts of column sums that there can be: one of every two CTAs, of up to 608 CTAs.  (With four times as
// many, where rows are short and more CTAs would live on an SM, joining them took longer than they
// saved.)  A multiple of four, as CTAs come by eights.
int64_t parts_for(int64_t T) {
  const int64_t n = (T + 7) / 8 * 4;
  return n < 304 ? n : 304;
}

struct NormGradParams {
  const void* gy; int64_t ldy;
  const void* h; int64_t ldh;
  const void* gh; int64_t ldg;                    // null: none
  const void* weight; bool weight_f32;
  const float* rstd;
  int64_t T; int H;
  void* gx;                                       // [T, H] contiguous
  float* part;                                    // [gridDim.x, H]
  uint32_t row_ctas;                              // CTAs that take rows; those after them take columns (few rows)
  float* gw;                                      // of the latter
};

// Few rows: gw needs nothing that the rows' pass finds, so CTAs of the same launch sum the columns, from the
// inputs (the second reading of few rows costs less than parts in memory and a kernel that joins them).  A CTA
// takes 8 vectors of columns, a lane one of them of every 4th of the warps' rows, or, where rows are not
// aligned, every 32nd column of the warp's rows.  red: a warp's sums of all the CTA's columns.
template <class T> constexpr int kColumns = 128 / sizeof(T);
template <class T, bool EDGES>
__device__ __forceinline__ void sum_columns(const NormGradParams& p, int block, float* red) {
  constexpr int VEC = 16 / sizeof(T), COLS = kColumns<T>, N = EDGES ? COLS / 32 : VEC, U = EDGES ? 8 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t c0 = (int64_t)block * COLS;
  const int64_t first = c0 + (EDGES ? lane : (lane & 7) * VEC);       // this lane's columns: VEC together, or 32 apart
  const int row0 = EDGES ? warp : warp * 4 + (lane >> 3), step = EDGES ? warps : 4 * warps, rows = (int)p.T;
  const T *gy = static_cast<const T*>(p.gy) + first, *h = static_cast<const T*>(p.h) + first;
  float acc[N], odd[N];                                               // of many rows two sums: shorter chains
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = odd[j] = 0.0f;
  for (int r0 = row0; r0 < rows; r0 += U * step) {                    // U rows asked for at once
    alignas(16) T y[U][N], x[U][N];
    float rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = r0 + u * step;
      const bool in = r < rows;
      rstd[u] = in ? p.rstd[r] : 0.0f;
      if constexpr (EDGES) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const bool at = in && first + 32 * j < p.H;
          y[u][j] = at ? gy[r * p.ldy + 32 * j] : from_f<T>(0.0f);
          x[u][j] = at ? h[r * p.ldh + 32 * j] : from_f<T>(0.0f);
        }
      } else {
        const bool at = in && first < p.H;
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(y[u]) = at ? *reinterpret_cast<const uint4*>(gy + r * p.ldy) : none;
        *reinterpret_cast<uint4*>(x[u]) = at ? *reinterpret_cast<const uint4*>(h + r * p.ldh) : none;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float& sum = EDGES && u % 2 ? odd[j] : acc[j];
        sum = fmaf(to_f(y[u][j]) * rstd[u], to_f(x[u][j]), sum);
      }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (EDGES) acc[j] += odd[j];
    if (!EDGES) {
      acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], 8);
      acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], 16);
    }
    if (EDGES || lane < 8) red[warp * COLS + (EDGES ? lane + 32 * j : lane * VEC + j)] = acc[j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < COLS && c0 + c < p.H; c += blockDim.x) {
    float a = 0.0f;
    for (int i = 0; i < warps; ++i) a += red[i * COLS + c];
    p.gw[c0 + c] = a;
  }
}

// The gradient in one pass.  As in the forward kernel, a CTA takes rows a grid apart through a ring in
// shared memory.  A row's sum of g h (g = gy w) has to be known before its first output, so each
// row is looked at twice, both times in shared memory.  A thread keeps the weights and the sums of
// gy h rstd of its IT vectors of columns in registers over all its rows; at the end the two CTAs
// of a cluster add theirs up through distributed shared memory, so that half as many parts of H
// sums go through memory to the joining kernel (clusters of eight did not all fit on the SMs at
// once: 95 us for 8192 x 5760).  Bound by HBM: four tensors of T H values.
constexpr int kGradCluster = 2;
template <class T, int IT, int MAXT, int MINB, bool EDGES>
__global__ void __launch_bounds__(MAXT, MINB)
norm_grad_kernel(const NormGradParams p, const Ring ring) {
  constexpr int VEC = 16 / sizeof(T), NP = VEC / 2;
  extern __shared__ __align__(16) unsigned char dyn[];      // the ring; then the column sums, [H] fp32
  __shared__ __align__(16) float sums[2][16];
  __shared__ __align__(8) uint64_t full[kStages];
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, warp = t >> 5;
  const int inputs = p.gh ? 3 : 2;
  const uint32_t stage_bytes = (uint32_t)inputs * ring.pitch;
  const int ctas = (int)p.row_ctas;
  const int rows = (int)(p.T > blockIdx.x ? (p.T - blockIdx.x + ctas - 1) / ctas : 0);
  const int apart = nt > 64 ? 32 : 1;                       // threads 0, 1, 2 of these fetch a tensor each
  const bool fetches = t % apart == 0 && t / apart < inputs;
  auto fill = [&](int i, int s) {
    const int64_t row = blockIdx.x + (int64_t)i * ctas;
    const int which = t / apart;
    const T* base = static_cast<const T*>(which == 0 ? p.gy : which == 1 ? p.h : p.gh);
    fill_row(dyn + s * stage_bytes + which * ring.pitch, base, which == 0 ? p.ldy : which == 1 ? p.ldh : p.ldg, row, p.T,
             p.H, smem_addr(&full[s]));
  };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel waits for this one's end
  if (p.gw && blockIdx.x >= p.row_ctas) {                   // whole clusters
    sum_columns<T, EDGES>(p, (int)(blockIdx.x - p.row_ctas), reinterpret_cast<float*>(dyn));
    return;
  }
  if (t < 16) sums[0][t] = sums[1][t] = 0.0f;
  if (t == 0) {
    for (int i = 0; i < ring.S; ++i) bar_init(smem_addr(&full[i]), inputs);
    bar_init_fence();
  }
  __syncthreads();
  if (fetches)
    for (int i = 0; i < ring.S && i < rows; ++i) fill(i, i);
  const int off = offset_of<T>(p.gy, p.ldy, blockIdx.x);
  f2 w[IT][NP], dw[IT][NP];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    weight_pairs(p, Columns<T, EDGES>(i * nt + t, off, p.H), w[i]);
#pragma unroll
    for (int j = 0; j < NP; ++j) dw[i][j] = 0ull;
  }
  const float inv_h = __fdiv_rn(1.0f, (float)p.H);
  bool ok = true;
  int s = 0, before = ring.S - 1;                           // row k's stage and row k - 1's
  uint32_t phase = 0;
  for (int k = 0; k < rows; ++k) {
    const int64_t row = blockIdx.x + (int64_t)k * ctas;
    const float rstd = p.rstd[row];
    ok = bar_wait(smem_addr(&full[s]), phase);
    const unsigned char* in = dyn + s * stage_bytes;
    f2 sum2 = 0ull;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Columns<T, EDGES> c(i * nt + t, off, p.H);
      if (!c.any()) continue;
      f2 y[NP], x[NP];
      read_pairs(in + (i * nt + t) * 16, c, y);
      read_pairs(in + ring.pitch + (i * nt + t) * 16, c, x);
#pragma unroll
      for (int j = 0; j < NP; ++j) sum2 = fma2(mul2(y[j], w[i][j]), x[j], sum2);
    }
    float s0, s1;
    halves(sum2, s0, s1);
    const float part = warp_sum(s0 + s1);
    if (lane == 0) sums[k & 1][warp] = part;                // the other half is the row before's
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    if (fetches && k >= 1 && k - 1 + ring.S < rows) fill(k - 1 + ring.S, before);   // all are past the row before
    before = s;
    if (++s == ring.S) {
      s = 0;
      phase ^= 1u;
    }
    // gx = (gy rstd) w + (gh - x coef), coef = rstd^3 mean(g h)
    const float coef = sum16(sums[k & 1]) * inv_h * rstd * rstd * rstd;
    const f2 r2 = pair(rstd, rstd), k2 = pair(-coef, -coef);
    T* gx = static_cast<T*>(p.gx) + row * p.H;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const Columns<T, EDGES> c(i * nt + t, off, p.H);
      if (!c.any()) continue;
      f2 y[NP], x[NP], g[NP];
      read_pairs(in + (i * nt + t) * 16, c, y);
      read_pairs(in + ring.pitch + (i * nt + t) * 16, c, x);
      if (inputs == 3) {
        read_pairs(in + 2 * ring.pitch + (i * nt + t) * 16, c, g);
      } else {
#pragma unroll
        for (int j = 0; j < NP; ++j) g[j] = 0ull;
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const f2 yr = mul2(y[j], r2);
        dw[i][j] = fma2(yr, x[j], dw[i][j]);
        g[j] = fma2(yr, w[i][j], fma2(x[j], k2, g[j]));
      }
      write_pairs(gx, c, g);
    }
  }
  if (!ok && t == 0) {                                      // a copy that never came: wait for the others, then end
    atomicExch(&g_norm_status, 1);
    for (int i = 0; i < ring.S; ++i) {
      (void)bar_wait(smem_addr(&full[i]), 0);
      (void)bar_wait(smem_addr(&full[i]), 1);
    }
  }
  if (p.gw) return;                                         // its columns are summed by others
  __syncthreads();
  float* const column_sums = reinterpret_cast<float*>(dyn);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const Columns<T, EDGES> c(i * nt + t, off, p.H);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float a, b;
      halves(dw[i][j], a, b);
      if (2 * j >= c.lo && 2 * j < c.hi) column_sums[c.first + 2 * j] = a;
      if (2 * j + 1 >= c.lo && 2 * j + 1 < c.hi) column_sums[c.first + 2 * j + 1] = b;
    }
  }
  cluster_sync();
  const int rank = blockIdx.x % kGradCluster;
  for (int col = rank * nt + t; col < p.H; col += kGradCluster * nt) {
    float v[kGradCluster];
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r)
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(in_cluster(column_sums + col, r)) : "memory");
    float a = v[0];
#pragma unroll
    for (int r = 1; r < kGradCluster; ++r) a += v[r];
    p.part[(int64_t)(blockIdx.x / kGradCluster) * p.H + col] = a;
  }
  cluster_sync();
}

// Short rows: a warp a row, as above but straight from memory, by vectors or, where rows are not aligned, by
// elements, the next row's values asked for before this one's are used, and with the sums of a CTA's warps
// for one part.  By the ring a row's copies, barriers and waits cost more than its values; so, and by the
// ring, bf16: 8192 x 512 10.3 us and 20.3, 100000 x 512 67 (6.1 TB/s) and 161, 100000 x 64 37 and 135, not
// aligned 100000 x 255 47 and 232, 1169 x 91 4.7 and 8.2.
constexpr int kShortWarps = 8;
template <class T, int VEC, int IT>
__global__ void __launch_bounds__(32 * kShortWarps, 2)
norm_grad_short_kernel(const NormGradParams p) {
  constexpr int COLS = 32 * VEC * IT;
  constexpr bool EDGES = VEC == 1;
  __shared__ __align__(16) float red[kShortWarps * (COLS > kColumns<T> ? COLS : kColumns<T>)];
  if (p.gw && blockIdx.x >= p.row_ctas) {
    sum_columns<T, EDGES>(p, (int)(blockIdx.x - p.row_ctas), red);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float w[IT][VEC], dw[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (i * 32 + lane) * VEC + j;
      w[i][j] = c >= p.H ? 0.0f : p.weight_f32 ? static_cast<const float*>(p.weight)[c] : to_f(static_cast<const T*>(p.weight)[c]);
      dw[i][j] = 0.0f;
    }
  const float inv_h = __fdiv_rn(1.0f, (float)p.H);
  const int64_t step = (int64_t)p.row_ctas * kShortWarps;
  using Raw = std::conditional_t<(VEC > 1), uint4, T>;     // a vector as words, not as elements a register each
  Raw raw[3][IT];
  float rstd = 0.0f;
  auto load = [&](int64_t row) {
    const bool in = row < p.T;
    rstd = in ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * 32 + lane) * VEC;
      if (!in || c >= p.H) continue;
      raw[0][i] = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.gy) + row * p.ldy + c);
      raw[1][i] = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.h) + row * p.ldh + c);
      if (p.gh) raw[2][i] = *reinterpret_cast<const Raw*>(static_cast<const T*>(p.gh) + row * p.ldg + c);
    }
  };
#pragma unroll
  for (int i = 0; i < IT; ++i) raw[0][i] = raw[1][i] = raw[2][i] = Raw{};   // what no load writes counts as zeros
  int64_t row = (int64_t)blockIdx.x * kShortWarps + warp;
  load(row);
  for (; row < p.T; row += step) {
    float y[IT][VEC], x[IT][VEC], g[IT][VEC], sum = 0.0f;
    const float r = rstd;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      load_f<T, VEC>(reinterpret_cast<const T*>(&raw[0][i]), y[i]);
      load_f<T, VEC>(reinterpret_cast<const T*>(&raw[1][i]), x[i]);
      load_f<T, VEC>(reinterpret_cast<const T*>(&raw[2][i]), g[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum = fmaf(y[i][j] * w[i][j], x[i][j], sum);
    }
    load(row + step);
    const float coef = warp_sum(sum) * inv_h * r * r * r;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * 32 + lane) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float yr = y[i][j] * r;
        dw[i][j] = fmaf(yr, x[i][j], dw[i][j]);
        g[i][j] = fmaf(yr, w[i][j], fmaf(x[i][j], -coef, g[i][j]));
      }
      if (c < p.H) store_f<T, VEC>(static_cast<T*>(p.gx) + row * p.H + c, g[i]);
    }
  }
  if (p.gw) return;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[warp * COLS + (i * 32 + lane) * VEC + j] = dw[i][j];
  __syncthreads();
  for (int c = threadIdx.x; c < p.H; c += 32 * kShortWarps) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kShortWarps; ++i) a += red[i * COLS + c];
    p.part[(int64_t)blockIdx.x * p.H + c] = a;
  }
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
// gw[c] = sum of the parts: 32 columns a CTA, sixteen threads a column.  Launched while the kernel before
// it still runs (its parts are waited for here).
__global__ void __launch_bounds__(512)
norm_grad_join_kernel(const float* part, int parts, int H, float* gw) {
  __shared__ float sm[16][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < H) {
    int b = g;
    for (; b + 48 < parts; b += 64)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += part[(int64_t)(b + 16 * i) * H + c];
    for (; b < parts; b += 16) acc[0] += part[(int64_t)b * H + c];
  }
  sm[g][lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  __syncthreads();
  if (g == 0 && c < H) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a += sm[i][lane];
    gw[c] = a;
  }
}

// Launches the kernel; the parts that it leaves for the joining kernel: none (0) where it sums the columns
// itself, and -1 if it failed.
template <class T, int IT, int MAXT, int MINB>
int launch_grad(const NormGradParams& given, int threads, bool aligned16, cudaStream_t st) {
  NormGradParams p = given;
  auto kernel = aligned16 ? norm_grad_kernel<T, IT, MAXT, MINB, false> : norm_grad_kernel<T, IT, MAXT, MINB, true>;
  static std::atomic<bool> flags[2][64];
  std::atomic<bool>* done = flags[aligned16];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(kernel), kMaxSmem - 1024, done)) return -1;
  int resident;
  const int inputs = p.gh ? 3 : 2;
  const Ring ring = ring_for(p.H, sizeof(T), aligned16, inputs, MAXT * MINB / threads, &resident);
  const int64_t most = (int64_t)emu_ops_sm_count() * resident;
  int64_t ctas = ((p.T < most ? p.T : most) + 7) / 8 * 8;  // whole clusters, and a CTA's rows lie alike
  if (ctas > parts_for(p.T) * kGradCluster) ctas = parts_for(p.T) * kGradCluster;
  size_t bytes = (size_t)ring.S * inputs * ring.pitch;      // two rows of two tensors at least: room for [H] fp32
  p.row_ctas = (uint32_t)ctas;
  // As few rows as a warp sums up soon, of tensors of 16 MiB at most.  So, and with parts and a joining kernel:
  // 1 x 1920 bf16 2.8 us and 5.6, 256 x 1920 3.8 and 6.9, 512 x 1920 6.0 and 7.9, 500 x 16384 20.7 and 23.7;
  // but 1000 x 16384 40.0 and 34.8; not aligned 128 x 1921 3.7 and 7.2, 200 x 2505 5.7 and 10.2, but 256 x
  // 953 (128 rows a warp) 8.5 and 7.9.
  const bool sums_columns = p.T <= (aligned16 ? 4 * 32 : 80) * (threads / 32) && p.T * p.H * (int64_t)sizeof(T) <= 16 << 20;
  if (sums_columns) {
    const size_t need = (size_t)(threads / 32) * 4 * kColumns<T>;
    bytes = bytes < need ? need : bytes;
    const int64_t blocks = (p.H + kColumns<T> - 1) / kColumns<T>;
    ctas += (blocks + kGradCluster - 1) / kGradCluster * kGradCluster;
  } else {
    p.gw = nullptr;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kGradCluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p, ring) != cudaSuccess) return -1;
  return sums_columns ? 0 : (int)(p.row_ctas / kGradCluster);
}

template <class T, int VEC, int IT> int launch_grad_short(const NormGradParams& given, cudaStream_t st) {
  NormGradParams p = given;
  const int64_t ctas = (p.T + kShortWarps - 1) / kShortWarps, most = parts_for(p.T);
  p.row_ctas = (uint32_t)(ctas < most ? ctas : most);
  // so, and with parts: 256 x 96 bf16 3.1 us and 3.6, 1000 x 96 7.3 and 4.3; not aligned 400 x 197 5.5 and 4.2
  const bool sums_columns = p.T <= (VEC > 1 ? 64 : 32) * kShortWarps;
  if (!sums_columns) p.gw = nullptr;
  const int64_t columns = sums_columns ? (p.H + kColumns<T> - 1) / kColumns<T> : 0;
  norm_grad_short_kernel<T, VEC, IT><<<(unsigned)(p.row_ctas + columns), 32 * kShortWarps, 0, st>>>(p);
  return sums_columns ? 0 : (int)p.row_ctas;
}

// The fewest vectors a thread that leave a CTA within its threads; as launch_grad.
template <class T> int pick_norm_grad(const NormGradParams& p, bool alike, bool aligned16, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const int nv = aligned16 ? p.H / V : (p.H + 2 * V - 2) / V;       // vectors that a row can touch
  if (aligned16 && nv <= 64) return nv <= 32 ? launch_grad_short<T, V, 1>(p, st) : launch_grad_short<T, V, 2>(p, st);
  if (!aligned16 && p.H <= 256) return p.H <= 128 ? launch_grad_short<T, 1, 4>(p, st) : launch_grad_short<T, 1, 8>(p, st);
  if (alike && nv <= 2048) {
    if (nv <= 256) return launch_grad<T, 2, 128, 6>(p, threads_for(nv, 2), aligned16, st);
    if (nv <= 1024) return launch_grad<T, 4, 256, 2>(p, threads_for(nv, 4), aligned16, st);
    return launch_grad<T, 4, 512, 1>(p, threads_for(nv, 4), aligned16, st);
  }
  const int parts = (int)parts_for(p.T);
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
  int rc = emu_ops_int8_status(&v, reset != 0);
  int b = 0;
  if (rc == EMU_OK) rc = emu_ops_block_status(&b, reset != 0);
  if (rc != EMU_OK) return rc;
  int n = 0;
  if (cudaMemcpyFromSymbol(&n, g_norm_status, sizeof n) != cudaSuccess) return emu_ops_launched("emu_ops_device_status");
  const int zero = 0;
  if (reset && cudaMemcpyToSymbol(g_norm_status, &zero, sizeof zero) != cudaSuccess)
    return emu_ops_launched("emu_ops_device_status");
  *status = v | b | n;
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
  const Span sx(x, T, ldx, H, es), sr(residual, T, ldr, H, es), so(residual_out, T, ldo, H, es);
  const Span sw(weight, 1, H, H, elem_bytes(weight_type)), ss(scale, 1, 1, 1, 4);
  // an output row may replace its input row, and may not meet any other
  if ((so.meets(sx) && !(residual_out == x && ldo == ldx)) || (so.meets(sr) && !(residual_out == residual && ldo == ldr)))
    return emu_ops_fail(EMU_EINVAL, "residual_out overlaps an input without being that input");
  if (!apart({so}, {sw, ss}) ||
      !apart({Span(q, T, H, H, 1), Span(rstd, 1, T, T, 4), Span(scale ? nullptr : scale_out, 1, T, T, 4)}, {sx, sr, so, sw, ss}))
    return emu_ops_fail(EMU_EINVAL, "an output overlaps an input or another output");
  NormParams p;
  p.x = x; p.ldx = ldx;
  p.residual = residual; p.ldr = ldr;
  p.weight = weight; p.weight_f32 = weight_type == EMU_OUT_F32;
  p.T = T; p.H = (int)H; p.eps = eps;
  p.qmax = q_format == EMU_Q_E4M3FN ? 448.0f : q_format == EMU_Q_E5M2 ? 57344.0f : 127.0f;
  p.scale = scale; p.q_format = (int)q_format;
  p.q = static_cast<uint8_t*>(q); p.scale_out = scale_out;
  p.residual_out = residual_out; p.ldo = ldo; p.rstd = rstd;
  // do all rows start on 16 bytes, or at least all tensors' alike
  auto at = [](const void* t) { return reinterpret_cast<uintptr_t>(t); };
  const uintptr_t starts = (at(x) ^ (residual ? at(residual) : at(x))) | (at(x) ^ (residual_out ? at(residual_out) : at(x)));
  const int64_t strides = (ldx - (residual ? ldr : ldx)) | (ldx - (residual_out ? ldo : ldx));
  const int64_t v = 16 / (int64_t)es;
  const bool alike = starts % 16 == 0 && strides % v == 0;
  const bool aligned16 = alike && aligned(x, 16) && ldx % v == 0 && H % v == 0 && aligned(weight, 16) && aligned(q, (size_t)v);
  const bool q_vec = at(q) % v == at(x) / es % v && (H - ldx) % v == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = type == EMU_OUT_F32    ? pick_norm<float>(p, alike, aligned16, q_vec, st)
       : type == EMU_OUT_BF16 ? pick_norm<__nv_bfloat16>(p, alike, aligned16, q_vec, st)
                              : pick_norm<__half>(p, alike, aligned16, q_vec, st);
  if (rc != EMU_OK) return rc;
  return emu_ops_launched("emu_rms_norm_quant");
}

size_t emu_rms_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T < 1 || H < 1 || H > (1 << 22)) return 0;
  return (size_t)parts_for(T) * (size_t)H * sizeof(float);
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
  const size_t need = emu_rms_norm_backward_workspace_bytes(T, H);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return emu_ops_fail(EMU_EINVAL, "workspace of %zu bytes needed, 16-byte aligned (got %zu)", need, workspace_bytes);
  if (!apart({Span(grad_x, T, H, H, es), Span(grad_weight, 1, H, H, 4), Span(workspace, 1, 1, 1, need)},
             {Span(grad_y, T, ldy, H, es), Span(hidden, T, ldh, H, es), Span(grad_residual, T, ldg, H, es),
              Span(rstd, 1, T, T, 4), Span(weight, 1, H, H, elem_bytes(weight_type))}))
    return emu_ops_fail(EMU_EINVAL, "an output or the workspace overlaps an input, or another of them");
  NormGradParams p;
  p.gy = grad_y; p.ldy = ldy; p.h = hidden; p.ldh = ldh; p.gh = grad_residual; p.ldg = ldg;
  p.weight = weight; p.weight_f32 = weight_type == EMU_OUT_F32; p.rstd = rstd;
  p.T = T; p.H = (int)H; p.gx = grad_x; p.part = static_cast<float*>(workspace);
  p.row_ctas = 0; p.gw = grad_weight;
  // do all rows start on 16 bytes, or at least all tensors' alike
  auto at = [](const void* t) { return reinterpret_cast<uintptr_t>(t); };
  const uintptr_t bases = (at(grad_y) ^ at(hidden)) | (at(grad_y) ^ at(grad_x)) |
                          (at(grad_y) ^ (grad_residual ? at(grad_residual) : at(grad_y)));
  const int64_t strides = (ldy - ldh) | (ldy - H) | (ldy - (grad_residual ? ldg : ldy));
  const int64_t v = 16 / (int64_t)es;
  const bool alike = bases % 16 == 0 && strides % v == 0;
  const bool aligned16 = alike && aligned(grad_y, 16) && ldy % v == 0 && H % v == 0;
  const int parts = type == EMU_OUT_F32    ? pick_norm_grad<float>(p, alike, aligned16, st)
                    : type == EMU_OUT_BF16 ? pick_norm_grad<__nv_bfloat16>(p, alike, aligned16, st)
                                           : pick_norm_grad<__half>(p, alike, aligned16, st);
  if (parts <= 0) return emu_ops_launched("emu_rms_norm_backward");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((H + 31) / 32));
  cfg.blockDim = dim3(512);
  cfg.stream = st;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const float* sums = p.part;
  if (cudaLaunchKernelEx(&cfg, norm_grad_join_kernel, sums, parts, p.H, grad_weight) != cudaSuccess)
    return emu_ops_launched("emu_rms_norm_backward");
  return emu_ops_launched("emu_rms_norm_backward");
}

}  // extern "C"
