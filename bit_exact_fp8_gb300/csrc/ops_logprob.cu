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

// Running (m, z, u) of a part of a row: z and u are relative to m, the largest logit so far or,
// before any, the lowest finite number (so that x - m is never -inf - -inf).  z == 0: nothing
// above -inf yet.  NaN and +inf end in z = NaN, which every later step keeps.
struct Soft {
  float m, z, u;
};
constexpr float kLowest = -3.40282347e38f;
__device__ __forceinline__ Soft soft_join(const Soft& a, const Soft& b) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf(a.m - m, -1e4f), db = fmaxf(b.m - m, -1e4f);    // e^-1e4 is 0
  const float fa = exp2_approx(da * kLog2e), fb = exp2_approx(db * kLog2e);
  return Soft{m, a.z * fa + b.z * fb, (a.u + a.z * da) * fa + (b.u + b.z * db) * fb};
}
__device__ __forceinline__ Soft soft_warp(Soft a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = soft_join(a, Soft{__shfl_xor_sync(0xFFFFFFFFu, a.m, o), __shfl_xor_sync(0xFFFFFFFFu, a.z, o),
                          __shfl_xor_sync(0xFFFFFFFFu, a.u, o)});
  return a;
}

// A row as 16-byte vectors at 16-byte addresses: vector v holds the logits v * VEC - off + j, those
// outside [0, V) read as -inf.
template <class T> struct Row {
  static constexpr int VEC = 16 / sizeof(T);
  const T* base;           // the row's start, rounded down to 16 bytes
  int off, V, nvec;
  __device__ __forceinline__ Row(const T* x, int V_) : V(V_) {
    off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
    base = x - off;
    nvec = (V + off + VEC - 1) / VEC;
  }
  __device__ __forceinline__ int first(int v) const { return v * VEC - off; }
  __device__ __forceinline__ bool whole(int v) const { return first(v) >= 0 && first(v) + VEC <= V; }
  __device__ __forceinline__ uint4 load_raw(int v) const {
    if (whole(v)) return *reinterpret_cast<const uint4*>(base + (int64_t)v * VEC);
    Pack<T, VEC> q;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int i = first(v) + j;
      q.v[j] = i >= 0 && i < V ? base[off + i] : from_f<T>(-INFINITY);
    }
    return *reinterpret_cast<const uint4*>(&q);
  }
  __device__ __forceinline__ void load(int v, float (&f)[VEC]) const { unpack(load_raw(v), f); }
  static __device__ __forceinline__ void unpack(const uint4& raw, float (&f)[VEC]) {
    const Pack<T, VEC> q = *reinterpret_cast<const Pack<T, VEC>*>(&raw);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = to_f(q.v[j]);
  }
};

// (key, position) of a logit as one number: the larger key first, then the lower position
__device__ __forceinline__ unsigned long long ranked(uint32_t key, uint32_t pos) {
  return ((unsigned long long)key << 32) | (0xFFFFFFFFu - pos);
}

// The largest and the smallest of N vectors' logits (NaN left out), two at a time in 16-bit types.
template <int N> __device__ __forceinline__ void extremes(const uint4 (&raw)[N], float& hi, float& lo, float) {
  hi = -INFINITY;
  lo = INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[4];
    Row<float>::unpack(raw[i], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi = fmaxf(hi, f[j]);
      lo = fminf(lo, f[j]);
    }
  }
}
template <class P, int N> __device__ __forceinline__ void extremes2(const uint4 (&raw)[N], P& h, P& l) {
  h = l = *reinterpret_cast<const P*>(&raw[0].x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const P* q = reinterpret_cast<const P*>(&raw[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h = __hmax2(h, q[j]);
      l = __hmin2(l, q[j]);
    }
  }
}
template <int N> __device__ __forceinline__ void extremes(const uint4 (&raw)[N], float& hi, float& lo, __nv_bfloat16) {
  __nv_bfloat162 h, l;
  extremes2(raw, h, l);
  hi = fmaxf(__bfloat162float(h.x), __bfloat162float(h.y));
  lo = fminf(__bfloat162float(l.x), __bfloat162float(l.y));
}
template <int N> __device__ __forceinline__ void extremes(const uint4 (&raw)[N], float& hi, float& lo, __half) {
  __half2 h, l;
  extremes2(raw, h, l);
  hi = fmaxf(__half2float(h.x), __half2float(h.y));
  lo = fminf(__half2float(l.x), __half2float(l.y));
}

// Logits below about -65504 moved up to there (NaN kept): next to one of -6e4 or more their weight is 0
// as it was, and x - m is finite.
__device__ __forceinline__ void floor_at(uint4& raw, float) {
  float* f = reinterpret_cast<float*>(&raw);
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = max_nan(f[j], -65536.0f);
}
template <class P> __device__ __forceinline__ void floor2(uint4& raw, P low) {
  P* q = reinterpret_cast<P*>(&raw);
#pragma unroll
  for (int j = 0; j < 4; ++j) q[j] = __hmax2_nan(q[j], low);
}
__device__ __forceinline__ void floor_at(uint4& raw, __nv_bfloat16) { floor2(raw, __float2bfloat162_rn(-65536.0f)); }
__device__ __forceinline__ void floor_at(uint4& raw, __half) { floor2(raw, __float2half2_rn(-65504.0f)); }

// A thread's part of a row.  Vectors whose largest logit is within -6e4 and 1e6 take the fast form:
// with L = log2 e and c = fp32(m L), a = x L - c is one rounding, e = 2^a, and the sums of e and
// e a run in fp32 pairs, about five instructions a logit.  (c differs from m L by a rounding that
// is the same for every logit, below 0.1; it is taken out at the end as d = c - m L.)  The others
// (masked whole, or out of range) go by x - m one by one.
template <class T> struct Streamed {
  static constexpr int VEC = Row<T>::VEC;
  float m = kLowest, c = kLowest;      // of the fast form
  f2 z = 0ull, w = 0ull;               // sums of e, of e a
  Soft slow{kLowest, 0.0f, 0.0f};
  float top = -INFINITY;               // the largest logit and the vector where it first stands
  int at;

  template <int N> __device__ __forceinline__ void take(uint4 (&raw)[N], int v, int step) {
    float hi, lo;
    extremes(raw, hi, lo, T());
    if (hi > top) {
      top = hi;
#pragma unroll
      for (int i = N - 1; i >= 0; --i) {
        const uint4 one[1] = {raw[i]};
        float h, l;
        extremes(one, h, l, T());
        if (h == hi) at = v + i * step;
      }
    }
    if (hi >= -6e4f && hi <= 1e6f) {
      if (!(lo >= -65504.0f)) {
#pragma unroll
        for (int i = 0; i < N; ++i) floor_at(raw[i], T());
      }
      if (hi > m) {
        const float cn = hi * kLog2e, d = fmaxf(c - cn, -1e4f), e = exp2_approx(d);
        const f2 e2 = pair(e, e);
        w = mul2(fma2(pair(d, d), z, w), e2);
        z = mul2(z, e2);
        m = hi;
        c = cn;
      }
      const f2 L2 = pair(kLog2e, kLog2e), c2 = pair(-c, -c);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[VEC];
        Row<T>::unpack(raw[i], f);
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const f2 a = fma2(pair(f[j], f[j + 1]), L2, c2);
          float a0, a1;
          halves(a, a0, a1);
          const f2 e = pair(exp2_approx(a0), exp2_approx(a1));
          z = add2(z, e);
          w = fma2(e, a, w);
        }
      }
      return;
    }
    if (hi > slow.m) {
      const float d = fmaxf(slow.m - hi, -1e4f), e = exp2_approx(d * kLog2e);
      slow.u = (slow.u + slow.z * d) * e;
      slow.z *= e;
      slow.m = hi;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[VEC];
      Row<T>::unpack(raw[i], f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t = f[j] - slow.m, e = exp2_approx(t * kLog2e);
        slow.z += e;
        slow.u = fmaf(e, fmaxf(t, -1e4f), slow.u);
      }
    }
  }
  __device__ __forceinline__ Soft sums() const {
    float z0, z1, w0, w1;
    halves(z, z0, z1);
    halves(w, w0, w1);
    const float d = m > kLowest ? fmaf(-m, kLog2e, c) : 0.0f, e = exp2_approx(d);
    const float zz = z0 + z1;
    return soft_join(Soft{m, zz * e, (w0 + w1 + d * zz) * e * 0.693147181f}, slow);
  }
};

// the vectors v0, v0 + step, ... below v1, LOADS of them asked for at a time
template <int LOADS, class T>
__device__ __forceinline__ Streamed<T> stream(const Row<T>& row, int v0, int v1, int step) {
  constexpr int U = 4;
  Streamed<T> s;
  s.at = v0;
  int v = v0;
  if (LOADS == 2 * U) {
    for (; v + (2 * U - 1) * step < v1; v += step * 2 * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int i = 0; i < U; ++i) a[i] = row.load_raw(v + i * step);
#pragma unroll
      for (int i = 0; i < U; ++i) b[i] = row.load_raw(v + (U + i) * step);
      s.take(a, v, step);
      s.take(b, v + U * step, step);
    }
  }
  for (; v + (U - 1) * step < v1; v += step * U) {
    uint4 raw[U];
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = row.load_raw(v + i * step);
    s.take(raw, v, step);
  }
  for (; v < v1; v += step) {
    uint4 raw[1] = {row.load_raw(v)};
    s.take(raw, v, step);
  }
  return s;
}

// the given token's logit, asked for before the row's pass; NaN outside [0, V)
template <class T> __device__ __forceinline__ float token_logit(const LogprobParams& p, int64_t row, bool& ignored) {
  const int64_t tok = p.tokens[row];
  ignored = tok == p.ignore;
  return tok < 0 || tok >= p.V ? NAN : to_f((static_cast<const T*>(p.x) + row * p.ldx)[tok]);
}
// the row's outputs but its alternatives; x - m is exact where it matters, so logprob is (x - m) - log z
__device__ __forceinline__ void finish_row(const LogprobParams& p, int64_t row, const Soft& s, float logit, bool ignored) {
  const bool empty = s.z == 0.0f;
  const float logz = logf(s.z);
  const float entropy = empty ? 0.0f : logz - s.u / s.z;
  p.logprob[row] = ignored ? 0.0f : empty && logit == logit ? -INFINITY : logit - s.m - logz;
  p.entropy[row] = entropy;
  p.lse[row] = empty ? -INFINITY : s.m + logz;
  float* st = p.stats + row * 3;
  st[0] = empty ? -INFINITY : s.m;
  st[1] = logz;
  st[2] = entropy;
}
// alternative `rank` of the row: logit of this key at this id
__device__ __forceinline__ void put_top(const LogprobParams& p, int64_t row, int rank, unsigned long long c, const Soft& s) {
  p.top_val[row * p.k + rank] = s.z == 0.0f ? -INFINITY : key_value((uint32_t)(c >> 32)) - s.m - logf(s.z);
  p.top_id[row * p.k + rank] = (int64_t)(0xFFFFFFFFu - (uint32_t)c);
}
// The alternatives of a row that holds NaN or +inf, whose z is NaN.  They are written without ranking: NaN
// has no place in the order of keys, and a vector of nothing else has no largest logit to be listed by.
__device__ __forceinline__ bool is_bad(const Soft& s) { return s.z != s.z; }
__device__ __forceinline__ void put_bad(const LogprobParams& p, int64_t row, int rank) {
  p.top_val[row * p.k + rank] = NAN;
  p.top_id[row * p.k + rank] = -1;
}

// The top k of a row in one more look at a few of its logits.  The pass above leaves each group of
// threads with its largest logit, its head.  The k-th largest head bounds the k-th largest logit
// from below (at least k logits reach it), so only the k groups with the largest heads hold
// logits to be taken, and of theirs only those from that bound on: for most rows little more
// than k.  They are listed, and each counts those above itself.  Heads and bound are compared
// with their vectors' positions, so equal logits come out by lower id and a row of equal ones
// lists few.  A list too short (many large logits at one period) is made up for by k searches.
//
// The logits of one vector that reach the bound, onto the list.
template <class T>
__device__ __forceinline__ void collect_vector(const Row<T>& row, int v, const uint4& raw, float least,
                                               unsigned long long bound, unsigned long long* list, int room, int* count) {
  constexpr int VEC = Row<T>::VEC;
  float hi, lo;
  const uint4 one[1] = {raw};
  extremes(one, hi, lo, T());
  if (!(hi >= least)) return;
  float f[VEC];
  Row<T>::unpack(raw, f);
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int id = row.first(v) + j;
    const uint32_t key = order_key(f[j]);
    if (id >= 0 && id < row.V && ranked(key, (uint32_t)v) >= bound) {
      const int n = atomicAdd(count, 1);
      if (n < room) list[n] = ranked(key, (uint32_t)id);
    }
  }
}
__device__ __forceinline__ float least_of(unsigned long long bound) {
  return bound ? key_value((uint32_t)(bound >> 32)) : -INFINITY;
}

// One warp a row: for short rows.
constexpr int kWarpRows = 4, kWarpList = 512;
template <class T>
__global__ void __launch_bounds__(32 * kWarpRows)
logprob_warp_kernel(const LogprobParams p) {
  __shared__ __align__(16) unsigned long long list_all[kWarpRows][kWarpList + 2];
  __shared__ int cand_all[kWarpRows][kMaxTop];
  __shared__ int count_all[kWarpRows];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t r = (int64_t)blockIdx.x * kWarpRows + w;
  if (r >= p.T) return;
  const Row<T> row(static_cast<const T*>(p.x) + r * p.ldx, p.V);
  bool ignored = false;
  const float logit = lane == 0 ? token_logit<T>(p, r, ignored) : 0.0f;
  const Streamed<T> mine = stream<4>(row, lane, row.nvec, 32);
  const Soft s = soft_warp(mine.sums());
  if (lane == 0) finish_row(p, r, s, logit, ignored);
  if (p.k == 0) return;
  if (is_bad(s)) {                                     // in every lane alike
    if (lane < p.k) put_bad(p, r, lane);
    return;
  }
  unsigned long long* list = list_all[w];
  int& count = count_all[w];
  if (lane == 0) count = 0;
  const unsigned long long head =
      lane < row.nvec ? ranked(order_key(mine.top), (uint32_t)mine.at) : 0ull;
  int above = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) above += __shfl_sync(0xFFFFFFFFu, head, i) > head;
  const uint32_t kth = __ballot_sync(0xFFFFFFFFu, head != 0ull && above == p.k - 1);
  const unsigned long long bound = kth ? __shfl_sync(0xFFFFFFFFu, head, __ffs(kth) - 1) : 0ull;
  if (head != 0ull && above < p.k) cand_all[w][above] = lane;
  const int taken = __popc(__ballot_sync(0xFFFFFFFFu, head != 0ull && above < p.k));
  __syncwarp();
  const float least = least_of(bound);
  const int len = (row.nvec + 31) / 32;                // a lane's vectors
  for (int q0 = lane; q0 < taken * len; q0 += 128) {   // those of the lanes taken, four at a time
    uint4 raw[4];
    int at[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = q0 + u * 32, c = q / len;
      at[u] = q < taken * len ? (q - c * len) * 32 + cand_all[w][c] : row.nvec;
      if (at[u] < row.nvec) raw[u] = row.load_raw(at[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at[u] < row.nvec) collect_vector(row, at[u], raw[u], least, bound, list, kWarpList, &count);
  }
  __syncwarp();
  const int n = count;
  if (n <= 32) {
    const unsigned long long mine = lane < n ? list[lane] : 0ull;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += list[j] > mine;
    if (lane < n && rank < p.k) put_top(p, r, rank, mine, s);
    return;
  }
  if (n <= kWarpList) {                                // four entries a lane against two at a time
    if (lane == 0 && n % 2) list[n] = 0ull;
    __syncwarp();
    for (int i0 = lane; i0 < n; i0 += 128) {
      unsigned long long mine[4];
      int rank[4] = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 4; ++u) mine[u] = i0 + 32 * u < n ? list[i0 + 32 * u] : ~0ull;
      for (int j = 0; j < n; j += 2) {
        const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(list + j);
#pragma unroll
        for (int u = 0; u < 4; ++u) rank[u] += (c.x > mine[u]) + (c.y > mine[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + 32 * u < n && rank[u] < p.k) put_top(p, r, rank[u], mine[u], s);
    }
    return;
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < p.k; ++i) {
    unsigned long long best = 0ull;
    for (int v = lane; v < p.V; v += 32) {
      const unsigned long long c = ranked(order_key(to_f(row.base[row.off + v])), (uint32_t)v);
      if (c < last && c > best) best = c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long c = __shfl_xor_sync(0xFFFFFFFFu, best, o);
      best = c > best ? c : best;
    }
    last = best;
    if (lane == 0) put_top(p, r, i, last, s);
  }
}

// A CTA, or the C CTAs of a cluster, a row: for long rows, and more CTAs a row the fewer rows there
// are.  Each CTA takes a run of the row's vectors; the first one joins the sums and the k
// largest of each through distributed shared memory.
constexpr int kGroups = 128, kMaxCluster = 8;
template <class T, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 5)
logprob_row_kernel(const LogprobParams p, int C) {
  constexpr int NW = NT / 32, GT = NT / kGroups;      // GT threads a group
  constexpr bool FEW = NT == 512;                      // the form for few rows
  constexpr int kList = FEW ? 1024 : 768;              // a row of equal logits lists 8 k GT
  __shared__ Soft warp_soft[NW];
  __shared__ __align__(16) unsigned long long heads[kGroups];
  __shared__ int cand[kMaxTop];
  __shared__ unsigned long long bound;
  __shared__ int count, taken;
  __shared__ unsigned long long list[kList];
  __shared__ unsigned long long kept[kMaxTop * (kList / kGroups)];       // of the list: k groups' at most
  __shared__ Soft parts[kMaxCluster];                                    // of the first CTA: all CTAs'
  __shared__ unsigned long long tops[kMaxCluster][kMaxTop];
  __shared__ unsigned long long best_of[NW];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int64_t r = blockIdx.x / C;
  const int part = blockIdx.x % C;
  const Row<T> row(static_cast<const T*>(p.x) + r * p.ldx, p.V);
  const int v0 = (int)((int64_t)row.nvec * part / C), v1 = (int)((int64_t)row.nvec * (part + 1) / C);
  // the last thread writes the row's own outputs, while the others rank its alternatives
  bool ignored = false;
  const float logit = tid == NT - 1 && part == 0 ? token_logit<T>(p, r, ignored) : 0.0f;
  const Streamed<T> mine = stream<FEW ? 8 : 4>(row, v0 + tid, v1, NT);
  const Soft ws = soft_warp(mine.sums());
  if (lane == 0) warp_soft[w] = ws;
  if (p.k > 0) {
    unsigned long long head =
        v0 + tid < v1 ? ranked(order_key(mine.top), (uint32_t)mine.at) : 0ull;
#pragma unroll
    for (int o = 1; o < GT; o <<= 1) {
      const unsigned long long c = __shfl_xor_sync(0xFFFFFFFFu, head, o);
      head = c > head ? c : head;
    }
    if (tid % GT == 0) heads[tid / GT] = head;
    if (tid == 0) {
      count = taken = 0;
      bound = 0ull;
    }
  }
  __syncthreads();
  Soft s = warp_soft[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) s = soft_join(s, warp_soft[i]);

  if (p.k > 0 && !is_bad(s)) {                         // in every thread alike; a bad part makes the row bad
    // how many heads exceed each group's, GT threads a head, each with its share of the others; the k-th is the bound
    auto rank_heads = [&](unsigned long long* at) {
      const unsigned long long head = heads[tid / GT];
      int above = 0;
#pragma unroll 16
      for (int i = 2 * (tid % GT); i < kGroups; i += 2 * GT) {
        const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(heads + i);
        above += (h.x > head) + (h.y > head);
      }
#pragma unroll
      for (int o = 1; o < GT; o <<= 1) above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
      if (tid % GT == 0 && head != 0ull && above == p.k - 1) *at = head;
      return tid % GT == 0 && head != 0ull && above < p.k ? above : -1;
    };
    const int place = rank_heads(&bound);
    if (place >= 0) {
      cand[place] = tid / GT;
      atomicAdd(&taken, 1);
    }
    __syncthreads();
    const float least = least_of(bound);
    // 32 vectors of a group taken at a time for each warp, four loads in flight: of one group, or (few rows,
    // whose parts have few vectors a group) of several
    constexpr int ROUND = 32 / GT * NT;
    if (FEW) {
      const int rounds = (v1 - v0 + ROUND - 1) / ROUND, all = taken * rounds;
      for (int q0 = w; q0 < all; q0 += 4 * NW) {
        uint4 raw[4];
        int v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int q = q0 + u * NW, c = q / rounds;
          v[u] = q < all ? v0 + (q - c * rounds) * ROUND + lane / GT * NT + cand[c] * GT + lane % GT : v1;
          if (v[u] < v1) raw[u] = row.load_raw(v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (v[u] < v1) collect_vector(row, v[u], raw[u], least, bound, list, kList, &count);
      }
    } else {
      for (int c = w; c < taken; c += NW) {
        for (int v = v0 + lane / GT * NT + cand[c] * GT + lane % GT; v < v1; v += 4 * ROUND) {
          uint4 raw[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (v + u * ROUND < v1) raw[u] = row.load_raw(v + u * ROUND);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (v + u * ROUND < v1) collect_vector(row, v + u * ROUND, raw[u], least, bound, list, kList, &count);
        }
      }
    }
    __syncthreads();
    const int n = count;
    const int id0 = max(row.first(v0), 0), id1 = min(row.first(v1), p.V);
    if (tid < kMaxTop) tops[part][tid] = 0ull;         // fewer logits than k in this run
    __syncthreads();
    if (n <= kList) {
      const unsigned long long* from = list;
      int m = n;
      if (n > kGroups) {                               // equal logits, above all: the same bound once more, for the listed
        unsigned long long head = 0ull;
        for (int i = tid; i < n; i += NT) head = list[i] > head ? list[i] : head;
#pragma unroll
        for (int o = 1; o < GT; o <<= 1) {
          const unsigned long long c = __shfl_xor_sync(0xFFFFFFFFu, head, o);
          head = c > head ? c : head;
        }
        if (tid % GT == 0) heads[tid / GT] = head;
        if (tid == 0) count = 0;
        __syncthreads();
        (void)rank_heads(&bound);
        __syncthreads();
        for (int i = tid; i < n; i += NT)
          if (list[i] >= bound) kept[atomicAdd(&count, 1)] = list[i];
        __syncthreads();
        from = kept;
        m = count;
      }
      for (int i = tid; i < m; i += NT) {
        const unsigned long long c = from[i];
        int rank = 0;
        for (int j = 0; j < m; ++j) rank += from[j] > c;
        if (rank < p.k) tops[part][rank] = c;
      }
      __syncthreads();
    } else {
      unsigned long long last = ~0ull;
      for (int i = 0; i < p.k; ++i) {
        unsigned long long best = 0ull;
        for (int id = id0 + tid; id < id1; id += NT) {
          const unsigned long long c = ranked(order_key(to_f(row.base[row.off + id])), (uint32_t)id);
          if (c < last && c > best) best = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long c = __shfl_xor_sync(0xFFFFFFFFu, best, o);
          best = c > best ? c : best;
        }
        if (lane == 0) best_of[w] = best;
        __syncthreads();
        last = best_of[0];
#pragma unroll
        for (int q = 1; q < NW; ++q) last = best_of[q] > last ? best_of[q] : last;
        __syncthreads();
        if (tid == 0) tops[part][i] = last;
      }
      __syncthreads();
    }
  }

  if (C > 1) {
    cluster_sync();                                    // every CTA of the cluster runs
    if (part > 0) {
      if (tid == 0) {
        const uint32_t a = in_cluster(&parts[part], 0);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(s.m) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(s.z) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(s.u) : "memory");
      }
      if (tid < p.k)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(in_cluster(&tops[part][tid], 0)), "l"(tops[part][tid])
                     : "memory");
    }
    cluster_sync();
    if (part > 0) return;
    for (int i = 1; i < C; ++i) s = soft_join(s, parts[i]);
  }
  if (tid == NT - 1) finish_row(p, r, s, logit, ignored);
  if (is_bad(s)) {
    if (tid < p.k) put_bad(p, r, tid);
    return;
  }
  for (int i = tid; i < C * kMaxTop; i += NT) {
    const int q = i / kMaxTop, j = i % kMaxTop;
    const unsigned long long c = j < p.k ? tops[q][j] : 0ull;
    if (c == 0ull) continue;
    int rank = j;                                      // within its own part; and those above it in the others
    for (int o = 0; o < C; ++o) {
      if (o == q) continue;
      int n = 0;                                       // the parts' lists fall: a search by halves
#pragma unroll
      for (int h = kMaxTop / 2; h > 0; h >>= 1)
        if (n + h <= p.k && tops[o][n + h - 1] > c) n += h;
      if (n < p.k && tops[o][n] > c) ++n;
      rank += n;
    }
    if (rank < p.k) put_top(p, r, rank, c, s);
  }
}

template <class T, int NT> int launch_row(const LogprobParams& p, int C, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  cfg.gridDim = dim3((unsigned)(p.T * C));               // C > 1 only for few rows
  if (cudaLaunchKernelEx(&cfg, logprob_row_kernel<T, NT>, p, C) != cudaSuccess) return emu_ops_launched("emu_token_logprobs");
  return EMU_OK;
}

template <class T> int pick_logprob(const LogprobParams& p, cudaStream_t st) {
  const int nvec = (int)(((int64_t)p.V + Row<T>::VEC - 1) / Row<T>::VEC);
  // A warp for short rows, and for many longer ones with few alternatives (with many, too much of a long row
  // reaches a bound that 32 lanes' maxima give): 6852 x 16658 fp16 with 5 alternatives 70 us by warps, 83 by
  // CTAs of 128 threads, but 300 rows 19 and 7.
  if (nvec <= 1024 || (nvec <= 2560 && p.k <= 8 && p.T >= 16 * emu_ops_sm_count())) {
    logprob_warp_kernel<T><<<(unsigned)((p.T + kWarpRows - 1) / kWarpRows), 32 * kWarpRows, 0, st>>>(p);
    return EMU_OK;
  }
  // Small CTAs for many rows of middling length: 6852 x 16658 fp16 with 32 alternatives 128 us, 139 by 256
  // threads; 2000 x 30000 bf16 with 5 38 and 42.
  if (nvec <= 4096 && p.T >= 2 * emu_ops_sm_count()) return launch_row<T, 128>(p, 1, st);
  // Few rows: CTAs of 512 threads with twice the loads in flight, one an SM, in clusters as long as they all
  // run at once and have four vectors a thread: 150 x 131072 bf16 with 5 alternatives 15.6 us, 23.3 by 256
  // threads, 38.6 in clusters of two, which take turns; 30 x 131072 with 20 9.6 us in clusters of four, 18.1 of
  // eight.  Rows of 4096 vectors or less gain nothing by more than 256 threads.
  const int sms = emu_ops_sm_count();
  int C = 1;
  while (C < kMaxCluster && 2 * p.T * C <= sms && nvec >= 2 * C * 512 * 4) C *= 2;
  return p.T <= sms && nvec >= 4096 ? launch_row<T, 512>(p, C, st) : launch_row<T, 256>(p, 1, st);
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

// gx = gl ([v = token] - p) - ge p (log p + H) = p (-ge log p - (ge H + gl)) + gl [v = token], with
// log p = (x - m) - log z.  TPR threads a row and part of it, four vectors each, in fp32 pairs;
// `same` says that logits and gradient rows lie alike about 16-byte addresses.
template <class T, int TPR>
__global__ void __launch_bounds__(256)
logprob_grad_kernel(const LogprobGradParams p, uint32_t parts, bool same) {
  constexpr int VEC = Row<T>::VEC, U = 4;
  const int t = threadIdx.x % TPR;
  const uint32_t unit = blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const uint32_t r32 = unit / parts;
  const int64_t r = r32;
  if (r >= p.T) return;
  const Row<T> row(static_cast<const T*>(p.x) + r * p.ldx, p.V);
  T* gx = static_cast<T*>(p.gx) + r * p.ldo;
  const int v0 = (int)(unit - r32 * parts) * (TPR * U) + t;
  uint4 raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i)
    if (v0 + i * TPR < row.nvec) raw[i] = row.load_raw(v0 + i * TPR);
  const float m = p.stats[r * 3], logz = p.stats[r * 3 + 1], H = p.stats[r * 3 + 2];
  const int64_t tok = p.tokens[r];
  const float given = p.g_logprob ? p.g_logprob[r] : 0.0f;     // asked for beside the token, not after it
  const bool out_of_range = tok != p.ignore && (tok < 0 || tok >= p.V);
  // out of range is an error of the caller's: NaN, even where nothing of the logprob's gradient is asked for
  const float gl = out_of_range ? NAN : tok == p.ignore ? 0.0f : given;
  const float ge = p.g_entropy ? p.g_entropy[r] : 0.0f;
  const bool empty = m == -INFINITY && logz == -INFINITY && !out_of_range;   // out of range: NaN below by gl
  const int hot = !empty && tok >= 0 && tok < p.V ? (int)tok : -1;
  const f2 m2 = pair(-m, -m), z2 = pair(-logz, -logz), L2 = pair(kLog2e, kLog2e), e2 = pair(-ge, -ge);
  const float rest = -fmaf(ge, H, gl);
  const f2 c2 = pair(rest, rest);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = v0 + i * TPR;
    if (v >= row.nvec) break;
    const int id0 = row.first(v);
    float f[VEC];
    Row<T>::unpack(raw[i], f);
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const f2 lp = add2(add2(pair(f[j], f[j + 1]), m2), z2);
      float l0, l1, a0, a1;
      halves(lp, l0, l1);
      halves(mul2(lp, L2), a0, a1);
      const f2 pr = pair(exp2_approx(a0), exp2_approx(a1));
      // p = 0 where log p is -inf: a finite number in its place
      halves(mul2(pr, fma2(pair(max_nan(l0, -1e4f), max_nan(l1, -1e4f)), e2, c2)), f[j], f[j + 1]);
    }
    if (empty) {
      asm volatile("");                                  // branches: few rows and vectors take them
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = 0.0f;
    }
    if ((uint32_t)(hot - id0) < (uint32_t)VEC && hot >= 0) {
      asm volatile("");
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] += id0 + j == hot ? gl : 0.0f;
    }
    if (same && row.whole(v)) {
      store_f<T, VEC>(gx + id0, f);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (id0 + j >= 0 && id0 + j < p.V) gx[id0 + j] = from_f<T>(f[j]);
    }
  }
}

template <class T> void pick_logprob_grad(const LogprobGradParams& p, cudaStream_t st) {
  const int nvec = p.V / Row<T>::VEC + 2;                // at most, wherever a row starts
  const bool same = ((reinterpret_cast<uintptr_t>(p.x) ^ reinterpret_cast<uintptr_t>(p.gx)) & 15u) == 0 &&
                    ((p.ldx - p.ldo) * (int64_t)sizeof(T)) % 16 == 0;
  // rows of parts, at most 2^31 - 1 CTAs a launch
  const int tpr = nvec <= 256 ? 32 : 256;
  const uint32_t parts = (uint32_t)((nvec + tpr * 4 - 1) / (tpr * 4));
  const int64_t rows = ((int64_t)1 << 30) / parts;
  for (int64_t r = 0; r < p.T; r += rows) {
    LogprobGradParams q = p;
    q.T = p.T - r < rows ? p.T - r : rows;
    q.x = static_cast<const T*>(p.x) + r * p.ldx;
    q.gx = static_cast<T*>(p.gx) + r * p.ldo;
    q.tokens += r;
    q.stats += 3 * r;
    if (q.g_logprob) q.g_logprob += r;
    if (q.g_entropy) q.g_entropy += r;
    const int64_t units = q.T * parts;
    if (tpr == 32) logprob_grad_kernel<T, 32><<<(unsigned)((units + 7) / 8), 256, 0, st>>>(q, parts, same);
    else logprob_grad_kernel<T, 256><<<(unsigned)units, 256, 0, st>>>(q, parts, same);
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
  if (!apart({Span(logprob, 1, T, T, 4), Span(entropy, 1, T, T, 4), Span(lse, 1, T, T, 4), Span(stats, T, 3, 3, 4),
              Span(top_logprobs, T, top_k, top_k, 4), Span(top_ids, T, top_k, top_k, 8)},
             {Span(logits, T, ldx, V, elem_bytes(type)), Span(tokens, 1, T, T, 8)}))
    return emu_ops_fail(EMU_EINVAL, "an output overlaps an input or another output");
  LogprobParams p;
  p.x = logits; p.ldx = ldx; p.tokens = tokens; p.ignore = ignore_index;
  p.T = T; p.V = (int)V; p.k = top_k;
  p.logprob = logprob; p.entropy = entropy; p.lse = lse; p.stats = stats; p.top_val = top_logprobs; p.top_id = top_ids;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == EMU_OUT_F32) rc = pick_logprob<float>(p, st);
  else if (type == EMU_OUT_BF16) rc = pick_logprob<__nv_bfloat16>(p, st);
  else rc = pick_logprob<__half>(p, st);
  if (rc != EMU_OK) return rc;
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
  const Span g(grad_logits, T, ldo, V, es);
  if (g.meets(Span(logits, T, ldx, V, es)) && !(grad_logits == logits && ldo == ldx))
    return emu_ops_fail(EMU_EINVAL, "grad_logits overlaps the logits without being them");
  if (!apart({g}, {Span(tokens, 1, T, T, 8), Span(stats, T, 3, 3, 4), Span(grad_logprob, 1, T, T, 4),
                   Span(grad_entropy, 1, T, T, 4)}))
    return emu_ops_fail(EMU_EINVAL, "grad_logits overlaps another input");
  LogprobGradParams p;
  p.x = logits; p.ldx = ldx; p.tokens = tokens; p.ignore = ignore_index; p.T = T; p.V = (int)V;
  p.stats = stats; p.g_logprob = grad_logprob; p.g_entropy = grad_entropy;
  p.gx = grad_logits; p.ldo = ldo;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (type == EMU_OUT_F32) pick_logprob_grad<float>(p, st);
  else if (type == EMU_OUT_BF16) pick_logprob_grad<__nv_bfloat16>(p, st);
  else pick_logprob_grad<__half>(p, st);
  return emu_ops_launched("emu_token_logprobs_backward");
}

}  // extern "C"
