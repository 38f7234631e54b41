// ops_block_quant.cu -- values to FP8 codes with a scale for each block of 128 (rows, columns or
// squares), and SwiGLU between two such products with its inputs kept in 8 bits for the backward
// pass (declared in include/emu_fp8.h).
#include "ops_block.cuh"

#include <type_traits>

namespace emu_ops {

constexpr float kBlockScaleMin = 1.17549435e-38f;        // 2^-126, the smallest scale of a block

struct BlockQuantParams {
  const void* x; int64_t ldx;                            // [T, H]; for SwiGLU [T, 2H]
  const uint8_t* x_end;                                  // where its memory ends
  int64_t T, H;
  int fmt; float qmax;
  uint8_t* q; float* scale;
  uint8_t* kept; float* kept_scale;                      // SwiGLU's checkpoint, or null
  int across;                                            // rows: warps of a CTA on one row, 1 or 8
};

// a block's scale from its largest magnitude (NaN if it holds NaN; Inf counts as NaN: x / Inf would be 0 for the others)
__device__ __forceinline__ float block_scale(float top, float qmax) {
  const float m = top < __int_as_float(0x7F800000) ? top : __int_as_float(0x7FC00000);
  return max_nan(m / qmax, kBlockScaleMin);
}
// 1 / v within 2^-23, of v and 1 / v in the normal range
__device__ __forceinline__ float fast_inverse(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// g / (1 + e^-g) * u by e = e^-|g|, as g - g e / (1 + e) of positive g (no less than g / 2, so that nothing cancels) and g e / (1 + e) of
// negative g: 1 + e^-g would be a divisor past 2^126 from g = -87 on, and infinite from -88.7 on.  e is the square of 2^(-|g| log2(e) / 2),
// which stays in the normal range: within 2^-21 (the instruction's 2^-22 twice) and |g| 2^-24 (its argument's rounding).
__device__ __forceinline__ float swiglu(float g, float u) {
  float root;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(fabsf(g) * -0.72134752f));
  const float e = root * root;
  return fmaf(-fabsf(g), e * fast_inverse(1.0f + e), fmaxf(g, 0.0f)) * u;
}

// ---- 16 bytes of values.  Their magnitudes' order is that of their bits without the sign, NaN above all, so
// the largest is found among whole numbers, of 16-bit types two at a time.
template <class T> struct Vec {
  static constexpr int N = 16 / sizeof(T);               // values
  static constexpr uint32_t MASK = sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
};
template <class T> __device__ __forceinline__ uint32_t top_word(uint32_t a, uint32_t b) {
  if (sizeof(T) == 2) return __vmaxu2(a, b);
  return a > b ? a : b;
}
template <class T> __device__ __forceinline__ uint32_t top_words(uint32_t top, const uint4& v) {
  constexpr uint32_t M = Vec<T>::MASK;
  return top_word<T>(top, top_word<T>(top_word<T>(v.x & M, v.y & M), top_word<T>(v.z & M, v.w & M)));
}
template <class T> __device__ __forceinline__ float2 two_of(uint32_t w);   // a word's values (of fp32 one)
template <> __device__ __forceinline__ float2 two_of<float>(uint32_t w) { return make_float2(__uint_as_float(w), 0.0f); }
template <> __device__ __forceinline__ float2 two_of<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 two_of<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// the largest magnitude that a word of tops holds
template <class T> __device__ __forceinline__ uint32_t join_top(uint32_t top) {
  return sizeof(T) == 2 ? top_word<T>(top, top >> 16) & 0xFFFFu : top;
}
template <class T> __device__ __forceinline__ float top_value(uint32_t top) { return two_of<T>(top).x; }
template <class T> __device__ __forceinline__ void values_of(const uint4& v, float (&f)[Vec<T>::N]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = two_of<T>(w[i]);
    if constexpr (sizeof(T) == 2) {
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    } else {
      f[i] = t.x;
    }
  }
}
template <int LANES> __device__ __forceinline__ uint32_t top_of_lanes(uint32_t v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    const uint32_t w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = w > v ? w : v;
  }
  return v;
}

// 16 bytes of a row's values, `left` of which (bytes) are the row's, zeros behind them.  Unaligned: the two 16-byte
// words that hold them, shifted into place, as far as these lie in the tensor's memory.
template <bool VEC> struct Values {
  Codes<VEC> codes;
  const int8_t* at;
  __device__ __forceinline__ void ask(const void* p, bool in, const void* from, const uint8_t* end) {
    at = static_cast<const int8_t*>(p);
    codes.ask(at, 0, in, static_cast<const int8_t*>(from), reinterpret_cast<uintptr_t>(end));
  }
  __device__ __forceinline__ uint4 get(int64_t left, bool in, const void* from, const uint8_t* end) const {
    return codes.get(at, 0, left < 16 ? (int)left : 16, in, static_cast<const int8_t*>(from), reinterpret_cast<uintptr_t>(end));
  }
};

// what a lane stores, BYTES at once (4, 8 or 16)
template <int BYTES> struct Piece;
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<8> { using type = uint2; };
template <> struct Piece<16> { using type = uint4; };
// the bytes of b behind the last `s` of a (0 < s < BYTES)
__device__ __forceinline__ uint32_t behind(uint32_t a, uint32_t b, int s) { return __funnelshift_l(a, b, 8 * s); }
__device__ __forceinline__ uint2 behind(uint2 a, uint2 b, int s) {
  const unsigned long long x = (unsigned long long)a.y << 32 | a.x, y = (unsigned long long)b.y << 32 | b.x, r = y << (8 * s) | x >> (64 - 8 * s);
  return make_uint2((uint32_t)r, (uint32_t)(r >> 32));
}
__device__ __forceinline__ uint4 behind(uint4 a, uint4 b, int s) { return bytes_from(a, b, 16 - s); }
__device__ __forceinline__ uint32_t before_lane(uint32_t v, int lanes) { return __shfl_up_sync(0xFFFFFFFFu, v, 1, lanes); }
__device__ __forceinline__ uint2 before_lane(uint2 v, int lanes) { return make_uint2(before_lane(v.x, lanes), before_lane(v.y, lanes)); }
__device__ __forceinline__ uint4 before_lane(uint4 v, int lanes) {
  return make_uint4(before_lane(v.x, lanes), before_lane(v.y, lanes), before_lane(v.z, lanes), before_lane(v.w, lanes));
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int lane, int lanes) { return __shfl_sync(0xFFFFFFFFu, v, lane, lanes); }
__device__ __forceinline__ uint2 of_lane(uint2 v, int lane, int lanes) { return make_uint2(of_lane(v.x, lane, lanes), of_lane(v.y, lane, lanes)); }
__device__ __forceinline__ uint4 of_lane(uint4 v, int lane, int lanes) {
  return make_uint4(of_lane(v.x, lane, lanes), of_lane(v.y, lane, lanes), of_lane(v.z, lane, lanes), of_lane(v.w, lane, lanes));
}
__device__ __forceinline__ uint8_t byte_of(uint32_t v, int i) { return (uint8_t)(v >> 8 * i); }
__device__ __forceinline__ uint8_t byte_of(uint2 v, int i) { return byte_of(i & 4 ? v.y : v.x, i & 3); }
__device__ __forceinline__ uint8_t byte_of(uint4 v, int i) { return i & 8 ? byte_of(make_uint2(v.z, v.w), i & 7) : byte_of(make_uint2(v.x, v.y), i & 7); }
// LANES lanes' pieces to `to` (the first lane's address), `count` bytes of them (all or less).  Unaligned: the pieces
// move on by the address's remainder, so that all but the ends are stored whole.  Called by whole warps.
template <int BYTES, int LANES, bool VEC>
__device__ __forceinline__ void store_pieces(uint8_t* to, typename Piece<BYTES>::type v, int64_t count, int in) {
  using P = typename Piece<BYTES>::type;
  if constexpr (VEC) {
    if (in * BYTES < count) *reinterpret_cast<P*>(to + in * BYTES) = v;
  } else {
    static_assert(LANES >= BYTES, "a lane for each byte of the ends");
    const int s = (int)(reinterpret_cast<uintptr_t>(to) & (BYTES - 1));
    const P last = before_lane(v, LANES), head = of_lane(v, 0, LANES), tail = of_lane(v, LANES - 1, LANES);
    const P w = s == 0 ? v : behind(last, v, s);
    const int64_t first = (int64_t)in * BYTES - s;       // of the bytes in w
    if (count >= LANES * BYTES) {
      if (first >= 0) *reinterpret_cast<P*>(to + first) = w;
      if (s > 0 && in < BYTES) {                         // the first BYTES - s bytes, and the last s: one a lane
        const bool at_head = in < BYTES - s;
        to[at_head ? in : (LANES - 1) * BYTES + in] = byte_of(at_head ? head : tail, in);
      }
    } else if ((int64_t)in * BYTES < count) {            // a row's end
#pragma unroll 1
      for (int i = 0; i < BYTES; ++i)
        if ((int64_t)in * BYTES + i < count) to[in * BYTES + i] = byte_of(v, i);
    }
  }
}

// What values are divided by, one scale or S neighbours' each its own: the scale's inverse as the sum of two numbers, so that x hi + x lo,
// the second rounded and the sum once more, is x / scale rounded to fp32 (up to 2^-40), and halfway between two codes where that is.
// hi is below the inverse by some 2^-21 of it and lo not below 0: -0 stays -0.
template <int S> struct Divisor {
  float hi[S], lo[S];
  __device__ __forceinline__ explicit Divisor(const float (&scale)[S]) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      hi[i] = fast_inverse(scale[i]) * (1.0f - 4.76837158e-7f);
      lo[i] = fmaf(-hi[i], scale[i], 1.0f) * hi[i];
    }
  }
};
// codes of a vector's values: their quotients to 8 bits, two at a time (PAIRS) or one by one
template <int FMT, int N, bool PAIRS, int S> __device__ __forceinline__ typename Piece<N>::type codes_of(const float (&v)[N], const Divisor<S>& d) {
  static_assert(S == 1 || S == N, "one scale or one each");
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    uint32_t two[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = 4 * i + 2 * j, a = S == 1 ? 0 : k, b = S == 1 ? 0 : k + 1;
      float q0, q1;
      if constexpr (PAIRS) {
        const f2 x = pair(v[k], v[k + 1]);
        halves(fma2(x, pair(d.hi[a], d.hi[b]), mul2(x, pair(d.lo[a], d.lo[b]))), q0, q1);
      } else {
        q0 = fmaf(v[k], d.hi[a], v[k] * d.lo[a]);
        q1 = fmaf(v[k + 1], d.hi[b], v[k + 1] * d.lo[b]);
      }
      two[j] = __nv_cvt_float2_to_fp8x2(make_float2(q0, q1), __NV_SATFINITE, FMT == EMU_E4M3FN ? __NV_E4M3 : __NV_E5M2);
    }
    w[i] = two[0] | two[1] << 16;
  }
  if constexpr (N == 4) return w[0];
  else return make_uint2(w[0], w[1]);
}
template <int FMT, int N> __device__ __forceinline__ typename Piece<N>::type codes_of(const float (&v)[N], float scale) {
  const float one[1] = {scale};
  return codes_of<FMT, N, true>(v, Divisor<1>(one));
}

// 1 x 128 blocks: 128 / N lanes hold one.  A warp takes UNROLL loads of a row (32 N values each) at a time, all asked for
// before the first is waited for.  Bound by the instructions around the maxima: 8192 x 5760 bf16 in 27 us, 5.2 TB/s.
template <class T, bool VEC, int FMT, bool SWIGLU, int UNROLL>
__global__ void __launch_bounds__(256) block_rows_kernel(const BlockQuantParams p) {
  constexpr int N = Vec<T>::N, LANES = 128 / N, BYTES = N;                // a lane's codes of a load are N bytes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = lane % LANES;
  const int64_t blocks = (p.H + 127) / 128, per = 32 * N;
  const int64_t seg = ((int64_t)blockIdx.x * p.across + warp % p.across) * UNROLL;
  for (int64_t row = (int64_t)blockIdx.y * (8 / p.across) + warp / p.across; row < p.T; row += (int64_t)gridDim.y * (8 / p.across)) {
    const T* const x = static_cast<const T*>(p.x) + row * p.ldx;
    Values<VEC> av[UNROLL], ag[SWIGLU ? UNROLL : 1];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int64_t col = (seg + i) * per + lane * N;
      if (SWIGLU) ag[i].ask(x + col, col < p.H, p.x, p.x_end);
      av[i].ask(x + (SWIGLU ? p.H : 0) + col, col < p.H, p.x, p.x_end);
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      if ((seg + i) * per >= p.H) break;                 // the same for all lanes
      const int64_t col = (seg + i) * per + lane * N, left = (p.H - col) * (int64_t)sizeof(T);
      const int64_t block = (seg + i) * (per / 128) + lane / LANES, from = block * 128;
      const uint4 r = av[i].get(left, col < p.H, p.x, p.x_end);
      float v[N], scale;
      values_of<T>(r, v);
      uint32_t top;
      if constexpr (SWIGLU) {
        const uint4 rg = ag[i].get(left, col < p.H, p.x, p.x_end);
        float g[N];
        values_of<T>(rg, g);
        if (p.kept) {
          const float sg = block_scale(top_value<T>(top_of_lanes<LANES>(join_top<T>(top_words<T>(0u, rg)))), 448.0f);
          const float su = block_scale(top_value<T>(top_of_lanes<LANES>(join_top<T>(top_words<T>(0u, r)))), 448.0f);
          uint8_t* const to = p.kept + row * 2 * p.H + from;
          store_pieces<BYTES, LANES, VEC>(to, codes_of<EMU_E4M3FN, N>(g, sg), p.H - from, in);
          store_pieces<BYTES, LANES, VEC>(to + p.H, codes_of<EMU_E4M3FN, N>(v, su), p.H - from, in);
          if (in == 0 && block < blocks) {
            p.kept_scale[row * 2 * blocks + block] = sg;
            p.kept_scale[row * 2 * blocks + blocks + block] = su;
          }
        }
        top = 0u;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          v[k] = swiglu(g[k], v[k]);
          top = top_word<float>(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        }
        scale = block_scale(__uint_as_float(top_of_lanes<LANES>(top)), p.qmax);
      } else {
        scale = block_scale(top_value<T>(top_of_lanes<LANES>(join_top<T>(top_words<T>(0u, r)))), p.qmax);
      }
      store_pieces<BYTES, LANES, VEC>(p.q + row * p.H + from, codes_of<FMT, N>(v, scale), p.H - from, in);
      if (in == 0 && block < blocks) p.scale[row * blocks + block] = scale;
    }
  }
}

// 128 x 1 and 128 x 128 blocks: a CTA of 256 threads holds 128 rows x 128 columns in registers, 128 / N threads a row, finds
// the columns' or the tile's largest magnitudes and writes the codes.  8192 x 5760 bf16: squares in 23 us, 6.2 TB/s (91% of a
// copy's rate), columns in 26.
template <class T, bool VEC, int FMT, bool SWIGLU, bool SQUARE>
__global__ void __launch_bounds__(256) block_tile_kernel(const BlockQuantParams p) {
  constexpr int N = Vec<T>::N, LANES = 128 / N, ROWS = 256 / LANES, PASSES = 128 / ROWS;
  __shared__ uint4 tops[SQUARE ? 1 : 8][SQUARE ? 2 : LANES];              // a warp's tops: of columns, or one word
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = threadIdx.x % LANES, r0 = threadIdx.x / LANES;
  const int64_t blocks = (p.H + 127) / 128, from = (int64_t)blockIdx.x * 128, col = from + in * N;
  const int64_t row0 = (int64_t)blockIdx.y * 128, left = (p.H - col) * (int64_t)sizeof(T);
  const T* const x = static_cast<const T*>(p.x);
  Values<VEC> av[PASSES], ag[SWIGLU ? PASSES : 1];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = row0 + r0 + i * ROWS;
    const bool in_x = row < p.T && col < p.H;
    if (SWIGLU) ag[i].ask(x + row * p.ldx + col, in_x, p.x, p.x_end);
    av[i].ask(x + row * p.ldx + (SWIGLU ? p.H : 0) + col, in_x, p.x, p.x_end);
  }
  uint4 raw[SWIGLU ? 1 : PASSES];
  float y[SWIGLU ? PASSES : 1][N];
  uint32_t top = 0u;
  uint4 tops4 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = row0 + r0 + i * ROWS;
    const bool in_x = row < p.T && col < p.H;
    const uint4 r = av[i].get(left, in_x, p.x, p.x_end);
    if constexpr (SWIGLU) {
      const uint4 rg = ag[i].get(left, in_x, p.x, p.x_end);
      float g[N], u[N];
      values_of<T>(rg, g);
      values_of<T>(r, u);
      if (p.kept) {
        const float sg = block_scale(top_value<T>(top_of_lanes<LANES>(join_top<T>(top_words<T>(0u, rg)))), 448.0f);
        const float su = block_scale(top_value<T>(top_of_lanes<LANES>(join_top<T>(top_words<T>(0u, r)))), 448.0f);
        uint8_t* const to = p.kept + row * 2 * p.H + from;
        const int64_t count = row < p.T ? p.H - from : 0;
        store_pieces<N, LANES, VEC>(to, codes_of<EMU_E4M3FN, N>(g, sg), count, in);
        store_pieces<N, LANES, VEC>(to + p.H, codes_of<EMU_E4M3FN, N>(u, su), count, in);
        if (in == 0 && row < p.T) {
          p.kept_scale[row * 2 * blocks + blockIdx.x] = sg;
          p.kept_scale[row * 2 * blocks + blocks + blockIdx.x] = su;
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        y[i][k] = swiglu(g[k], u[k]);
        top = top_word<float>(top, __float_as_uint(y[i][k]) & 0x7FFFFFFFu);
      }
    } else {
      raw[i] = r;
      constexpr uint32_t M = Vec<T>::MASK;
      if (SQUARE) top = top_words<T>(top, r);
      else tops4 = make_uint4(top_word<T>(tops4.x, r.x & M), top_word<T>(tops4.y, r.y & M), top_word<T>(tops4.z, r.z & M),
                              top_word<T>(tops4.w, r.w & M));
    }
  }
  float scale[SQUARE ? 1 : N];
  if constexpr (SQUARE) {
    uint32_t* const words = reinterpret_cast<uint32_t*>(tops);
    const uint32_t one = __reduce_max_sync(0xFFFFFFFFu, SWIGLU ? top : join_top<T>(top));
    if (lane == 0) words[warp] = one;
    __syncthreads();
    uint32_t all = words[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) all = words[i] > all ? words[i] : all;
    scale[0] = block_scale(SWIGLU ? __uint_as_float(all) : top_value<T>(all), p.qmax);
    if (threadIdx.x == 0) p.scale[(int64_t)blockIdx.y * blocks + blockIdx.x] = scale[0];
  } else {
#pragma unroll
    for (int o = LANES; o < 32; o *= 2)                  // rows that share a warp
      tops4 = make_uint4(top_word<T>(tops4.x, __shfl_xor_sync(0xFFFFFFFFu, tops4.x, o)), top_word<T>(tops4.y, __shfl_xor_sync(0xFFFFFFFFu, tops4.y, o)),
                         top_word<T>(tops4.z, __shfl_xor_sync(0xFFFFFFFFu, tops4.z, o)), top_word<T>(tops4.w, __shfl_xor_sync(0xFFFFFFFFu, tops4.w, o)));
    if (lane < LANES) tops[warp][lane] = tops4;
    __syncthreads();
    uint4 all = tops[0][in];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const uint4 t = tops[i][in];
      all = make_uint4(top_word<T>(all.x, t.x), top_word<T>(all.y, t.y), top_word<T>(all.z, t.z), top_word<T>(all.w, t.w));
    }
    float of[N];
    values_of<T>(all, of);
#pragma unroll
    for (int k = 0; k < N; ++k) scale[k] = block_scale(of[k], p.qmax);
    if (r0 == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (col + k < p.H) p.scale[(int64_t)blockIdx.y * p.H + col + k] = scale[k];
    }
  }
  constexpr bool PAIRS = SWIGLU || !SQUARE || !VEC;       // squares of aligned rows: 22.7 us so, 25.8 in pairs; columns 26.6 and 26.0
  const Divisor<SQUARE ? 1 : N> divisor(scale);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = row0 + r0 + i * ROWS;
    float v[N];
    if constexpr (SWIGLU) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = y[i][k];
    } else {
      values_of<T>(raw[i], v);
    }
    store_pieces<N, LANES, VEC>(p.q + row * p.H + from, codes_of<FMT, N, PAIRS>(v, divisor), row < p.T ? p.H - from : 0, in);
  }
}

struct SwigluGradParams {
  const void* gy; int64_t ldy; const uint8_t* gy_end;    // [T, H]
  int64_t T, H;
  const uint8_t* kept; const uint8_t* kept_end; const float* kept_scale;
  void* out;                                             // [T, 2H]
};

// the values of N codes, the first in the lowest byte
template <int N> __device__ __forceinline__ void values_of_codes(const uint32_t (&w)[N / 4], float scale, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[i / 2] >> (i & 1) * 16), __NV_E4M3)));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}
// Gradients by g and u, in their places, with 1 / (1 + e^-g) as in swiglu: of fp32 with expf (the fast exponential is off by 1.2 |g| 2^-23,
// which 16-bit gradients round away; 4096 x 5760 takes the same 50 us).  By a root as in swiglu: more registers, 64 us instead of 58.
template <class T, int N> __device__ __forceinline__ void swiglu_grads(const float (&gy)[N], float (&g)[N], float (&u)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float e = sizeof(T) == 4 ? expf(-fabsf(g[k])) : __expf(-fabsf(g[k]));
    const float sig = (g[k] < 0.0f ? e : 1.0f) * fast_inverse(1.0f + e);
    const float a = gy[k] * sig, grad_u = a * g[k];
    g[k] = u[k] * fmaf(a, g[k] * (1.0f - sig), a);
    u[k] = grad_u;
  }
}

// Aligned rows: a vector of grad_y a thread at a time; its 1 x 128 blocks are those of both halves.  8192 x 5760 bf16 in 58 us:
// 6.5 TB/s, 96% of a copy's rate.  (256, 8): 32 registers, so that the SM is full of warps (fp32 with 40 53 us instead of 50).
template <class T>
__global__ void __launch_bounds__(256, 8) swiglu_grad_kernel(const SwigluGradParams p) {
  constexpr int N = Vec<T>::N;
  const int64_t blocks = (p.H + 127) / 128, per_row = p.H / N, total = p.T * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row, col = (i - row * per_row) * N;
    float gy[N], g[N], u[N];
    load_f<T, N>(static_cast<const T*>(p.gy) + row * p.ldy + col, gy);
    const float* const s = p.kept_scale + row * 2 * blocks + col / 128;
    alignas(N) uint32_t wg[N / 4], wu[N / 4];
    *reinterpret_cast<typename Piece<N>::type*>(wg) = *reinterpret_cast<const typename Piece<N>::type*>(p.kept + row * 2 * p.H + col);
    *reinterpret_cast<typename Piece<N>::type*>(wu) = *reinterpret_cast<const typename Piece<N>::type*>(p.kept + row * 2 * p.H + p.H + col);
    values_of_codes<N>(wg, s[0], g);
    values_of_codes<N>(wu, s[blocks], u);
    swiglu_grads<T, N>(gy, g, u);
    T* const out = static_cast<T*>(p.out) + row * 2 * p.H + col;
    store_f<T, N>(out, g);
    store_f<T, N>(out + p.H, u);
  }
}

// N codes of a row, `left` of which are the row's, as 16 bytes of which the first N are taken
template <int N> struct KeptCodes {
  Codes<false> sixteen;
  const int8_t* at;
  __device__ __forceinline__ void ask(const uint8_t* p, bool in, const uint8_t* from, const uint8_t* end) {
    at = reinterpret_cast<const int8_t*>(p);
    sixteen.ask(at, 0, in, reinterpret_cast<const int8_t*>(from), reinterpret_cast<uintptr_t>(end));
  }
  __device__ __forceinline__ void get(int64_t left, bool in, const uint8_t* from, const uint8_t* end, uint32_t (&r)[N / 4]) const {
    const uint4 v = sixteen.get(at, 0, left < N ? (int)left : N, in, reinterpret_cast<const int8_t*>(from), reinterpret_cast<uintptr_t>(end));
    r[0] = v.x;
    if constexpr (N == 8) r[1] = v.y;
  }
};

// Rows at any address: a warp's lanes take a row's neighbouring vectors.  8192 x 5761 bf16 in 122 us.
template <class T>
__global__ void __launch_bounds__(256) swiglu_grad_unaligned_kernel(const SwigluGradParams p) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t blocks = (p.H + 127) / 128, first = (int64_t)blockIdx.x * 32 * N, col = first + lane * N;
  const bool in = col < p.H;
  for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < p.T; row += (int64_t)gridDim.y * 8) {
    Values<false> ay;
    KeptCodes<N> ag, au;
    ay.ask(static_cast<const T*>(p.gy) + row * p.ldy + col, in, p.gy, p.gy_end);
    ag.ask(p.kept + row * 2 * p.H + col, in, p.kept, p.kept_end);
    au.ask(p.kept + row * 2 * p.H + p.H + col, in, p.kept, p.kept_end);
    const float* const s = p.kept_scale + row * 2 * blocks + col / 128;
    const float sg = in ? __ldg(s) : 0.0f, su = in ? __ldg(s + blocks) : 0.0f;
    float gy[N], g[N], u[N];
    uint32_t wg[N / 4], wu[N / 4];
    values_of<T>(ay.get((p.H - col) * (int64_t)sizeof(T), in, p.gy, p.gy_end), gy);
    ag.get(p.H - col, in, p.kept, p.kept_end, wg);
    au.get(p.H - col, in, p.kept, p.kept_end, wu);
    values_of_codes<N>(wg, sg, g);
    values_of_codes<N>(wu, su, u);
    swiglu_grads<T, N>(gy, g, u);
    Pack<T, N> og, ou;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      og.v[k] = from_f<T>(g[k]);
      ou.v[k] = from_f<T>(u[k]);
    }
    uint8_t* const out = static_cast<uint8_t*>(p.out) + (row * 2 * p.H + first) * (int64_t)sizeof(T);
    const int64_t count = (p.H - first) * (int64_t)sizeof(T);
    store_pieces<16, 32, false>(out, *reinterpret_cast<const uint4*>(&og), count, lane);
    store_pieces<16, 32, false>(out + p.H * (int64_t)sizeof(T), *reinterpret_cast<const uint4*>(&ou), count, lane);
  }
}

// so many rows of CTAs (grid.y) that a few rounds of them fill the device: starting tens of thousands takes longer than
// their work
int64_t rows_of_ctas(int64_t wide, int64_t an_sm) {
  const int64_t ctas = emu_ops_sm_count() * an_sm, rows = (ctas + wide - 1) / wide;
  return rows < 65535 ? rows : 65535;
}

template <class T, int FMT, bool SWIGLU> int launch_quant(const BlockQuantParams& p, emu_block_t block, bool vec, cudaStream_t st) {
  const int64_t blocks = (p.H + 127) / 128;
  if (block == EMU_BLOCK_ROWS) {
    // Loads of a warp at a time, as long as the device is full: 8192 x 5760 bf16 27 us with four or two, 39 with one, fp32 42, 48
    // and 55; unaligned 8192 x 5761 49 with two, 62 with four, 53 with one; SwiGLU 79 with two, 86 with one, unaligned
    // 4096 x 5761 71 with one, 81 with two.
    constexpr int MANY = SWIGLU ? 2 : 4, SOME = SWIGLU ? 1 : 2;
    const int64_t loads = (p.H + 32 * Vec<T>::N - 1) / (32 * Vec<T>::N);
    const int unroll = p.T * loads < (int64_t)emu_ops_sm_count() * 32 * MANY ? 1 : vec ? MANY : SOME;
    BlockQuantParams s = p;
    const int64_t segs = (loads + unroll - 1) / unroll;
    s.across = p.T < 8 ? 8 : 1;                          // few rows: the warps of a CTA side by side
    const int64_t rows = (p.T + 8 / s.across - 1) / (8 / s.across);
    const int64_t wide = (segs + s.across - 1) / s.across, most = rows_of_ctas(wide, 16);
    const dim3 grid((unsigned)wide, (unsigned)(rows < most ? rows : most));
    if (unroll == 1) {
      if (vec) block_rows_kernel<T, true, FMT, SWIGLU, 1><<<grid, 256, 0, st>>>(s);
      else block_rows_kernel<T, false, FMT, SWIGLU, 1><<<grid, 256, 0, st>>>(s);
    } else {
      if (vec) block_rows_kernel<T, true, FMT, SWIGLU, MANY><<<grid, 256, 0, st>>>(s);
      else block_rows_kernel<T, false, FMT, SWIGLU, SOME><<<grid, 256, 0, st>>>(s);
    }
    return EMU_OK;
  }
  const int64_t tall = (int64_t)65535 * 128;             // rows of tiles on grid.y
  for (int64_t t = 0; t < p.T; t += tall) {
    BlockQuantParams s = p;
    s.T = p.T - t < tall ? p.T - t : tall;
    s.x = static_cast<const T*>(p.x) + t * p.ldx;
    s.q += t * p.H;
    s.scale += t / 128 * (block == EMU_BLOCK_COLUMNS ? p.H : blocks);
    if (s.kept) {
      s.kept += t * 2 * p.H;
      s.kept_scale += t * 2 * blocks;
    }
    const dim3 grid((unsigned)blocks, (unsigned)((s.T + 127) / 128));
    if (block == EMU_BLOCK_SQUARES) {
      if (vec) block_tile_kernel<T, true, FMT, SWIGLU, true><<<grid, 256, 0, st>>>(s);
      else block_tile_kernel<T, false, FMT, SWIGLU, true><<<grid, 256, 0, st>>>(s);
    } else if constexpr (!SWIGLU) {
      if (vec) block_tile_kernel<T, true, FMT, false, false><<<grid, 256, 0, st>>>(s);
      else block_tile_kernel<T, false, FMT, false, false><<<grid, 256, 0, st>>>(s);
    }
  }
  return EMU_OK;
}
template <bool SWIGLU> int pick_quant(const BlockQuantParams& p, emu_out_t type, emu_block_t block, bool vec, cudaStream_t st) {
  auto fmt = [&](auto t) {
    using T = decltype(t);
    return p.fmt == EMU_E4M3FN ? launch_quant<T, EMU_E4M3FN, SWIGLU>(p, block, vec, st)
                               : launch_quant<T, EMU_E5M2, SWIGLU>(p, block, vec, st);
  };
  if (type == EMU_OUT_F32) return fmt(float());
  return type == EMU_OUT_BF16 ? fmt(__nv_bfloat16()) : fmt(__half());
}

// what the three calls check alike; EMU_OK with *empty set where there is nothing to do
int check_quant(emu_out_t type, int64_t T, int64_t H, bool* empty) {
  if (!is_float_type(type)) return emu_ops_fail(EMU_EINVAL, "the values are fp32, bf16 or fp16 (got %d)", (int)type);
  if (T < 0 || H < 0) return emu_ops_fail(EMU_EINVAL, "negative size (%lld, %lld)", (long long)T, (long long)H);
  if (T >= (int64_t)1 << 31 || H >= (int64_t)1 << 30) return emu_ops_fail(EMU_EUNSUPPORTED, "sizes must be below 2^31 rows and 2^30 values");
  *empty = T == 0 || H == 0;
  return EMU_OK;
}
int64_t scale_rows_of(emu_block_t b, int64_t T) { return b == EMU_BLOCK_ROWS ? T : (T + 127) / 128; }
int64_t scale_cols_of(emu_block_t b, int64_t H) { return b == EMU_BLOCK_COLUMNS ? H : (H + 127) / 128; }

}  // namespace emu_ops

using namespace emu_ops;

extern "C" {

int emu_block_quant(const void* x, int64_t ldx, emu_out_t type, int64_t T, int64_t H, emu_block_t block,
                    emu_fp8_t q_format, void* q, float* scale, void* stream) {
  emu_ops_begin();
  bool empty;
  int rc = check_quant(type, T, H, &empty);
  if (rc != EMU_OK) return rc;
  if (block != EMU_BLOCK_ROWS && block != EMU_BLOCK_COLUMNS && block != EMU_BLOCK_SQUARES)
    return emu_ops_fail(EMU_EINVAL, "unknown block shape %d", (int)block);
  if (q_format != EMU_E4M3FN && q_format != EMU_E5M2) return emu_ops_fail(EMU_EINVAL, "unknown FP8 format %d", (int)q_format);
  if (empty) return EMU_OK;
  if (!x || !q || !scale) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (ldx < H) return emu_ops_fail(EMU_EINVAL, "the row stride is below the row's %lld values", (long long)H);
  const size_t es = elem_bytes(type);
  if (!aligned(x, es) || !aligned(scale, 4)) return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  const int64_t sr = scale_rows_of(block, T), sc = scale_cols_of(block, H);
  if (!apart({Span(q, T, H, H, 1), Span(scale, sr, sc, sc, 4)}, {Span(x, T, ldx, H, es)}))
    return emu_ops_fail(EMU_EINVAL, "an output overlaps the input, or the other");
  const int64_t v = 16 / (int64_t)es;
  const bool vec = H % v == 0 && ldx % v == 0 && aligned(x, 16) && aligned(q, (size_t)v);
  const BlockQuantParams p = {x, ldx, static_cast<const uint8_t*>(x) + ((T - 1) * ldx + H) * (int64_t)es, T, H, (int)q_format, q_format == EMU_E4M3FN ? 448.0f : 57344.0f,
                              static_cast<uint8_t*>(q), scale, nullptr, nullptr, 1};
  rc = pick_quant<false>(p, type, block, vec, static_cast<cudaStream_t>(stream));
  return rc == EMU_OK ? emu_ops_launched("emu_block_quant") : rc;
}

int emu_swiglu_quant(const void* gate_up, int64_t ldx, emu_out_t type, int64_t T, int64_t H, emu_block_t block,
                     emu_fp8_t q_format, void* q, float* scale, void* checkpoint, float* checkpoint_scale,
                     void* stream) {
  emu_ops_begin();
  bool empty;
  int rc = check_quant(type, T, H, &empty);
  if (rc != EMU_OK) return rc;
  if (block != EMU_BLOCK_ROWS && block != EMU_BLOCK_SQUARES)
    return emu_ops_fail(EMU_EINVAL, "the output is quantised in rows or squares (got %d)", (int)block);
  if (q_format != EMU_E4M3FN && q_format != EMU_E5M2) return emu_ops_fail(EMU_EINVAL, "unknown FP8 format %d", (int)q_format);
  if (!checkpoint != !checkpoint_scale) return emu_ops_fail(EMU_EINVAL, "the checkpoint's codes go with its scales");
  if (empty) return EMU_OK;
  if (!gate_up || !q || !scale) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (ldx < 2 * H) return emu_ops_fail(EMU_EINVAL, "the row stride is below the row's %lld values", (long long)(2 * H));
  const size_t es = elem_bytes(type);
  if (!aligned(gate_up, es) || !aligned(scale, 4) || !aligned(checkpoint_scale, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  const int64_t sr = scale_rows_of(block, T), sc = scale_cols_of(block, H), kc = 2 * ((H + 127) / 128);
  if (!apart({Span(q, T, H, H, 1), Span(scale, sr, sc, sc, 4), Span(checkpoint, T, 2 * H, 2 * H, 1), Span(checkpoint_scale, T, kc, kc, 4)},
             {Span(gate_up, T, ldx, 2 * H, es)}))
    return emu_ops_fail(EMU_EINVAL, "an output overlaps the input, or another");
  const int64_t v = 16 / (int64_t)es;
  const bool vec = H % v == 0 && ldx % v == 0 && aligned(gate_up, 16) && aligned(q, (size_t)v) && aligned(checkpoint, (size_t)v);
  const BlockQuantParams p = {gate_up, ldx, static_cast<const uint8_t*>(gate_up) + ((T - 1) * ldx + 2 * H) * (int64_t)es, T, H, (int)q_format, q_format == EMU_E4M3FN ? 448.0f : 57344.0f,
                              static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(checkpoint), checkpoint_scale, 1};
  rc = pick_quant<true>(p, type, block, vec, static_cast<cudaStream_t>(stream));
  return rc == EMU_OK ? emu_ops_launched("emu_swiglu_quant") : rc;
}

int emu_swiglu_backward(const void* grad_y, int64_t ldy, emu_out_t type, int64_t T, int64_t H, const void* checkpoint,
                        const float* checkpoint_scale, void* grad_gate_up, void* stream) {
  emu_ops_begin();
  bool empty;
  const int rc = check_quant(type, T, H, &empty);
  if (rc != EMU_OK) return rc;
  if (empty) return EMU_OK;
  if (!grad_y || !checkpoint || !checkpoint_scale || !grad_gate_up) return emu_ops_fail(EMU_EINVAL, "null tensor");
  if (ldy < H) return emu_ops_fail(EMU_EINVAL, "the row stride is below the row's %lld values", (long long)H);
  const size_t es = elem_bytes(type);
  if (!aligned(grad_y, es) || !aligned(grad_gate_up, es) || !aligned(checkpoint_scale, 4))
    return emu_ops_fail(EMU_EINVAL, "a tensor is not aligned to its elements");
  const int64_t kc = 2 * ((H + 127) / 128);
  if (!apart({Span(grad_gate_up, T, 2 * H, 2 * H, es)},
             {Span(grad_y, T, ldy, H, es), Span(checkpoint, T, 2 * H, 2 * H, 1), Span(checkpoint_scale, T, kc, kc, 4)}))
    return emu_ops_fail(EMU_EINVAL, "the output overlaps an input");
  const int64_t v = 16 / (int64_t)es;
  const bool vec = H % v == 0 && ldy % v == 0 && aligned(grad_y, 16) && aligned(grad_gate_up, 16) && aligned(checkpoint, (size_t)v);
  const SwigluGradParams p = {grad_y, ldy, static_cast<const uint8_t*>(grad_y) + ((T - 1) * ldy + H) * (int64_t)es, T, H,
                              static_cast<const uint8_t*>(checkpoint), static_cast<const uint8_t*>(checkpoint) + T * 2 * H, checkpoint_scale,
                              grad_gate_up};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto t) {
    using V = decltype(t);
    const int64_t sms = emu_ops_sm_count();
    if (vec) {
      const int64_t ctas = (T * (H / v) + 255) / 256;
      swiglu_grad_kernel<V><<<(unsigned)(ctas < sms * 64 ? ctas : sms * 64), 256, 0, st>>>(p);
    } else {
      const int64_t segs = (H + 32 * v - 1) / (32 * v), rows = (T + 7) / 8, most = rows_of_ctas(segs, 64);
      swiglu_grad_unaligned_kernel<V><<<dim3((unsigned)segs, (unsigned)(rows < most ? rows : most)), 256, 0, st>>>(p);
    }
  };
  if (type == EMU_OUT_F32) go(float());
  else if (type == EMU_OUT_BF16) go(__nv_bfloat16());
  else go(__half());
  return emu_ops_launched("emu_swiglu_backward");
}

}  // extern "C"
