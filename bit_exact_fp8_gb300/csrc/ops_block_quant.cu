// ops_block_quant.cu -- values to FP8 codes with a scale for each block of 128 (rows, columns or
// squares), and SwiGLU between two such products with its inputs kept in 8 bits for the backward
// pass (declared in include/emu_fp8.h).
#include "ops_block.cuh"

#include <type_traits>

namespace emu_ops {

constexpr float kBlockScaleMin = 1.17549435e-38f;        // 2^-126, the smallest scale of a block

struct BlockQuantParams {
  const void* x; int64_t ldx;                            // [T, H]; for SwiGLU [T, 2H]
  int64_t T, H;
  int fmt; float qmax;
  uint8_t* q; float* scale;
  uint8_t* kept; float* kept_scale;                      // SwiGLU's checkpoint, or null
};

// what a block's values are multiplied by, and its scale, from its largest magnitude (NaN if it holds
// NaN; Inf counts as NaN: x / Inf would be 0 for the others)
__device__ __forceinline__ void block_factor(float top, float qmax, float& by, float& scale) {
  const float m = top < __int_as_float(0x7F800000) ? top : __int_as_float(0x7FC00000);
  scale = max_nan(m / qmax, kBlockScaleMin);
  by = m < qmax * kBlockScaleMin ? 1.0f / kBlockScaleMin : qmax / m;
}
__device__ __forceinline__ float top_of(float a, float b) { return max_nan(a, fabsf(b)); }
__device__ __forceinline__ float swiglu(float g, float u) { return g * __fdividef(1.0f, 1.0f + __expf(-g)) * u; }

// two codes, the first in the low byte
template <int FMT> __device__ __forceinline__ uint32_t codes2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, FMT == EMU_E4M3FN ? __NV_E4M3 : __NV_E5M2);
}
template <int FMT, int N> __device__ __forceinline__ void store_codes(uint8_t* to, const float (&v)[N], float by) {
  if constexpr (N == 1) {
    *to = (uint8_t)codes2<FMT>(v[0] * by, 0.0f);
  } else {
    Pack<uint16_t, N / 2> p;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p.v[i] = (uint16_t)codes2<FMT>(v[2 * i] * by, v[2 * i + 1] * by);
    *reinterpret_cast<Pack<uint16_t, N / 2>*>(to) = p;
  }
}
template <int LANES> __device__ __forceinline__ float top_of_lanes(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// 1 x 128 blocks: LANES lanes hold one, VEC values a load.  Each warp takes UNROLL times 32 / LANES blocks at a
// time, all loads asked for before the first is waited for.
template <class T, int VEC, int FMT, bool SWIGLU, int UNROLL>
__global__ void __launch_bounds__(256) block_rows_kernel(const BlockQuantParams p) {
  constexpr int LANES = 128 / VEC < 32 ? 128 / VEC : 32, PARTS = 128 / (LANES * VEC), EACH = 32 / LANES;
  const int lane = threadIdx.x & 31, in = lane % LANES;
  const int64_t blocks = (p.H + 127) / 128, total = p.T * blocks;
  const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (UNROLL * EACH) + lane / LANES;
  const T* const x = static_cast<const T*>(p.x);
  float v[UNROLL][PARTS][VEC], g[SWIGLU ? UNROLL : 1][PARTS][VEC];
  int64_t row[UNROLL];
  int block[UNROLL];
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    const int64_t unit = first + i * EACH;
    row[i] = unit < total ? unit / blocks : -1;
    block[i] = (int)(unit - row[i] * blocks);
#pragma unroll
    for (int j = 0; j < PARTS; ++j) {
      const int64_t col = (int64_t)block[i] * 128 + (j * LANES + in) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i][j][k] = 0.0f;
      if (SWIGLU) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) g[i][j][k] = 0.0f;
      }
      if (row[i] >= 0 && col < p.H) {
        if (SWIGLU) load_f<T, VEC>(x + row[i] * p.ldx + col, g[i][j]);
        load_f<T, VEC>(x + row[i] * p.ldx + (SWIGLU ? p.H : 0) + col, v[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    if (SWIGLU && p.kept) {
      float tg = 0.0f, tu = 0.0f, bg, bu, sg, su;
#pragma unroll
      for (int j = 0; j < PARTS; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          tg = top_of(tg, g[i][j][k]);
          tu = top_of(tu, v[i][j][k]);
        }
      block_factor(top_of_lanes<LANES>(tg), 448.0f, bg, sg);
      block_factor(top_of_lanes<LANES>(tu), 448.0f, bu, su);
      if (row[i] >= 0) {
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
          const int64_t col = (int64_t)block[i] * 128 + (j * LANES + in) * VEC;
          if (col < p.H) {
            store_codes<EMU_E4M3FN, VEC>(p.kept + row[i] * 2 * p.H + col, g[i][j], bg);
            store_codes<EMU_E4M3FN, VEC>(p.kept + row[i] * 2 * p.H + p.H + col, v[i][j], bu);
          }
        }
        if (in == 0) {
          p.kept_scale[row[i] * 2 * blocks + block[i]] = sg;
          p.kept_scale[row[i] * 2 * blocks + blocks + block[i]] = su;
        }
      }
    }
    float top = 0.0f, by, scale;
#pragma unroll
    for (int j = 0; j < PARTS; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (SWIGLU) v[i][j][k] = swiglu(g[i][j][k], v[i][j][k]);
        top = top_of(top, v[i][j][k]);
      }
    if (!SWIGLU || p.q) {
      block_factor(top_of_lanes<LANES>(top), p.qmax, by, scale);
      if (row[i] >= 0) {
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
          const int64_t col = (int64_t)block[i] * 128 + (j * LANES + in) * VEC;
          if (col < p.H) store_codes<FMT, VEC>(p.q + row[i] * p.H + col, v[i][j], by);
        }
        if (in == 0) p.scale[row[i] * blocks + block[i]] = scale;
      }
    }
  }
}

// 128 x 1 and 128 x 128 blocks: a CTA holds 128 rows x 128 columns in registers, 128 / VEC threads a row
// (unaligned: one value a load), finds the columns' or the tile's largest magnitudes and writes the codes.
template <class T, int VEC, int FMT, bool SWIGLU, bool SQUARE, int THREADS>
__global__ void __launch_bounds__(THREADS) block_tile_kernel(const BlockQuantParams p) {
  constexpr int ACROSS = 128 / VEC, ROWS = THREADS / ACROSS, PASSES = 128 / ROWS, WARPS = THREADS / 32;
  __shared__ float tops[SQUARE ? 1 : ROWS][SQUARE ? 32 : 128];
  const int in = threadIdx.x % ACROSS, r0 = threadIdx.x / ACROSS, lane = threadIdx.x & 31;
  const int64_t blocks = (p.H + 127) / 128;
  const int64_t row0 = (int64_t)blockIdx.y * 128, col = (int64_t)blockIdx.x * 128 + in * VEC;
  const T* const x = static_cast<const T*>(p.x);
  float v[PASSES][VEC];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = row0 + r0 + i * ROWS;
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[i][k] = 0.0f;
    if (row < p.T && col < p.H) load_f<T, VEC>(x + row * p.ldx + (SWIGLU ? p.H : 0) + col, v[i]);
  }
  if constexpr (SWIGLU) {
    static_assert(VEC == 1 || ACROSS <= 32, "a row of the tile in one warp's lanes");
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int64_t row = row0 + r0 + i * ROWS;
      const bool there = row < p.T && col < p.H;
      float g[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) g[k] = 0.0f;
      if (there) load_f<T, VEC>(x + row * p.ldx + col, g);
      if (p.kept) {
        float tg = 0.0f, tu = 0.0f, bg, bu, sg, su;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          tg = top_of(tg, g[k]);
          tu = top_of(tu, v[i][k]);
        }
        tg = top_of_lanes<(ACROSS < 32 ? ACROSS : 32)>(tg);
        tu = top_of_lanes<(ACROSS < 32 ? ACROSS : 32)>(tu);
        if constexpr (ACROSS > 32) {                     // a row in four warps
          __shared__ float part[2][WARPS];
          __syncthreads();
          if (lane == 0) {
            part[0][threadIdx.x / 32] = tg;
            part[1][threadIdx.x / 32] = tu;
          }
          __syncthreads();
          const int w = threadIdx.x / 32 / 4 * 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            tg = max_nan(tg, part[0][w + k]);
            tu = max_nan(tu, part[1][w + k]);
          }
        }
        block_factor(tg, 448.0f, bg, sg);
        block_factor(tu, 448.0f, bu, su);
        if (there) {
          store_codes<EMU_E4M3FN, VEC>(p.kept + row * 2 * p.H + col, g, bg);
          store_codes<EMU_E4M3FN, VEC>(p.kept + row * 2 * p.H + p.H + col, v[i], bu);
          if (in == 0) {
            p.kept_scale[row * 2 * blocks + blockIdx.x] = sg;
            p.kept_scale[row * 2 * blocks + blocks + blockIdx.x] = su;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i][k] = swiglu(g[k], v[i][k]);
    }
  }
  float by[VEC], scale[VEC];
  if constexpr (SQUARE) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) top = top_of(top, v[i][k]);
    top = warp_max_nan(top);
    if (lane == 0) tops[0][threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WARPS; ++k) top = max_nan(top, tops[0][k]);
    block_factor(top, p.qmax, by[0], scale[0]);
#pragma unroll
    for (int k = 1; k < VEC; ++k) by[k] = by[0];
    if (threadIdx.x == 0) p.scale[(int64_t)blockIdx.y * blocks + blockIdx.x] = scale[0];
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) top = top_of(top, v[i][k]);
      tops[r0][in * VEC + k] = top;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float top = 0.0f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) top = max_nan(top, tops[r][in * VEC + k]);
      block_factor(top, p.qmax, by[k], scale[k]);
    }
    if (r0 == 0 && col < p.H) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) p.scale[(int64_t)blockIdx.y * p.H + col + k] = scale[k];
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = row0 + r0 + i * ROWS;
    if (row < p.T && col < p.H) {
      uint8_t* const to = p.q + row * p.H + col;
      if constexpr (SQUARE) {
        store_codes<FMT, VEC>(to, v[i], by[0]);
      } else {
        float w[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) w[k] = v[i][k] * by[k];
        store_codes<FMT, VEC>(to, w, 1.0f);
      }
    }
  }
}

struct SwigluGradParams {
  const void* gy; int64_t ldy;                           // [T, H]
  int64_t T, H;
  const uint8_t* kept; const float* kept_scale;
  void* out;                                             // [T, 2H]
};

template <int VEC> __device__ __forceinline__ void load_codes(const uint8_t* from, float scale, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = __half2float(__half(__nv_cvt_fp8_to_halfraw(*from, __NV_E4M3))) * scale;
  } else {
    const Pack<uint16_t, VEC / 2> c = *reinterpret_cast<const Pack<uint16_t, VEC / 2>*>(from);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c.v[i], __NV_E4M3)));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
}

// one vector of grad_y a thread at a time; its 1 x 128 blocks are those of both halves
template <class T, int VEC>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(const SwigluGradParams p) {
  const int64_t blocks = (p.H + 127) / 128, per_row = (p.H + VEC - 1) / VEC, total = p.T * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per_row, col = (i - row * per_row) * VEC;
    float gy[VEC], g[VEC], u[VEC];
    load_f<T, VEC>(static_cast<const T*>(p.gy) + row * p.ldy + col, gy);
    const float* const s = p.kept_scale + row * 2 * blocks + col / 128;
    load_codes<VEC>(p.kept + row * 2 * p.H + col, s[0], g);
    load_codes<VEC>(p.kept + row * 2 * p.H + p.H + col, s[blocks], u);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float e = __expf(-g[k]), sig = __fdividef(1.0f, 1.0f + e), silu = g[k] * sig;
      const float grad_u = gy[k] * silu;
      g[k] = gy[k] * u[k] * (sig + silu * (1.0f - sig));
      u[k] = grad_u;
    }
    T* const out = static_cast<T*>(p.out) + row * 2 * p.H + col;
    store_f<T, VEC>(out, g);
    store_f<T, VEC>(out + p.H, u);
  }
}

template <class T, int FMT, bool SWIGLU> int launch_quant(const BlockQuantParams& p, emu_block_t block, bool vec, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t blocks = (p.H + 127) / 128;
  if (block == EMU_BLOCK_ROWS) {
    constexpr int UNROLL = SWIGLU ? 2 : 4;
    const int64_t each = 8 * UNROLL * (vec ? (128 / VEC < 32 ? 32 / (128 / VEC) : 1) : 1);
    const int64_t ctas = (p.T * blocks + each - 1) / each;
    if (ctas >= (int64_t)1 << 31) return emu_ops_fail(EMU_EUNSUPPORTED, "too many blocks");
    if (vec) block_rows_kernel<T, VEC, FMT, SWIGLU, UNROLL><<<(unsigned)ctas, 256, 0, st>>>(p);
    else block_rows_kernel<T, 1, FMT, SWIGLU, UNROLL><<<(unsigned)ctas, 256, 0, st>>>(p);
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
      if (vec) block_tile_kernel<T, VEC, FMT, SWIGLU, true, 256><<<grid, 256, 0, st>>>(s);
      else block_tile_kernel<T, 1, FMT, SWIGLU, true, 512><<<grid, 512, 0, st>>>(s);
    } else if constexpr (!SWIGLU) {
      if (vec) block_tile_kernel<T, VEC, FMT, false, false, 256><<<grid, 256, 0, st>>>(s);
      else block_tile_kernel<T, 1, FMT, false, false, 512><<<grid, 512, 0, st>>>(s);
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
  const bool vec = H % v == 0 && ldx % v == 0 && aligned(x, 16) && aligned(q, (size_t)v) && aligned(scale, 16);
  const BlockQuantParams p = {x, ldx, T, H, (int)q_format, q_format == EMU_E4M3FN ? 448.0f : 57344.0f,
                              static_cast<uint8_t*>(q), scale, nullptr, nullptr};
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
  const BlockQuantParams p = {gate_up, ldx, T, H, (int)q_format, q_format == EMU_E4M3FN ? 448.0f : 57344.0f,
                              static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(checkpoint), checkpoint_scale};
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
  const SwigluGradParams p = {grad_y, ldy, T, H, static_cast<const uint8_t*>(checkpoint), checkpoint_scale, grad_gate_up};
  const int64_t work = T * (vec ? H / v : H), most = (int64_t)emu_ops_sm_count() * 64, ctas = (work + 255) / 256;
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto t) {
    using V = decltype(t);
    if (vec) swiglu_grad_kernel<V, 16 / sizeof(V)><<<grid, 256, 0, st>>>(p);
    else swiglu_grad_kernel<V, 1><<<grid, 256, 0, st>>>(p);
  };
  if (type == EMU_OUT_F32) go(float());
  else if (type == EMU_OUT_BF16) go(__nv_bfloat16());
  else go(__half());
  return emu_ops_launched("emu_swiglu_backward");
}

}  // extern "C"
