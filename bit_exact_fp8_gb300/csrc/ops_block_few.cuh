// ops_block_few.cuh -- the FP8 products with block scales for up to eight tokens.
//
// What counts is reading the weights once, and how many of their bytes are under way.  A warp takes 16 rows of
// the weights (the M side of mma.sync m16n8k32) by 8 tokens, and its lanes load fragments straight from
// memory: the order of K within a block is free as long as both sides keep to one, so a quad's lanes take 16
// contiguous codes each of either half of a row's block, four MMAs' worth together.  The warps of a CTA
// share out the blocks of K, and their sums meet in shared memory in a fixed order.
// 1 x 5760 x 1920 in 4.2 us, 2.0 of them the launch (by tcgen05 7.4: its steps are longer).
#pragma once
#include "ops_block.cuh"

namespace emu_ops {

struct BlockFewParams {
  const uint8_t* w; int64_t w_row; uintptr_t w_end;      // [N][K], and where its memory ends
  const float* ws; int ws_shift; int64_t ws_row, ws_k;
  const uint8_t* t; int64_t t_row; uintptr_t t_end;      // [M][K]
  const float* ts; int ts_shift; int64_t ts_row, ts_k;
  int64_t N;
  int M, K, share;                                          // warps that share out K: 1, 2, 4 or 8
  void* out; int out_type;                               // [M, N]
};

template <int FW, int FT> __device__ __forceinline__ void mma_fp8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                                  uint32_t b0, uint32_t b1) {
#define EMU_MMA(A, B)                                                                                                       \
  asm("mma.sync.aligned.m16n8k32.row.col.f32." A "." B ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};" \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if (FW == EMU_E4M3FN && FT == EMU_E4M3FN) EMU_MMA("e4m3", "e4m3");
  else if (FW == EMU_E4M3FN) EMU_MMA("e4m3", "e5m2");
  else if (FT == EMU_E4M3FN) EMU_MMA("e5m2", "e4m3");
  else EMU_MMA("e5m2", "e5m2");
#undef EMU_MMA
}

// VEC: rows of whole 16-byte chunks; else a chunk is the two aligned words that hold it, shifted into place (1 x 5760 x 1921
// 9.5 us so, 12.8 by way of aligned copies).
template <int FW, int FT, bool VEC>
__global__ void __launch_bounds__(256) block_few_kernel(const BlockFewParams p) {
  __shared__ float sums[8][8][17];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int kb_all = (p.K + kBlock - 1) / kBlock;
  const int rows = 16 * (8 / p.share), part = warp % p.share;            // of a CTA; this warp's part of K
  const int64_t n0 = (int64_t)blockIdx.x * rows, n = n0 + warp / p.share * 16 + g;
  const bool in0 = n < p.N, in1 = n + 8 < p.N, tin = g < p.M;
  const uint8_t* const w0 = p.w + n * p.w_row + q * 16;
  const uint8_t* const w1 = w0 + 8 * p.w_row;
  const uint8_t* const tok = p.t + g * p.t_row + q * 16;
  const float* const s0 = p.ws + ((in0 ? n : 0) >> p.ws_shift) * p.ws_row;
  const float* const s1 = p.ws + ((in1 ? n + 8 : 0) >> p.ws_shift) * p.ws_row;
  const float* const st0 = p.ts + ((q * 2) >> p.ts_shift) * p.ts_row;
  const float* const st1 = p.ts + ((q * 2 + 1) >> p.ts_shift) * p.ts_row;
  const int8_t* const w_at = reinterpret_cast<const int8_t*>(p.w);
  const int8_t* const t_at = reinterpret_cast<const int8_t*>(p.t);
  float acc[4] = {};
#pragma unroll (VEC ? 2 : 1)
  for (int kb = part; kb < kb_all; kb += p.share) {
    const int left = p.K - (kb * kBlock + q * 16);       // codes of the row from the first chunk's on
    const int64_t at = (int64_t)kb * kBlock;
    Codes<VEC> ask[6];
    const int8_t* const from[3] = {reinterpret_cast<const int8_t*>(w0 + at), reinterpret_cast<const int8_t*>(w1 + at),
                                   reinterpret_cast<const int8_t*>(tok + at)};
    const bool in[3] = {in0, in1, tin};
#pragma unroll
    for (int i = 0; i < 6; ++i)
      ask[i].ask(from[i / 2] + i % 2 * 64, 0, in[i / 2] && left > i % 2 * 64, i < 4 ? w_at : t_at, i < 4 ? p.w_end : p.t_end);
    const float sw0 = __ldg(s0 + kb * p.ws_k), sw1 = __ldg(s1 + kb * p.ws_k);
    const float t0 = q * 2 < p.M ? __ldg(st0 + kb * p.ts_k) : 0.0f, t1 = q * 2 + 1 < p.M ? __ldg(st1 + kb * p.ts_k) : 0.0f;
    uint4 v[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int rest = left - i % 2 * 64;
      v[i] = ask[i].get(from[i / 2] + i % 2 * 64, 0, rest < 16 ? rest : 16, in[i / 2] && rest > 0, i < 4 ? w_at : t_at, i < 4 ? p.w_end : p.t_end);
    }
    const uint4 &a0 = v[0], &a1 = v[1], &c0 = v[2], &c1 = v[3], &b0 = v[4], &b1 = v[5];
    float d[4] = {};
    mma_fp8<FW, FT>(d, a0.x, c0.x, a0.y, c0.y, b0.x, b0.y);
    mma_fp8<FW, FT>(d, a0.z, c0.z, a0.w, c0.w, b0.z, b0.w);
    mma_fp8<FW, FT>(d, a1.x, c1.x, a1.y, c1.y, b1.x, b1.y);
    mma_fp8<FW, FT>(d, a1.z, c1.z, a1.w, c1.w, b1.z, b1.w);
    acc[0] = fmaf(d[0], sw0 * t0, acc[0]);               // rows g and g + 8 by tokens 2 q and 2 q + 1
    acc[1] = fmaf(d[1], sw0 * t1, acc[1]);
    acc[2] = fmaf(d[2], sw1 * t0, acc[2]);
    acc[3] = fmaf(d[3], sw1 * t1, acc[3]);
  }
  sums[warp][q * 2][g] = acc[0];
  sums[warp][q * 2 + 1][g] = acc[1];
  sums[warp][q * 2][g + 8] = acc[2];
  sums[warp][q * 2 + 1][g + 8] = acc[3];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (int)p.M; i += 256) {
    const int r = i % rows, token = i / rows;
    float v = 0.0f;
    for (int s = 0; s < p.share; ++s) v += sums[r / 16 * p.share + s][token][r % 16];
    if (n0 + r < p.N) put(p.out, p.out_type, token * p.N + n0 + r, v);
  }
}

}  // namespace emu_ops
