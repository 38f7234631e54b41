// ops_block_mm.cu -- FP8 products with a scale for each block of 128 of K, dense, by expert over
// ragged groups of rows, and the experts' weights' gradients (declared in include/emu_fp8.h):
//   out[m, n] = sum over blocks kb of (sum over k in kb of a[m, k] b[n, k]) * (sa[m, kb] * sb[n, kb])
#include "ops_block.cuh"

#include <cuda.h>             // CUtensorMap (the type only; the driver is called through an entry point)
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

namespace emu_ops {

// 1 once a bounded wait of the pipeline gave up (the outputs of that call are not valid)
__device__ int g_block_status = 0;

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // ops_int8.cu

}  // namespace emu_ops

#include "ops_block_few.cuh"
#include "ops_block_tc.cuh"

namespace emu_ops {

struct BlockMm {
  emu_block_operand_t a, b;                              // M and N rows
  BlockKind kind;
  int64_t M, N, K;                                       // grouped: M tokens; wgrad: K tokens
  const int32_t* offsets; int E;
  bool zero_rest;
  void* out; int out_type;                               // [M, N], wgrad [E, M, N]
};

// An operand's codes as `outer` vectors of `inner` contiguous codes, `stride` apart, in groups.
struct CodesView {
  const uint8_t* at;
  int64_t inner, outer, stride, groups, group_stride;
  bool mn;                                               // the contiguous codes are those of a K position
  bool fits() const {                                    // what a tensor map asks for
    return aligned(at, 16) && (outer <= 1 || stride % 16 == 0) && (groups <= 1 || group_stride % 16 == 0);
  }
  size_t laid_out() const { return fits() ? 0 : ((size_t)groups * (size_t)outer * (size_t)((inner + 15) / 16 * 16) + 255) / 256 * 256; }
};
CodesView view_of(const emu_block_operand_t& o, int64_t rows, int64_t K, int64_t groups, bool mn) {
  const bool by_k = !mn && (o.k_stride == 1 || K == 1) && (rows <= 1 || o.row_stride >= K);
  const uint8_t* at = static_cast<const uint8_t*>(o.codes);
  if (by_k) return {at, K, rows, o.row_stride, groups, o.group_stride, false};
  return {at, rows, K, o.k_stride, groups, o.group_stride, true};
}

// Codes to rows whose length is a multiple of 16 (zeros behind their ends), for operands that a tensor map does
// not take.  A thread takes 16 codes.
struct LayOut {
  const uint8_t* from; uintptr_t end;
  int64_t inner, outer, stride, group_stride, vectors;   // vectors: of all groups
  uint8_t* to; int64_t chunks;                           // 16 codes each, of a vector
};
__global__ void __launch_bounds__(256) lay_out_kernel(const LayOut a, const LayOut b) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product waits for this kernel's end
  const int64_t na = a.vectors * a.chunks, total = na + b.vectors * b.chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const LayOut& s = i < na ? a : b;
    const int64_t j = i < na ? i : i - na, v = j / s.chunks, k = (j - v * s.chunks) * 16, g = v / s.outer;
    const int8_t* const row = reinterpret_cast<const int8_t*>(s.from + g * s.group_stride + (v - g * s.outer) * s.stride) + k;
    const int left = s.inner - k < 16 ? (int)(s.inner - k) : 16;
    Codes<false> codes;
    codes.ask(row, 0, true, reinterpret_cast<const int8_t*>(s.from), s.end);
    *reinterpret_cast<uint4*>(s.to + v * s.chunks * 16 + k) = codes.get(row, 0, left, true, reinterpret_cast<const int8_t*>(s.from), s.end);
  }
}
LayOut lay_out_of(CodesView& v, unsigned char*& ws) {
  LayOut l = {};
  if (v.fits()) return l;
  const int64_t chunks = (v.inner + 15) / 16;
  const int64_t span = (v.groups - 1) * v.group_stride + (v.outer - 1) * v.stride + v.inner;
  l = {v.at, reinterpret_cast<uintptr_t>(v.at) + (size_t)span, v.inner, v.outer, v.stride, v.group_stride, v.groups * v.outer, ws, chunks};
  const size_t bytes = v.laid_out();
  v.at = ws;
  v.stride = chunks * 16;
  v.group_stride = v.outer * v.stride;
  ws += bytes;
  return l;
}

// boxes of 128 contiguous codes by `box` vectors under the 128-byte swizzle
int codes_map(CUtensorMap* map, const CodesView& v, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t stride = v.outer > 1 ? (cuuint64_t)v.stride : (cuuint64_t)((v.inner + 15) / 16 * 16);
  const cuuint64_t group = v.groups > 1 ? (cuuint64_t)v.group_stride : stride * (cuuint64_t)v.outer;
  const cuuint64_t dims[3] = {(cuuint64_t)v.inner, (cuuint64_t)v.outer, (cuuint64_t)v.groups}, strides[2] = {stride, group};
  const cuuint32_t boxes[3] = {128u, (cuuint32_t)box, 1u}, step[3] = {1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(v.at), dims, strides, boxes, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EMU_OK : emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// the output [groups, rows, cols], boxes of 128 bytes by 32 rows
int out_map(CUtensorMap* map, void* out, int type, int64_t rows, int64_t cols, int64_t groups) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t es = elem_bytes((emu_out_t)type);
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)groups}, strides[2] = {cols * es, cols * es * (cuuint64_t)rows};
  const cuuint32_t boxes[3] = {(cuuint32_t)(128 / es), 32u, 1u}, step[3] = {1u, 1u, 1u};
  const CUtensorMapDataType t = type == EMU_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : type == EMU_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = enc(map, t, 3, out, dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EMU_OK : emu_ops_fail(EMU_ECUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

BlockSide side_of(const emu_block_operand_t& o, int64_t rows, bool mn) {
  return {o.scale, o.scale_rows == 1 ? 0 : 7, o.scale_row_stride, o.scale_k_stride, o.scale_group_stride, (int)rows, mn ? 1 : 0};
}

// Clusters of so many CTAs (1 to 8) that the device holds at once, each CTA with an SM to itself.  The SMs of a cluster share a part of
// the chip, whose number need not be a multiple of it: of 152 SMs 76 clusters of two, but 36 of four and 15 of eight.
int clusters_at_once(int ctas) {
  static std::atomic<int> cached[64][9];
  static std::atomic<bool> done[64];
  const int sms = emu_ops_sm_count();
  int dev = 0;
  if (ctas == 1 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms / ctas;
  int v = cached[dev][ctas].load(std::memory_order_relaxed);
  if (v == 0) {
    const void* const kernel = reinterpret_cast<const void*>(block_tc_kernel<256, kScaleLane>);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kTcThreads8);
    cfg.dynamicSmemBytes = BlockTcShape<256>::smem(kMaxExperts);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    v = emu_ops_allow_smem(kernel, (int)cfg.dynamicSmemBytes, done) && cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0
            ? n : sms / ctas;
    cached[dev][ctas].store(v, std::memory_order_relaxed);
  }
  return v;
}

// `early`: launched while its operands are still laid out (it waits for them itself)
template <int BN> int launch_tc(const BlockTcParams& p, int mode, int64_t tiles, const CUtensorMap (&maps)[3], bool early, cudaStream_t st) {
  using SH = BlockTcShape<BN>;
  auto kernel = mode == kScaleLane ? block_tc_kernel<BN, kScaleLane> : mode == kScaleColumns ? block_tc_kernel<BN, kScaleColumns>
                                                                                              : block_tc_kernel<BN, kScaleBoth>;
  static std::atomic<bool> done[3][64];
  if (!emu_ops_allow_smem(reinterpret_cast<const void*>(kernel), SH::smem(kMaxExperts), done[mode])) return emu_ops_launched("cudaFuncSetAttribute");
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTcThreads8);
  cfg.dynamicSmemBytes = SH::smem(p.kind == BlockKind::dense ? 0 : p.E);
  cfg.stream = st;
  const int cluster = (SH::PAIR ? 2 : 1) * p.slices;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = cluster > 1 ? at : at + 1;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  const int64_t room = clusters_at_once(SH::PAIR ? 2 : 1);
  cfg.gridDim = dim3((unsigned)(p.slices > 1 || tiles < room ? tiles : room) * cluster);
  if (early) ++cfg.numAttrs;
  if (cudaLaunchKernelEx(&cfg, kernel, p, maps[0], maps[1], maps[2]) != cudaSuccess) return emu_ops_launched("emu_block_scaled_mm");
  return EMU_OK;
}

// Up to eight tokens of a dense product, K-major on both sides, where latency counts; where bandwidth does, the TMA's
// deep queues win, and where a long K does, the slices: eight warps share K's blocks, 0.58 us a round (unaligned 1.5).  In us, so
// and by tcgen05: 1 x 5760 x 1920 4.2 and 7.4, 8 x 4096 x 4096 5.3 and 7.7, 8 x 4096 x 6144 7.4 and 9.0, 8 x 16384 x 2048 11.5 and 8.8;
// 8 x 1024 x 8192 7.2 and 6.7, 1 x 2048 x 8192 7.1 and 7.8, 1 x 2304 x 10240 8.3 and 8.7, 8 x 512 x 16384 12.2 and 8.1,
// 1 x 512 x 32768 21 and 10.5; unaligned 1 x 5760 x 1921 9.7 and 12.9, 1 x 2048 x 6001 11.9 and 13.5, 8 x 512 x 8200 15.3 and
// 9.5; of 16 tokens 8.1 and 8.4.
bool few_tokens(int64_t M, int64_t N, int64_t K, const CodesView& va, const CodesView& vb) {
  return M <= 8 && K > 0 && K <= 8192 && !va.mn && !vb.mn && N * K <= (int64_t)24 << 20;
}
void run_few_tokens(const BlockMm& p, const CodesView& va, const CodesView& vb, cudaStream_t st) {
  BlockFewParams q = {};
  const uintptr_t w = reinterpret_cast<uintptr_t>(vb.at), t = reinterpret_cast<uintptr_t>(va.at);
  q.w = vb.at; q.w_row = vb.stride; q.w_end = w + (size_t)((p.N - 1) * vb.stride + p.K);
  q.ws = p.b.scale; q.ws_shift = p.b.scale_rows == 1 ? 0 : 7; q.ws_row = p.b.scale_row_stride; q.ws_k = p.b.scale_k_stride;
  q.t = va.at; q.t_row = va.stride; q.t_end = t + (size_t)((p.M - 1) * va.stride + p.K);
  q.ts = p.a.scale; q.ts_shift = p.a.scale_rows == 1 ? 0 : 7; q.ts_row = p.a.scale_row_stride; q.ts_k = p.a.scale_k_stride;
  q.M = (int)p.M; q.N = p.N; q.K = (int)p.K;
  const int64_t kb = (p.K + kBlock - 1) / kBlock;
  q.share = kb >= 8 ? 8 : kb >= 4 ? 4 : kb >= 2 ? 2 : 1;
  q.out = p.out; q.out_type = p.out_type;
  auto pick = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    return p.b.format == EMU_E4M3FN
               ? p.a.format == EMU_E4M3FN ? block_few_kernel<EMU_E4M3FN, EMU_E4M3FN, VEC> : block_few_kernel<EMU_E4M3FN, EMU_E5M2, VEC>
               : p.a.format == EMU_E4M3FN ? block_few_kernel<EMU_E5M2, EMU_E4M3FN, VEC> : block_few_kernel<EMU_E5M2, EMU_E5M2, VEC>;
  };
  const bool vec = p.K % 16 == 0 && va.fits() && vb.fits();
  auto kernel = vec ? pick(std::true_type()) : pick(std::false_type());
  const int64_t rows = 16 * (8 / q.share);
  kernel<<<(unsigned)((p.N + rows - 1) / rows), 256, 0, st>>>(q);
}

int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }
// Which tiles: pairs of CTAs on 256 x 256, or 128 of the weights' rows by BN tokens, and of how many slices of K.
// Measured, in us: a call takes `base`, and each of K's blocks `first` in the first round of tiles and `next` in
// those after it (where more SMs share the memory); slices 0.9 more, of pairs 3.  As BN 32, 64 and pairs: 64 x 5760 x 1920 7.4, 8.9
// and 11.1, 128 x 5760 x 1920 11.3, 9.5 and 11.5, 256 x 4096 x 4096 17.0, 15.3 and 14.7, 512 x 5760 x 1920 24, 22 and
// 12.5; 64 x 1920 x 5760 11.3 in one slice, 8.1 in four, 777 x 1920 x 5760 in pairs 24.4 and in two slices 19.1.
struct Form { int BN, slices; bool tail; };
Form pick_form(const BlockMm& p, bool tokens_mn, int64_t rows) {
  if (p.kind == BlockKind::wgrad) return {256, 1, false};
  // by expert the tiles are not known, but the rows an expert has, about (those behind the last group count as well).  In BN 32, 64
  // and pairs: 32 experts of 5760 x 1920 with 32 rows each 60, 71 and 88 us, with 64 89, 78 and 89, with 128 167, 132 and 92; 8 of
  // 1920 x 5760 with 16 20, 21 and 27, with 64 26, 23 and 27, with 128 41, 33 and 29; 16 of 1024 x 1024 with 64 11.0, 9.6 and
  // 10.5, with 128 17.0, 15.0 and 10.9
  if (p.kind == BlockKind::grouped) return {rows <= 32 ? 32 : rows <= 64 ? 64 : 256, 1, false};
  struct Cost { int BN; double base, first, next; };
  const Cost costs[3] = {{32, 4.7, 0.16, 0.25}, {64, 5.3, 0.22, 0.38}, {256, 5.5, 0.41, 0.49}};
  const int64_t kb = up(p.K, kBlock);
  Form best = {256, 1, false};
  double least = 0.0;
  for (const Cost& c : costs) {
    const bool pair = c.BN == 256;
    if (tokens_mn && !pair) continue;                    // narrow tiles take the tokens K-major
    const int64_t tiles = up(p.N, pair ? 256 : 128) * up(p.M, c.BN), room = clusters_at_once(pair ? 2 : 1);
    for (int slices = 1; slices <= (pair ? 2 : 8); slices *= 2) {
      if (slices > 1 && (tiles > clusters_at_once((pair ? 2 : 1) * slices) || slices > kb)) break;
      const double t = c.base + (double)up(kb, slices) * (c.first + (double)(up(tiles, room) - 1) * c.next) + (slices == 1 ? 0.0 : pair ? 3.0 : 0.9);
      if (least == 0.0 || t < least) {
        least = t;
        best = {c.BN, slices, false};
      }
    }
  }
  // A last round of tiles that leaves half of the pairs without any goes in two slices, in a launch of its own, where half of
  // K's blocks take longer than a launch and the slices' exchange: 5760 x 1920 x 8192 (184 tiles for 76 pairs) 150 -> 138 us.
  const int64_t tiles = up(p.N, 256) * up(p.M, 256), pairs = clusters_at_once(2), rest = tiles % pairs;
  best.tail = best.BN == 256 && best.slices == 1 && tiles > pairs && rest > 0 && rest <= clusters_at_once(4) && kb >= 32;
  return best;
}

int run_block_mm(const BlockMm& p, void* workspace, cudaStream_t st) {
  const bool wgrad = p.kind == BlockKind::wgrad, grouped = p.kind == BlockKind::grouped;
  CodesView va = view_of(p.a, p.M, p.K, 1, wgrad), vb = view_of(p.b, p.N, p.K, grouped ? p.E : 1, wgrad);
  const int64_t rows_of_group = grouped ? (p.M + (p.E > 0 ? p.E : 1) - 1) / (p.E > 0 ? p.E : 1) : p.M;   // about
  if (p.kind == BlockKind::dense && few_tokens(p.M, p.N, p.K, va, vb)) {
    run_few_tokens(p, va, vb, st);
    return emu_ops_launched("emu_block_scaled_mm");
  }
  const bool any = p.K > 0 && !(grouped && p.E == 0);    // anything to multiply
  LayOut lay_a = {}, lay_b = {};
  if (any) {
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    lay_a = lay_out_of(va, ws);
    lay_b = lay_out_of(vb, ws);
  }
  const int64_t kb = (p.K + kBlock - 1) / kBlock;
  const int64_t groups = wgrad ? p.E : 1;
  const Form form = pick_form(p, va.mn, rows_of_group);
  const int BN = form.BN, slices = form.slices;
  const bool swap = BN < 256;
  BlockTcParams q = {};
  q.kind = p.kind;
  q.l = swap ? side_of(p.b, p.N, vb.mn) : side_of(p.a, p.M, va.mn);
  q.c = swap ? side_of(p.a, p.M, va.mn) : side_of(p.b, p.N, vb.mn);
  const emu_block_operand_t& ol = swap ? p.b : p.a;
  const emu_block_operand_t& oc = swap ? p.a : p.b;
  q.idesc = (1u << 4) | ((ol.format == EMU_E5M2 ? 1u : 0u) << 7) | ((oc.format == EMU_E5M2 ? 1u : 0u) << 10) | ((uint32_t)q.l.mn << 15) |
            ((uint32_t)q.c.mn << 16) | ((uint32_t)((swap ? BN : 128) >> 3) << 17) | ((swap ? 8u : 16u) << 24);
  const int64_t tl = up(q.l.rows, swap ? 128 : 256), tc = up(q.c.rows, BN);
  // the most tiles there can be: of ragged groups, each may add one
  const int64_t tiles = grouped ? (swap ? tl * (tc + p.E) : (tl + p.E) * tc) : tl * tc * groups;
  if (tiles * slices >= (int64_t)1 << 31) return emu_ops_fail(EMU_EUNSUPPORTED, "too many tiles");
  q.tiles_l = (int)tl;
  q.tiles_c = (int)tc;
  q.k_blocks = any ? (int)kb : 0;
  q.slices = slices;
  q.offsets = p.offsets;
  q.E = p.E;
  q.T = (int)(wgrad ? p.K : p.M);
  q.zero_rest = p.zero_rest;
  q.out = p.out;
  q.out_type = p.out_type;
  q.ldl = swap ? 1 : p.N;
  q.ldc = swap ? p.N : 1;
  q.out_group = p.M * p.N;
  CUtensorMap maps[3] = {};
  if (any) {
    int rc = codes_map(&maps[0], swap ? vb : va, 128);
    const CodesView& vc = swap ? va : vb;
    if (rc == EMU_OK) rc = codes_map(&maps[1], vc, vc.mn || BN > 128 ? 128 : BN);
    if (rc != EMU_OK) return rc;
  }
  if (!swap && aligned(p.out, 16) && p.N * (int64_t)elem_bytes((emu_out_t)p.out_type) % 16 == 0) {
    const int rc = out_map(&maps[2], p.out, p.out_type, p.M, p.N, groups);
    if (rc != EMU_OK) return rc;
    q.out_map = 1;
  }
  // a lane's scale alone, where the columns of a warp share theirs; else the lanes' in the columns' if they all share it
  const bool tokens_c = grouped && swap, tokens_l = grouped && !swap;
  const int mode = q.c.shift == 7 && !tokens_c ? kScaleLane : q.l.shift == 7 && !tokens_l ? kScaleColumns : kScaleBoth;
  const int64_t work = lay_a.vectors * lay_a.chunks + lay_b.vectors * lay_b.chunks, ctas = up(work, 256);
  if (work > 0) lay_out_kernel<<<(unsigned)(ctas < 16384 ? ctas : 16384), 256, 0, st>>>(lay_a, lay_b);
  q.from = 0;
  q.to = (int)tiles;
  if (form.tail) {
    q.to = (int)(tiles - tiles % clusters_at_once(2));
    const int rc = launch_tc<256>(q, mode, q.to, maps, work > 0, st);
    if (rc != EMU_OK) return rc;
    q.from = q.to;
    q.to = (int)tiles;
    q.slices = 2;
  }
  if (BN == 256) return launch_tc<256>(q, mode, q.to - q.from, maps, work > 0 && q.from == 0, st);
  if (BN == 64) return launch_tc<64>(q, mode, tiles, maps, work > 0, st);
  return launch_tc<32>(q, mode, tiles, maps, work > 0, st);
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
  const int64_t most = ((int64_t)1 << 31) - 256;         // so that a tile's end is a 32-bit number
  if (M >= most || N >= most || K >= most) return emu_ops_fail(EMU_EUNSUPPORTED, "sizes must be below 2^31 - 256");
  if (E > kMaxExperts) return emu_ops_fail(EMU_EUNSUPPORTED, "more than %d experts", kMaxExperts);
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

int emu_ops_block_status(int* status, bool reset) {
  const int zero = 0;
  if (cudaMemcpyFromSymbol(status, g_block_status, sizeof *status) != cudaSuccess ||
      (reset && cudaMemcpyToSymbol(g_block_status, &zero, sizeof zero) != cudaSuccess))
    return emu_ops_launched("emu_ops_device_status");
  return EMU_OK;
}

extern "C" {

size_t emu_block_mm_workspace_bytes(const emu_block_operand_t* a, const emu_block_operand_t* b, int64_t M, int64_t N, int64_t K) {
  if (!a || !b || M < 1 || N < 1 || K < 1) return 0;
  const CodesView va = view_of(*a, M, K, 1, false), vb = view_of(*b, N, K, 1, false);
  return few_tokens(M, N, K, va, vb) ? 0 : va.laid_out() + vb.laid_out();
}
size_t emu_grouped_block_mm_workspace_bytes(const emu_block_operand_t* a, const emu_block_operand_t* b, int64_t T, int64_t N, int64_t K,
                                            int64_t E) {
  if (!a || !b || T < 1 || N < 1 || K < 1 || E < 1) return 0;
  return view_of(*a, T, K, 1, false).laid_out() + view_of(*b, N, K, E, false).laid_out();
}
size_t emu_grouped_block_wgrad_workspace_bytes(const emu_block_operand_t* a, const emu_block_operand_t* b, int64_t T, int64_t N,
                                               int64_t K) {
  if (!a || !b || T < 1 || N < 1 || K < 1) return 0;
  return view_of(*a, N, T, 1, true).laid_out() + view_of(*b, K, T, 1, true).laid_out();
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
  BlockMm p = {*a, *b, BlockKind::dense, M, N, K, nullptr, 0, false, out, (int)out_dtype};
  return run_block_mm(p, workspace, static_cast<cudaStream_t>(stream));
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
  return run_block_mm(p, workspace, static_cast<cudaStream_t>(stream));
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
  return run_block_mm(p, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
