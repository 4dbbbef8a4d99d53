// linear8_api.cu -- the C ABI's entry points of the linear layer in 8 bits
// (include/trimul.h): argument checks, tensor maps, and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "trimul.h"
#include "api_checks.h"
#include "api_status.h"
#include "linear8.h"

using namespace trimul;

namespace {

constexpr int kMostWidth = 65536;
constexpr int kMostPairs = 128, kMostSms = 256;  // what workspaces are sized for
constexpr int kChunk = 32;                       // blocks of 128 rows that a weight gradient's accumulation takes
// 256-wide tiles of the other operand up to which rounding on the way (k13_fused8.cu) is faster than a pass of its own: each tile
// rounds again.  us: by rows 2^20 of 1024 to 256 channels (one tile) 415 to 794, 2^19 of 512 to 512 (two) 236 to 282, 2^18 of 1024 to 768
// (three) 311 to 303; by columns 2^20 of 1024 to 256 579 to 929, 2^19 of 512 to 512 358 to 398, 2^18 of 1024 to 1024 (four) 588 to 488.
constexpr int kFusedRows = 2, kFusedColumns = 2;
constexpr unsigned long long kTimeoutNs = 4000000000ull, kStallTimeoutNs = 200000000ull;
constexpr size_t kStatusBytes = 256;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

// Two-dimensional maps: codes (boxes of 128 rows x 128 of depth, zeros past the
// operand's) and scales (boxes of one tile).
trimul_status operand_maps(CUtensorMap* codes, CUtensorMap* scales, const Operand8& o, const uint8_t* at, const uint8_t* scales_at) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return fail(TRIMUL_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t one[2] = {1, 1};
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(o.mn ? o.rows : o.depth), static_cast<cuuint64_t>(o.mn ? o.depth : o.rows)}, stride[1] = {static_cast<cuuint64_t>(o.ld())};
  const cuuint32_t box[2] = {L8_BLOCK, 128};
  CUresult r = fn(codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(at), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) {
    const cuuint64_t sdim[2] = {L8_SCALE_TILE / 4, static_cast<cuuint64_t>(l8_blocks(o.rows) * o.groups())}, sstride[1] = {L8_SCALE_TILE};
    const cuuint32_t sbox[2] = {L8_SCALE_TILE / 4, 1};
    r = fn(scales, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<uint8_t*>(scales_at), sdim, sstride, sbox, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (r != CUDA_SUCCESS) return fail(TRIMUL_ERR_CUDA, "tensor map of an 8-bit operand rejected (CUresult %d)", static_cast<int>(r));
  return TRIMUL_OK;
}

// bf16 [rows][cols] in boxes of `box_rows` rows and 64 columns; past the end zeros are read and nothing is written.
trimul_status bf16_map(CUtensorMap* m, const uint16_t* at, long long cols, long long rows, unsigned box_rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return fail(TRIMUL_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t one[2] = {1, 1}, box[2] = {64, box_rows};
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)}, stride[1] = {static_cast<cuuint64_t>(cols) * 2};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(at), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TRIMUL_ERR_CUDA, "tensor map of a bf16 operand rejected (CUresult %d)", static_cast<int>(r));
  return TRIMUL_OK;
}

// CTA pairs that are resident at once; asked for once a device (the current one).
int pairs_of(int device, int sms) {
  static std::atomic<int> known[64];
  int n = device < 64 ? known[device].load() : 0;
  if (n == 0) {
    n = std::min(kMostPairs, gemm8_max_pairs(sms));
    if (device < 64) known[device].store(n);
  }
  return n;
}

int tiles_of(int n) { return (n + L8_TILE - 1) / L8_TILE; }

// Slices of `blocks` of depth for M x N outputs: one tile a pair, each a multiple of four blocks (a group of scales).  None
// where there are no blocks (the workspace of no rows is asked for too).
void slices(int M, int N, int blocks, int pairs, int* per_z, int* n_z) {
  const int tiles = tiles_of(M) * tiles_of(N), want = std::max(1, std::min((blocks + 3) / 4, pairs / tiles));
  *per_z = std::max(4, ((blocks + want - 1) / want + 3) / 4 * 4);
  *n_z = (blocks + *per_z - 1) / *per_z;
}

// An operand and where its codes and scales are.
struct Placed8 {
  Operand8 o;
  const uint8_t *codes, *scales;
  Placed8(const Operand8& op, const uint8_t* at) : o(op), codes(at), scales(at + op.scales_at()) {}
  Placed8(const Operand8& op, const uint8_t* at, const uint8_t* scales_at) : o(op), codes(at), scales(scales_at) {}
};

trimul_status run_gemm(const Placed8& a, const Placed8& b, void* c, bool f32, const float* bias, int per_z, int n_z, int* status,
                       int pairs, cudaStream_t s, unsigned flags) {
  Gemm8Args p{};
  p.M = static_cast<int>(a.o.rows), p.N = static_cast<int>(b.o.rows);
  p.a_mn = a.o.mn, p.b_mn = b.o.mn;
  p.blocks = static_cast<int>(l8_blocks(a.o.depth));
  p.per_z = per_z ? per_z : p.blocks;
  p.n_z = n_z;
  p.chunk = f32 ? kChunk : p.per_z;
  p.tiles_m = tiles_of(p.M), p.tiles_n = tiles_of(p.N);
  p.run = 1;
  p.c = c, p.bias = bias, p.status = status;
  p.timeout_ns = flags & TRIMUL_FLAG_INJECT_STALL ? kStallTimeoutNs : kTimeoutNs;
  p.stall = flags & TRIMUL_FLAG_INJECT_STALL;
  Gemm8Maps m;
  TRY(operand_maps(&m.a, &m.a_scale, a.o, a.codes, a.scales));
  TRY(operand_maps(&m.b, &m.b_scale, b.o, b.codes, b.scales));
  TRY_CUDA(launch_gemm8(p, m, f32, pairs, s), "8-bit product launch");
  return TRIMUL_OK;
}

// Whether a row of tiles can share its codes in a fused product by rows: they fit, and there are rows enough for all pairs.
bool runs_of_tiles(long long M, int blocks, int pairs) { return blocks <= FUSED8_FEW_BLOCKS && M >= 2ll * L8_TILE * pairs; }
// Whether a product by rows rounds on its way (asked for without a device too, for the workspaces: kMostPairs there, at least as many as any has).
bool fused_rows(long long M, int N, int depth) {
  return tiles_of(N) <= kFusedRows || runs_of_tiles(M, static_cast<int>(l8_blocks(depth)), kMostPairs);
}

// C = Q(t) b^T with t, bf16, rounded on its way: by rows (t [M][depth], bf16 C) or by columns (t [depth][M], f32 slices).
trimul_status run_fused(const uint16_t* from, long long M, long long depth, bool cols, const Placed8& b, void* c, const float* bias,
                        float* sums, int per_z, int n_z, int* status, bool clear, int pairs, cudaStream_t s, unsigned flags) {
  Fused8Args p{};
  p.clear = clear;
  p.sums = sums;
  p.depth = depth;
  p.g.M = static_cast<int>(M), p.g.N = static_cast<int>(b.o.rows);
  p.g.b_mn = b.o.mn;
  p.g.blocks = static_cast<int>(l8_blocks(depth));
  p.g.per_z = per_z ? per_z : p.g.blocks;
  p.g.n_z = n_z;
  p.g.chunk = cols ? kChunk : p.g.per_z;
  p.g.tiles_m = tiles_of(p.g.M), p.g.tiles_n = tiles_of(p.g.N);
  p.g.run = !cols && runs_of_tiles(p.g.M, p.g.blocks, pairs) ? p.g.tiles_n : 1;
  p.g.c = c, p.g.bias = bias, p.g.status = status;
  p.g.timeout_ns = flags & TRIMUL_FLAG_INJECT_STALL ? kStallTimeoutNs : kTimeoutNs;
  p.g.stall = flags & TRIMUL_FLAG_INJECT_STALL;
  Fused8Maps m;
  TRY(bf16_map(&m.t, from, cols ? M : depth, cols ? depth : M, 128));
  TRY(operand_maps(&m.b, &m.b_scale, b.o, b.codes, b.scales));
  if (cols)
    m.c = m.t;  // not used
  else
    TRY(bf16_map(&m.c, static_cast<const uint16_t*>(c), b.o.rows, M, 32));
  TRY_CUDA(launch_fused8(p, m, cols, pairs, s), "8-bit product launch");
  return TRIMUL_OK;
}

trimul_status finish8(const int* status, cudaStream_t s, unsigned flags) {
  if (!(flags & TRIMUL_FLAG_CHECK)) return TRIMUL_OK;
  TRY_CUDA(cudaStreamSynchronize(s), "stream synchronize");
  int word = 0;
  TRY_CUDA(cudaMemcpy(&word, status, sizeof(word), cudaMemcpyDeviceToHost), "status read");
  if (word != 0) return fail(TRIMUL_ERR_TIMEOUT, "a kernel gave up on a bounded wait (site 0x%x)", word);
  return TRIMUL_OK;
}

trimul_status check_widths(int N, int K) {
  for (int w : {N, K})
    if (w < 8 || w > kMostWidth || w % 8 != 0)
      return fail(TRIMUL_ERR_SHAPE, "N (%d) and K (%d) must be multiples of 8 in [8, %d]", N, K, kMostWidth);
  return TRIMUL_OK;
}

trimul_status check_rows(int64_t rows) {
  if (rows < 0 || rows >= INT32_MAX - 255) return fail(TRIMUL_ERR_SHAPE, "rows (%lld) must be in [0, 2^31 - 256)", static_cast<long long>(rows));
  return TRIMUL_OK;
}

// A packed weight: codes [N][K], the scales of the operand {N, K}, then those of {K, N}.
struct Packed {
  Operand8 w, wt;
  size_t wt_scales_at, bytes;
  Packed(int N, int K) : w{N, K, false}, wt{K, N, true}, wt_scales_at(w.bytes()), bytes(wt_scales_at + wt.scale_bytes()) {}
};

// How a backward goes about it, and the offsets in its workspace.
struct Backward8 {
  bool dx_fused, dw_fused, dw_swapped;  // dw_swapped: x is A, and the slices are of dW^T
  bool sums_alone;  // dbias does not come from the pass over dy that rounds it by columns, as there is none
  Operand8 dy_rows, dy_cols, x_cols;
  size_t dy_rows_at, dy_cols_at, x_cols_at, slices_at, sums_at, bytes;
  Backward8(int64_t rows, int N, int K) : dy_rows{rows, N, false}, dy_cols{N, rows, true}, x_cols{K, rows, true} {
    dx_fused = fused_rows(rows, K, N);
    // the wider one is rounded on its way
    dw_swapped = K >= N;
    dw_fused = tiles_of(dw_swapped ? N : K) <= kFusedColumns;
    if (!dw_fused) dw_swapped = false;
    sums_alone = dw_fused && !dw_swapped;
    int per_z, n_z;
    slices(N, K, static_cast<int>(l8_blocks(rows)), kMostPairs, &per_z, &n_z);
    dy_rows_at = kStatusBytes;
    dy_cols_at = dy_rows_at + (dx_fused ? 0 : dy_rows.bytes());
    x_cols_at = dy_cols_at + (dw_fused && !dw_swapped ? 0 : dy_cols.bytes());
    slices_at = x_cols_at + (dw_fused && dw_swapped ? 0 : x_cols.bytes());
    // (as many slices as kMostPairs allow, whatever rounding makes of fewer)
    const int most_z = std::max(n_z, kMostPairs / (tiles_of(N) * tiles_of(K)));
    sums_at = slices_at + (most_z == 1 && !dw_swapped ? 0 : up256(static_cast<size_t>(most_z) * N * K * 4));  // (one slice is dW itself)
    bytes = sums_at + up256(static_cast<size_t>(sums_alone ? 2 * most_z : quantize_columns_parts(rows, N, kMostSms)) * N * 4);
  }
};

}  // namespace

extern "C" {

size_t trimul_linear8_packed_bytes(int N, int K) { return check_widths(N, K) == TRIMUL_OK ? Packed(N, K).bytes : 0; }

trimul_status trimul_linear8_pack(const void* W, trimul_dtype type, int N, int K, void* packed, size_t packed_bytes, int device,
                                  void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK));
  TRY(check_widths(N, K));
  if (type != TRIMUL_BF16 && type != TRIMUL_F32) return fail(TRIMUL_ERR_INVALID_ARG, "type must be BF16 or F32");
  if (!W || !aligned(W, type_bytes(type))) return fail(TRIMUL_ERR_INVALID_ARG, "W is null or not aligned to its type");
  const Packed l(N, K);
  if (!packed || packed_bytes < l.bytes)
    return fail(TRIMUL_ERR_INVALID_ARG, "packed holds %zu bytes, %zu are needed", packed ? packed_bytes : 0, l.bytes);
  if (!aligned(packed, 256)) return fail(TRIMUL_ERR_INVALID_ARG, "packed must be 256-byte aligned");
  if (overlap(W, static_cast<size_t>(N) * K * type_bytes(type), packed, l.bytes)) return fail(TRIMUL_ERR_INVALID_ARG, "packed overlaps W");
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* const to = static_cast<uint8_t*>(packed);
  return finish(launch_quantize_weight(W, type == TRIMUL_F32, N, K, to, to + l.w.scales_at(), to + l.wt_scales_at, s), s, flags, "weight quantisation launch");
}

size_t trimul_linear8_forward_workspace_bytes(int64_t rows, int N, int K) {
  if (check_widths(N, K) != TRIMUL_OK || check_rows(rows) != TRIMUL_OK) return 0;
  return kStatusBytes + (fused_rows(rows, N, K) ? 0 : Operand8{rows, K, false}.bytes());
}

trimul_status trimul_linear8_forward(const void* packed, const float* bias, const uint16_t* x, int64_t rows, int N, int K,
                                     uint16_t* y, void* workspace, size_t workspace_bytes, int device, void* stream,
                                     unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK | TRIMUL_FLAG_INJECT_STALL));
  TRY(check_widths(N, K));
  TRY(check_rows(rows));
  if (!packed || !aligned(packed, 256)) return fail(TRIMUL_ERR_INVALID_ARG, "packed is null or not 256-byte aligned");
  if (!aligned(bias, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "bias must be 16-byte aligned");
  if (rows == 0) return TRIMUL_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "x or y is null or not 16-byte aligned");
  const size_t need = trimul_linear8_forward_workspace_bytes(rows, N, K);
  TRY(check_workspace(workspace, workspace_bytes, need, 256));
  const Packed l(N, K);
  const size_t xb = static_cast<size_t>(rows) * K * 2, yb = static_cast<size_t>(rows) * N * 2;
  const Buffer in[] = {{nullptr, 0, ""}, {x, xb, "x"}, {packed, l.bytes, "packed"}, {bias, static_cast<size_t>(N) * 4, "bias"}};
  const Buffer to[] = {{y, yb, "y"}, {workspace, need, "workspace"}};
  TRY(check_apart(in, 4, to, 2));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int* const status = static_cast<int*>(workspace);
  const Placed8 w(l.w, static_cast<const uint8_t*>(packed));
  const int pairs = pairs_of(device, sms);
  if (fused_rows(rows, N, K)) {
    TRY(run_fused(x, rows, K, false, w, y, bias, nullptr, 0, 1, status, true, pairs, s, flags));
  } else {
    uint8_t* const codes = static_cast<uint8_t*>(workspace) + kStatusBytes;
    TRY_CUDA(launch_quantize_rows(x, rows, K, codes, status, sms, s), "quantisation launch");
    TRY(run_gemm(Placed8(Operand8{rows, K, false}, codes), w, y, false, bias, 0, 1, status, pairs, s, flags));
  }
  return finish8(status, s, flags);
}

size_t trimul_linear8_backward_workspace_bytes(int64_t rows, int N, int K) {
  if (check_widths(N, K) != TRIMUL_OK || check_rows(rows) != TRIMUL_OK) return 0;
  return Backward8(rows, N, K).bytes;
}

trimul_status trimul_linear8_backward(const void* packed, const uint16_t* x, const uint16_t* dy, int64_t rows, int N, int K,
                                      uint16_t* dx, float* dW, float* dbias, void* workspace, size_t workspace_bytes, int device,
                                      void* stream, unsigned flags) {
  TRY(check_flags(flags, TRIMUL_FLAG_CHECK | TRIMUL_FLAG_INJECT_STALL));
  TRY(check_widths(N, K));
  TRY(check_rows(rows));
  if (!packed || !aligned(packed, 256)) return fail(TRIMUL_ERR_INVALID_ARG, "packed is null or not 256-byte aligned");
  if (!aligned(dW, 16) || !aligned(dbias, 16)) return fail(TRIMUL_ERR_INVALID_ARG, "dW and dbias must be 16-byte aligned");
  const size_t wb = static_cast<size_t>(N) * K * 4, bb = static_cast<size_t>(N) * 4;
  const size_t need = trimul_linear8_backward_workspace_bytes(rows, N, K);
  if (rows > 0) {
    if (!x || !dy || !aligned(x, 16) || !aligned(dy, 16) || !aligned(dx, 16))
      return fail(TRIMUL_ERR_INVALID_ARG, "x or dy is null, or x, dy or dx not 16-byte aligned");
    TRY(check_workspace(workspace, workspace_bytes, need, 256));
  }
  const Packed l(N, K);
  const size_t xb = static_cast<size_t>(rows) * K * 2, yb = static_cast<size_t>(rows) * N * 2;
  const Buffer in[] = {{nullptr, 0, ""}, {x, xb, "x"}, {dy, yb, "dy"}, {packed, l.bytes, "packed"}};
  const Buffer to[] = {{dx, xb, "dx"}, {dW, wb, "dW"}, {dbias, bb, "dbias"}, {workspace, rows > 0 ? need : 0, "workspace"}};
  TRY(check_apart(in, 4, to, 4));
  int sms = 0;
  TRY(device_sms(device, &sms));
  DeviceScope scope;
  TRY(scope.enter(device));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dW) TRY_CUDA(cudaMemsetAsync(dW, 0, wb, s), "dW");
    if (dbias) TRY_CUDA(cudaMemsetAsync(dbias, 0, bb, s), "dbias");
    return finish(cudaSuccess, s, flags, "linear8 backward");
  }
  const Backward8 b(rows, N, K);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  int* const status = static_cast<int*>(workspace);
  const uint8_t* const pk = static_cast<const uint8_t*>(packed);
  const int pairs = pairs_of(device, sms);
  const Placed8 w(l.wt, pk, pk + l.wt_scales_at), dy_rows(b.dy_rows, ws + b.dy_rows_at), dy_cols(b.dy_cols, ws + b.dy_cols_at),
      x_cols(b.x_cols, ws + b.x_cols_at);
  const bool codes_of_dy = (dbias || dW) && !b.sums_alone;  // by columns
  float* const sums = reinterpret_cast<float*>(ws + b.sums_at);
  uint8_t* const rows_of_dy = dx && !b.dx_fused ? ws + b.dy_rows_at : nullptr;
  if (codes_of_dy)
    TRY_CUDA(launch_quantize_columns(dy, rows, N, ws + b.dy_cols_at, rows_of_dy, dbias, sums, status, sms, s),
             "quantisation launch");
  else if (rows_of_dy)
    TRY_CUDA(launch_quantize_rows(dy, rows, N, rows_of_dy, status, sms, s), "quantisation launch");
  if (dx) {
    if (b.dx_fused)
      TRY(run_fused(dy, rows, N, false, w, dx, nullptr, nullptr, 0, 1, status, !codes_of_dy, pairs, s, flags));
    else
      TRY(run_gemm(dy_rows, w, dx, false, nullptr, 0, 1, status, pairs, s, flags));
  }
  int per_z, n_z;
  slices(N, K, static_cast<int>(l8_blocks(rows)), pairs, &per_z, &n_z);
  const Join8 of_sums = dbias && b.sums_alone ? Join8{sums, 2 * n_z, N, 0, dbias} : Join8{};
  Join8 of_dw{};
  if (dW) {
    float* const part = n_z == 1 && !b.dw_swapped ? dW : reinterpret_cast<float*>(ws + b.slices_at);
    if (part != dW) of_dw = Join8{part, n_z, static_cast<long long>(N) * K, b.dw_swapped ? N : 0, dW};
    if (!b.dw_swapped)
      TRY_CUDA(launch_quantize_columns(x, rows, K, ws + b.x_cols_at, nullptr, nullptr, nullptr, dx || codes_of_dy ? nullptr : status, sms, s),
               "quantisation launch");
    if (!b.dw_fused)
      TRY(run_gemm(dy_cols, x_cols, part, true, nullptr, per_z, n_z, status, pairs, s, flags));
    else if (b.dw_swapped)
      TRY(run_fused(x, K, rows, true, dy_cols, part, nullptr, nullptr, per_z, n_z, status, false, pairs, s, flags));
    else
      TRY(run_fused(dy, N, rows, true, x_cols, part, nullptr, of_sums.out ? sums : nullptr, per_z, n_z, status, false, pairs, s, flags));
  } else if (of_sums.out) {
    TRY_CUDA(launch_column_sums(dy, rows, N, per_z, n_z, sums, dx ? nullptr : status, s), "column sum launch");
  }
  if (of_dw.out || of_sums.out) TRY_CUDA(launch_join(of_dw, of_sums, s), "join launch");
  if (!dx && !dW && !dbias) return finish(cudaSuccess, s, flags, "linear8 backward");
  return finish8(status, s, flags);
}

}  // extern "C"
