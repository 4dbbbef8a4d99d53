// linear8.h -- operands in 8 bits with a power of two for each block of 128,
// and launchers of the linear layer in 8 bits (internal).
//
// An operand of the product is a matrix of rows x depth e4m3 codes, `depth`
// being what the product sums over, with one scale for each row and 128 of
// depth.  The codes lie row by row ([rows][depth]) or depth by depth
// ([depth][rows], `mn`): the tensor cores take both, so that a tensor's codes
// are written the way that the tensor itself lies.  A scale is a power of two,
// held as its biased exponent in a byte (ue8m0).  The scales lie as the tensor
// cores take them: tiles of 512 bytes for 128 rows and four blocks of depth, row
// r's byte of block b at (r % 32) 16 + (r % 128) / 32 4 + b % 4 in tile
// [r / 128][b / 4].
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace trimul {

constexpr int L8_BLOCK = 128;        // numbers that share a scale
constexpr int L8_SCALE_TILE = 512;   // bytes
constexpr int L8_TILE = 256;         // rows and columns of a product's tile (a CTA pair)

__host__ __device__ constexpr long long l8_blocks(long long n) { return (n + L8_BLOCK - 1) / L8_BLOCK; }

// One operand in memory: codes, then scales, each from a multiple of 256 bytes on.
struct Operand8 {
  long long rows, depth;
  bool mn;
  __host__ __device__ long long ld() const { return ((mn ? rows : depth) + 15) / 16 * 16; }  // bytes from line to line
  __host__ __device__ long long groups() const { return (l8_blocks(depth) + 3) / 4; }
  __host__ __device__ size_t code_bytes() const { return static_cast<size_t>(mn ? depth : rows) * ld(); }
  __host__ __device__ size_t scale_bytes() const { return (static_cast<size_t>(l8_blocks(rows)) * groups() * L8_SCALE_TILE + 255) / 256 * 256; }
  __host__ __device__ size_t scales_at() const { return (code_bytes() + 255) / 256 * 256; }
  __host__ __device__ size_t bytes() const { return scales_at() + scale_bytes(); }
};
// Where a row's byte of a block is among the scales, `groups` of them a row of tiles.
__host__ __device__ __forceinline__ size_t l8_scale_at(long long row, long long block, long long groups) {
  return (static_cast<size_t>(row / 128) * groups + block / 4) * L8_SCALE_TILE + (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4;
}

// A launch; `early`: it may begin while the kernel before it in the stream runs, whose results it waits for by itself (after_previous).
// The kernels of a call follow one another so, which hides a launch's latency and a kernel's preparations; the first one, which
// clears the status word, comes behind all that was before the call.
template <typename... Params, typename... Args>
cudaError_t launch8(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, bool early, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = threads;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, static_cast<Params>(args)...);
}

// ---------------------------------------------------------------- rounding to 8 bits (k11_quantize8.cu)
// Each clears the word `status` for the products behind it; null: it is not a call's first kernel.
// bf16 [rows][depth], a scale for each row and 128 columns: the operand {rows, depth}.
cudaError_t launch_quantize_rows(const uint16_t* x, long long rows, int depth, uint8_t* out, int* status, int num_sms, cudaStream_t s);
// bf16 [rows][cols], a scale for each column and 128 rows: the operand {cols, rows, mn}; with by_rows (or null) also as
// launch_quantize_rows, and with column_sums (or null) the sums of the columns, f32 [cols], by way of `part`.
int quantize_columns_parts(long long rows, int cols, int num_sms);
cudaError_t launch_quantize_columns(const uint16_t* x, long long rows, int cols, uint8_t* out, uint8_t* by_rows,
                                    float* column_sums, float* part, int* status, int num_sms, cudaStream_t s);
// A weight [N][K], a scale for each 128 x 128: codes [N][K], which are the operands {N, K} and {K, N, mn}, and the scales of both.
cudaError_t launch_quantize_weight(const void* w, bool f32, int N, int K, uint8_t* codes, uint8_t* scales, uint8_t* scales_mn,
                                   cudaStream_t s);

// ---------------------------------------------------------------- products (k12_gemm8.cu)
struct Gemm8Args {
  int M, N;
  int a_mn, b_mn;        // how the operands lie
  int blocks;            // of 128 depth in all
  int chunk;             // blocks that one accumulation takes
  int per_z, n_z;        // blocks of a slice of the depth, and the slices
  int tiles_m, tiles_n;
  int run;               // tiles beside one another that a pair takes in turn
  void* c;               // bf16 [M][N], or f32 [n_z][M][N]
  const float* bias;     // f32 [N] or null (bf16 output)
  int* status;
  unsigned long long timeout_ns;
  int stall;             // test hook: nothing is loaded
};
struct Gemm8Maps {
  CUtensorMap a, b, a_scale, b_scale;
};
// The same with A as bf16 that is rounded on its way (k13_fused8.cu): by rows from t [M][depth] to bf16, or by columns from
// t [depth][M] to f32 slices.  By rows of at most FUSED8_FEW_BLOCKS blocks, C is written by way of its map `c` (boxes of 32 rows and
// 64 columns), and with g.run > 1 a run's tiles share the codes, rounded once.
constexpr int FUSED8_FEW_BLOCKS = 3;
struct Fused8Args {
  Gemm8Args g;
  long long depth;
  int clear;             // clear the status word first
  float* sums;           // by columns: [2 g.n_z][M], whose sum is that of t's columns; or null
};
struct Fused8Maps {
  CUtensorMap t, b, b_scale, c;
};
cudaError_t launch_fused8(const Fused8Args& a, const Fused8Maps& m, bool cols, int pairs, cudaStream_t s);
int gemm8_max_pairs(int num_sms);
cudaError_t launch_gemm8(const Gemm8Args& a, const Gemm8Maps& m, bool f32, int pairs, cudaStream_t s);
// The same sums without the product, bit for bit: of t [rows][cols], slices of per_z blocks of 128 rows.
cudaError_t launch_column_sums(const uint16_t* t, long long rows, int cols, int per_z, int n_z, float* sums, int* status, cudaStream_t s);
// out = the sum of n_z slices of n floats; cols > 0: of matrices [n / cols][cols], transposed.
struct Join8 {
  const float* part;
  int n_z;
  long long n;
  int cols;
  float* out;
};
// Two of them in one launch, either of them of nothing; `few`: of few sums.
cudaError_t launch_join(const Join8& a, const Join8& few, cudaStream_t s);

}  // namespace trimul
