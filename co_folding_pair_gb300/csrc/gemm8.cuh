// gemm8.cuh -- what the products in 8 bits share: the tensor cores' block-scaled
// instruction, the walk over tiles, and the epilogue's stores.
#pragma once

#include "linear8.h"
#include "pair_ops.cuh"
#include "sm103_ptx.cuh"

namespace trimul {

// Instruction descriptor of kind::mxf8f6f4: E4M3 A and B (format 0), the
// operands' majors (bits 15 and 16: 1 for depth by depth), N >> 3 at bit 17, ue8m0 scales (bit 23), M >> 4 at bit 24; the byte of B's
// and A's scale words at bits 4 and 29.
constexpr uint32_t kIdesc8 = ((L8_TILE >> 3) << 17) | (1u << 23) | ((L8_TILE >> 4) << 24);

__device__ __forceinline__ void mma_block_scaled_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                      uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}

// 32 rows of 16 bytes from shared memory to four TMEM columns, in each quadrant of lanes, in both CTAs.
__device__ __forceinline__ void copy_scales_pair(uint32_t tmem, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sdesc) : "memory");
}

// Shared-memory descriptor without swizzle: groups of eight 16-byte rows, 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(128 >> 4) << 32 | 1ull << 46;
}

// tmem_ld32 and its wait as one statement: between two, the compiler may place a use of what has not arrived yet.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 8 x 8 chunks of 16 bytes inside each group of 8 lanes: lane 8a + b holds
// chunks of its row, and afterwards chunk b of rows 8a .. 8a + 7.
__device__ __forceinline__ void transpose8(uint4 (&R)[8], uint32_t gb) {
#pragma unroll
  for (int k = 4; k >= 1; k >>= 1) {
    const bool upper = (gb & k) != 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j & k) continue;
      const uint4 lo = R[j], hi = R[j | k];
      const uint4 send = upper ? lo : hi;
      uint4 recv;
      recv.x = __shfl_xor_sync(0xffffffffu, send.x, k);
      recv.y = __shfl_xor_sync(0xffffffffu, send.y, k);
      recv.z = __shfl_xor_sync(0xffffffffu, send.z, k);
      recv.w = __shfl_xor_sync(0xffffffffu, send.w, k);
      R[j] = upper ? recv : lo;
      R[j | k] = upper ? hi : recv;
    }
  }
}

// The same for 4 x 4 chunks inside each group of 4 lanes.
__device__ __forceinline__ void transpose4(uint4 (&R)[4], uint32_t lane4) {
#pragma unroll
  for (int k = 2; k >= 1; k >>= 1) {
    const bool upper = (lane4 & k) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & k) continue;
      const uint4 lo = R[j], hi = R[j | k];
      const uint4 send = upper ? lo : hi;
      uint4 recv;
      recv.x = __shfl_xor_sync(0xffffffffu, send.x, k);
      recv.y = __shfl_xor_sync(0xffffffffu, send.y, k);
      recv.z = __shfl_xor_sync(0xffffffffu, send.z, k);
      recv.w = __shfl_xor_sync(0xffffffffu, send.w, k);
      R[j] = upper ? recv : lo;
      R[j | k] = upper ? hi : recv;
    }
  }
}

// The bias is added from shared memory: read from global memory where it is added,
// sixteen times a block of columns, the loads' latency made the epilogue twice as long
// (2^20 rows of 256 to 1024: 954 us against 463 without a bias).  A warp's 64 columns of it:
__device__ __forceinline__ void stage_bias(float* to, const float* bias, int c0, int N, int lane) {
  const int col = c0 + 2 * lane;  // N is even
  *reinterpret_cast<float2*>(to + 2 * lane) = col < N ? *reinterpret_cast<const float2*>(bias + col) : make_float2(0.f, 0.f);
}
// Adds kCount of them to a row's columns.
template <int kCount>
__device__ __forceinline__ void add_bias(uint32_t (&r)[kCount], const float* from) {
  auto two = [](uint32_t& lo, uint32_t& hi, float a, float b) {
    const float2 s = split2(add2(pair2(__uint_as_float(lo), __uint_as_float(hi)), pair2(a, b)));
    lo = __float_as_uint(s.x), hi = __float_as_uint(s.y);
  };
#pragma unroll
  for (int v = 0; v < kCount / 4; ++v) {
    const float4 b = reinterpret_cast<const float4*>(from)[v];
    two(r[4 * v], r[4 * v + 1], b.x, b.y);
    two(r[4 * v + 2], r[4 * v + 3], b.z, b.w);
  }
}

// One accumulation: blocks [b0, b1) of a tile.  A pair takes runs of p.run tiles
// beside one another, each tile with its accumulations, in turn; all warps walk them alike.
struct Walk {
  const Gemm8Args& p;
  uint32_t at, step, total;  // of runs: fewer than 2^31, for rows and columns below 2^31 and 2^16
  int runs, z, tm, tn, tn_end, b0, b1, z_end;
  __device__ __forceinline__ Walk(const Gemm8Args& a, uint32_t first, uint32_t pairs)
      : p(a), at(first), step(pairs), runs((a.tiles_n + a.run - 1) / a.run) {
    total = static_cast<uint32_t>(a.tiles_m) * runs * a.n_z;
    if (more()) begin();
  }
  __device__ __forceinline__ bool more() const { return at < total; }
  __device__ __forceinline__ void begin() {
    const uint32_t per_z = static_cast<uint32_t>(p.tiles_m) * runs;
    z = static_cast<int>(at / per_z);
    const uint32_t rem = at - z * per_z;
    tm = static_cast<int>(rem / runs), tn = static_cast<int>(rem - tm * runs) * p.run;
    tn_end = min(tn + p.run, p.tiles_n);
    z_end = min((z + 1) * p.per_z, p.blocks);
    begin_tile();
  }
  __device__ __forceinline__ void begin_tile() {
    b0 = z * p.per_z;
    b1 = min(b0 + p.chunk, z_end);
  }
  __device__ __forceinline__ bool first() const { return b0 == z * p.per_z; }
  __device__ __forceinline__ bool last() const { return b1 == z_end; }
  __device__ __forceinline__ bool last_tile() const { return tn + 1 == tn_end; }
  __device__ __forceinline__ void next() {
    if (!last()) {
      b0 = b1;
      b1 = min(b0 + p.chunk, z_end);
    } else if (!last_tile()) {
      ++tn;
      begin_tile();
    } else {
      next_run();
    }
  }
  __device__ __forceinline__ void next_run() {
    at += step;
    if (more()) begin();
  }
};
}  // namespace trimul
