// k12_gemm8.cu -- the product of two operands in 8 bits (linear8.h) on the
// tensor cores, which apply the blocks' scales themselves.
//
//   C[m][n] = sum over blocks b of 2^(ea[m][b] + eb[n][b]) sum over k in b of A[m][k] B[n][k]
//
// tcgen05.mma.kind::mxf8f6f4.block_scale takes a power of two for each row and
// 32 of the depth from TMEM.  A block of 128 is four such instructions with
// the same scale: a 512-byte tile of scales (128 rows, four blocks) is copied
// to four TMEM columns (tcgen05.cp), each row's four bytes in one word, and
// the instruction descriptor names the byte.  So the scales cost no arithmetic
// and the accumulation is one, in fp32, without promotions.
//
// Tile and pipeline: a CTA pair computes 256 x 256 with cta_group::2 (M = 256,
// N = 256, K = 32); each CTA stages its own 128 rows of A and 128 of B, a block
// of 128 deep, through a ring of six stages; a stage that begins a group of
// four blocks brings the group's scales as well: those of the CTA's own rows
// of A, and those of all 256 rows of B, which both CTAs' multiplications take.
//
// TMEM: two accumulators of 256 columns and the scales do not fit 512, so the
// accumulators overlap: columns 0..255 and 192..447; the scales have 448..495,
// three sets of 16 (4 for A, 8 for B) in turn.  When a set is written again its
// readers are done: two groups lie between, and if both belong to its own or
// the next accumulation one of them is whole, so that the block being staged is
// at least six behind, the ring's depth; else the accumulation two before this
// one is among them, which the epilogue has read by then.  The epilogue reads
// the 64 columns that overlap first, and the next tile's multiplications begin
// as soon as it has.
//
// Epilogue: 16 warps, one for 32 rows and 64 columns.  bf16 output (with the
// bias) as it is; fp32 output (weight gradients, summed over as many as
// millions of rows): an accumulation takes `chunk` blocks, and the warps add
// the accumulations in registers, because the tensor cores' own additions
// truncate, which over thousands of them in a row drifts.  Slices of the depth
// (n_z) give the pairs work where there are few tiles.
#include "gemm8.cuh"

namespace trimul {

namespace {
constexpr int ROWS = 128;  // rows of A (and of B) per CTA
constexpr int STAGES = 6;
constexpr uint32_t CODE_BYTES = ROWS * L8_BLOCK;  // 16 KB
constexpr uint32_t A_SCALES = 2 * CODE_BYTES;     // where a stage's scales are
constexpr uint32_t B_SCALES = A_SCALES + L8_SCALE_TILE;
constexpr uint32_t STAGE_BYTES = 34 * 1024;       // 32 KB of codes, 1.5 KB of scales; codes begin on 1024-byte boundaries
constexpr uint32_t BAR_BYTES = 256;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC_STEP = 192;                // from one accumulator to the other
constexpr uint32_t SCALE_COLS = 448, SCALE_SET = 16, SCALE_SETS = 3;
constexpr int EPI_WARPS = 16;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
static_assert(B_SCALES + 2 * L8_SCALE_TILE <= STAGE_BYTES, "the scales fit the stage");
static_assert(ACC_STEP + L8_TILE <= SCALE_COLS && SCALE_COLS + SCALE_SETS * SCALE_SET <= TMEM_COLS, "TMEM");

constexpr uint32_t BIAS_BYTES = EPI_WARPS * 64 * 4;
constexpr size_t kSmem = 1024 + STAGES * STAGE_BYTES + BAR_BYTES + BIAS_BYTES;

}  // namespace

template <bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k12_gemm8(const __grid_constant__ Gemm8Maps maps, const Gemm8Args p) {
  let_next_begin();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + STAGES * STAGE_BYTES;
  // full[STAGES] empty[STAGES] tfull[2] tempty[2] over, drain, then the TMEM base word
  const uint32_t full0 = bars, empty0 = bars + 8 * STAGES, tfull0 = bars + 16 * STAGES;
  const uint32_t tempty0 = tfull0 + 16, over = tempty0 + 16, drain = over + 8;
  const uint32_t tmem_slot = drain + 8;
  volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(base_ptr + (tmem_slot - base));

  const KStatus st{p.status, p.timeout_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: issues the MMAs
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);   // leader only: one expect_tx arrival; bytes of both CTAs
      mbar_init(empty0 + 8 * s, 1);  // one multicast commit per phase
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);               // one multicast commit per phase
      mbar_init(tempty0 + 8 * a, 2 * EPI_WARPS);  // leader only: every epilogue warp of each CTA
    }
    mbar_init(over, 2 * 4);  // leader only: the warps that have read the columns that overlap
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  after_previous();
  const uint32_t tmem_base = *tmem_slot_ptr;
  Walk w(p, blockIdx.x >> 1, gridDim.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0 && !p.stall) {
      tma_prefetch_desc(&maps.a);
      tma_prefetch_desc(&maps.b);
      tma_prefetch_desc(&maps.a_scale);
      tma_prefetch_desc(&maps.b_scale);
      const int groups = (p.blocks + 3) / 4, a_tiles = (p.M + ROWS - 1) / ROWS, b_tiles = (p.N + ROWS - 1) / ROWS;
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (; w.more() && ok; w.next()) {
        // a box wholly past M (N) may not complete its bytes: it loads row 0
        // instead, whose products land only in rows / columns that are not stored
        const int at = w.tm * 2 + static_cast<int>(rank), bt = w.tn * 2 + static_cast<int>(rank);
        const int ra = at < a_tiles ? at * ROWS : 0, rb = bt < b_tiles ? bt * ROWS : 0;
        for (int b = w.b0; b < w.b1; ++b) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, st, SITE_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t sa = base + stage * STAGE_BYTES, sb = sa + CODE_BYTES;
          const uint32_t fb = mapa_shared(full0 + 8 * stage, 0);
          const bool scales = b % 4 == 0 || b == w.b0;
          if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * (2 * CODE_BYTES + (scales ? 3 * L8_SCALE_TILE : 0)));
          const int d = b * L8_BLOCK;
          tma_load_2d_pair(sa, &maps.a, fb, p.a_mn ? ra : d, p.a_mn ? d : ra);
          tma_load_2d_pair(sb, &maps.b, fb, p.b_mn ? rb : d, p.b_mn ? d : rb);
          if (scales) {
            const int g = b / 4, b1 = w.tn * 2 + 1;
            tma_load_2d_pair(sa + A_SCALES, &maps.a_scale, fb, 0, (at < a_tiles ? at : 0) * groups + g);
            tma_load_2d_pair(sa + B_SCALES, &maps.b_scale, fb, 0, w.tn * 2 * groups + g);
            tma_load_2d_pair(sa + B_SCALES + L8_SCALE_TILE, &maps.b_scale, fb, 0, (b1 < b_tiles ? b1 : 0) * groups + g);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        int s = stage;
        uint32_t ph = phase;
        for (long long i = 0; i < issued && i < STAGES; ++i) {
          if (--s < 0) {
            s = STAGES - 1;
            ph ^= 1u;
          }
          mbar_wait_drain(full0 + 8 * s, ph, p.timeout_ns);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && leader) {
      // row by row: 128 rows of 128 bytes of depth, 32 bytes a step.  Depth by
      // depth: 128 lines of 128 rows, eight lines 1024 bytes, 32 lines a step (a
      // CTA's 128 rows are one line, so the offset between lines' parts is not used)
      const uint64_t adesc0 = sdesc_sw128(base, p.a_mn ? CODE_BYTES : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(base + CODE_BYTES, p.b_mn ? CODE_BYTES : 16, 1024);
      const uint32_t astep = p.a_mn ? 32 * 128 >> 4 : 32 >> 4, bstep = p.b_mn ? 32 * 128 >> 4 : 32 >> 4;
      const uint32_t majors = static_cast<uint32_t>(p.a_mn) << 15 | static_cast<uint32_t>(p.b_mn) << 16;
      const uint64_t as0 = sdesc_scales(base + A_SCALES), bs0 = sdesc_scales(base + B_SCALES);
      int stage = 0, acc = 0;
      uint32_t phase = 0, aphase = 0, ophase = 1, set = 0;
      bool ok = true;
      for (; w.more() && ok; w.next()) {
        // the accumulator before the last one, and of the last one the columns that this one shares with it
        if (!mbar_wait(tempty0 + 8 * acc, aphase ^ 1u, st, SITE_MMA) || !mbar_wait(over, ophase, st, SITE_MMA)) {
          ok = false;
          break;
        }
        ophase ^= 1u;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_STEP;
        uint32_t sf = 0;
        for (int b = w.b0; b < w.b1; ++b) {
          if (!mbar_wait(full0 + 8 * stage, phase, st, SITE_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t soff = (stage * STAGE_BYTES) >> 4;
          if (b % 4 == 0 || b == w.b0) {
            sf = tmem_base + SCALE_COLS + set * SCALE_SET;
            if (++set == SCALE_SETS) set = 0;
            copy_scales_pair(sf, as0 + soff);
            copy_scales_pair(sf + 4, bs0 + soff);
            copy_scales_pair(sf + 8, bs0 + soff + (L8_SCALE_TILE >> 4));
          }
          const uint32_t idesc = kIdesc8 | majors | static_cast<uint32_t>(b % 4) << 4 | static_cast<uint32_t>(b % 4) << 29;
#pragma unroll
          for (int kk = 0; kk < L8_BLOCK / 32; ++kk)
            mma_block_scaled_pair(d_tmem, adesc0 + soff + kk * astep, bdesc0 + soff + kk * bstep, idesc, sf, sf + 4,
                                  (b != w.b0 || kk != 0) ? 1u : 0u);
          mma_commit_pair(empty0 + 8 * stage, 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair(tfull0 + 8 * acc, 0x3);
        if (++acc == 2) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) {
        mma_commit_pair(drain, 0x1);
        mbar_wait_drain(drain, 0, p.timeout_ns);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;          // TMEM lane quadrant of this warp
    const int cb = (warp - 2) >> 2;  // its 64-column block
    const uint32_t gb = lane & 7, ga = lane >> 3;
    int acc = 0;
    uint32_t aphase = 0;
    float sum[kF32 ? 64 : 1];
    float* const bias_at = reinterpret_cast<float*>(base_ptr + STAGES * STAGE_BYTES + BAR_BYTES) + (warp - 2) * 64;
    for (; w.more(); w.next()) {
      if (!kF32 && p.bias) {
        __syncwarp();  // the last tile's have been read
        stage_bias(bias_at, p.bias, w.tn * L8_TILE + cb * 64, p.N, lane);
        __syncwarp();
      }
      const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * acc, aphase, st, SITE_EPI));
      if (!ok) break;
      tc_fence_after();
      const int row0 = w.tm * L8_TILE + static_cast<int>(rank) * ROWS + q * 32 + static_cast<int>(ga) * 8;
      const int c0 = w.tn * L8_TILE + cb * 64;
      const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * ACC_STEP + cb * 64;
      // this warp has read its columns: the accumulator's are free when all have, the shared ones when their four warps have
      auto hand_back = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (cb == (acc == 0 ? 3 : 0)) mbar_arrive_remote(mapa_shared(over, 0));
          mbar_arrive_remote(mapa_shared(tempty0 + 8 * acc, 0));
        }
      };
      if constexpr (!kF32) {
        uint4 R[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tmem_read32(t_addr + h * 32, r);
          if (p.bias) add_bias(r, bias_at + h * 32);
          auto pack = [](uint32_t lo, uint32_t hi) { return pack_bf162(__uint_as_float(lo), __uint_as_float(hi)); };
#pragma unroll
          for (int v = 0; v < 4; ++v)
            R[h * 4 + v] = make_uint4(pack(r[v * 8 + 0], r[v * 8 + 1]), pack(r[v * 8 + 2], r[v * 8 + 3]),
                                      pack(r[v * 8 + 4], r[v * 8 + 5]), pack(r[v * 8 + 6], r[v * 8 + 7]));
        }
        hand_back();
        transpose8(R, gb);
        const int col = c0 + static_cast<int>(gb) * 8;
        if (col < p.N) {  // N is a multiple of 8: a chunk is all in or all out
#pragma unroll
          for (int s8 = 0; s8 < 8; ++s8) {
            const int row = row0 + s8;
            if (row < p.M) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c) + static_cast<size_t>(row) * p.N + col) = R[s8];
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tmem_read32(t_addr + h * 32, r);
          if (w.first()) {
#pragma unroll
            for (int v = 0; v < 32; ++v) sum[h * 32 + v] = __uint_as_float(r[v]);
          } else {
#pragma unroll
            for (int v = 0; v < 32; ++v) sum[h * 32 + v] += __uint_as_float(r[v]);
          }
        }
        hand_back();
        if (w.last()) {
          float* const cz = static_cast<float*>(p.c) + static_cast<size_t>(w.z) * p.M * p.N;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 32 columns: 8 chunks of 4 fp32
            uint4 R[8];
#pragma unroll
            for (int v = 0; v < 8; ++v)
              R[v] = make_uint4(__float_as_uint(sum[h * 32 + v * 4]), __float_as_uint(sum[h * 32 + v * 4 + 1]),
                                __float_as_uint(sum[h * 32 + v * 4 + 2]), __float_as_uint(sum[h * 32 + v * 4 + 3]));
            transpose8(R, gb);
            const int col = c0 + h * 32 + static_cast<int>(gb) * 4;
            if (col < p.N) {
#pragma unroll
              for (int s8 = 0; s8 < 8; ++s8) {
                const int row = row0 + s8;
                if (row < p.M) *reinterpret_cast<uint4*>(cz + static_cast<size_t>(row) * p.N + col) = R[s8];
              }
            }
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        aphase ^= 1u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

cudaError_t launch_gemm8(const Gemm8Args& a, const Gemm8Maps& m, bool f32, int pairs, cudaStream_t s) {
  auto kernel = f32 ? k12_gemm8<true> : k12_gemm8<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(a.tiles_m) * a.tiles_n * a.n_z;
  const int grid = 2 * static_cast<int>(tiles < pairs ? tiles : pairs);
  return launch8(kernel, grid, THREADS, kSmem, true, s, m, a);
}

int gemm8_max_pairs(int num_sms) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms & ~1, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(k12_gemm8<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k12_gemm8<false>, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return num_sms / 2;
  }
  return n;
}

}  // namespace trimul
