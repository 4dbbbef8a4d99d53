// k13_fused8.cu -- the product in 8 bits (k12_gemm8.cu) with one operand taken
// as bf16 and rounded on its way to the tensor cores, so that its codes never
// reach memory.
//
//   by rows (kCols false)    C[m][n] = Q(t)[m][:] . B[n][:]     t: bf16 [M][depth], 128 of a row share a power: y and dx
//   by columns (kCols true)  C[m][n] = Q(t)[:][m] . B[n][:]     t: bf16 [depth][M], 128 of a column share a power: dW
//
// A pair stack's layers are narrow (K of 1024 at most) and have millions of
// rows: bf16 in, bf16 out bounds them, and a pass of its own for the codes would
// write and read half of the input again.  The price is that a tile of t is
// rounded once for every 256 columns of C, unless it has few blocks (below).
//
// Two neighbouring CTAs have 128 rows of a tile each, and share nothing else: each loads
// all of B's tile (TMA; the second read is L2's) and multiplies by itself (M = 128, N = 256,
// cta_group::1).  As one pair as in k12_gemm8.cu, the odd CTA's codes had to be made known to the even CTA by a release at
// cluster scope for every block, which takes about as long as rounding it (550 to 860 us at 2^20 rows of 1024 to 256,
// whichever warps did it).
//
// Per CTA: warp 0 loads B and the last one the CTA's tile of t, 1 issues the
// multiplications, 2..9 are the epilogue, and the others round, in teams of eight.  A tile of t waits as bf16
// in a ring of its own.  Eight lanes take a row's 128 numbers (by columns, a warp sixteen
// columns), and the codes go to shared memory as TMA would have put them
// there, with the block's powers beside them; a proxy fence makes them visible to the
// tensor cores.  (The rounding warps load nothing from global memory themselves: with
// the next block's loads on their way in registers each fence waited for those.)
//
// TMEM as in k12_gemm8.cu; A's powers are copied for each block (eight sets of four
// columns, more than the ring is deep: a set's readers are done when it is written
// again), B's for each group of four.
//
// fp32 output: an accumulation takes `chunk` blocks, and the epilogue adds it to
// what it has written before.  Each element has one thread, whichever accumulator
// it is in, whose additions to it come in its program's order: the order is fixed.
// They are done in L2 (red): with a load, an addition and a store the warps waited for the
// loads, and dW of 2^20 rows of 1024 to 256 channels took 80 us more (579 now, dy's codes among them).
#include "gemm8.cuh"
#include "quantize8.cuh"

namespace trimul {

namespace {
constexpr int ROWS = 128;
// Blocks of t that are asked for in L2 ahead of their turn, as the tiles that are on their way are too few: 2^20 rows of 1024 to 256
// channels take 459 us without, 417 with two and 419 with four, 256 to 256 take 241, 163 and 209.  Where a run's tiles share the
// codes it does not help: 256 to 1024 takes 433 to 435 us without and 429 to 435 with two.
constexpr int AHEAD = 2;
constexpr uint32_t CODE_BYTES = ROWS * L8_BLOCK;
constexpr uint32_t B_BYTES = 2 * CODE_BYTES;  // 256 rows of B
constexpr uint32_t RAW_HALF = 128 * 128, RAW_BYTES = 2 * RAW_HALF;  // 128 rows of 64 bf16 numbers, twice
constexpr uint32_t OUT_BYTES = 32 * 128;  // of an epilogue warp: 32 rows of 64 bf16 numbers
constexpr uint32_t BAR_BYTES = 512;
constexpr uint32_t BIAS_BYTES = 8192;
constexpr int ALL_BIAS = BIAS_BYTES / 4;  // up to so many outputs it is all there; past that each epilogue warp has that of its tile
constexpr uint32_t TMEM_COLS = 512, ACC_STEP = 192;
constexpr uint32_t A_COLS = 448, A_SETS = 8, B_COLS = 480, B_SETS = 4;
static_assert(A_COLS + 4 * A_SETS <= B_COLS && B_COLS + 8 * B_SETS <= TMEM_COLS, "TMEM");
constexpr int EPI0 = 2, EPI_WARPS = 8, ROUND0 = EPI0 + EPI_WARPS, TEAM_WARPS = 8;
constexpr int TURNS = 16 / EPI_WARPS;  // 64-column blocks of an epilogue warp
// How the warps and the shared memory are shared out.  kFew: by rows, with few blocks of depth (FUSED8_FEW_BLOCKS).  There the
// way out counts: a tile goes by way of shared memory and TMA.  (Turned in registers by shuffles and stored by the warps, 2^20 rows of
// 256 to 1024 channels took 455 us and with a bias 531; this way 433 and 435.  128 to 128: 119 and 145, now 89 and 93.)
// The room is a tile of t's, one team is enough for what is left to round, and the warps have more registers.
// Else rounding has two teams: with one, or with one tile of t on its way, it falls behind.
template <bool kFew>
struct Plan {
  static constexpr int A_SLOTS = 3, B_STAGES = 3, RAW_SLOTS = kFew ? 1 : 2;
  static constexpr int TEAMS = kFew ? 1 : 2, RAW = ROUND0 + TEAMS * TEAM_WARPS, THREADS = 32 * (RAW + 1);
  static constexpr int EMPTIES = B_STAGES * TEAMS;  // barriers of B's stages that say they are free
  // rings: A's codes, B's codes, tiles of t, what is on its way out, A's and B's scales
  static constexpr uint32_t B0 = A_SLOTS * CODE_BYTES, RAW0 = B0 + B_STAGES * B_BYTES, OUT0 = RAW0 + RAW_SLOTS * RAW_BYTES;
  static constexpr uint32_t AS0 = OUT0 + (kFew ? EPI_WARPS * OUT_BYTES : 0);
  static constexpr uint32_t BS0 = AS0 + A_SLOTS * L8_SCALE_TILE, BARS = BS0 + B_STAGES * 2 * L8_SCALE_TILE;
  static constexpr size_t SMEM = 1024 + BARS + BAR_BYTES + BIAS_BYTES;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert(8 * (B_STAGES + EMPTIES + 2 * A_SLOTS + 2 * RAW_SLOTS + 6) + 4 <= BAR_BYTES && 16 * 64 * 4 <= BIAS_BYTES, "the barriers and the bias fit");
  static_assert(kFew ? FUSED8_FEW_BLOCKS <= A_SLOTS : A_SLOTS == B_STAGES, "a run's codes wait in their slots, or go with a stage of B's");
  static_assert(A_SETS > B_STAGES + 1 && B_STAGES <= B_SETS, "a set's readers are done when it is written again");
  // A team waits for its own blocks alone.  A wait that has skipped a phase of its barrier would take the one before for the one it
  // wants, and pass at once.  So a slot of t is always the same team's, and a stage of B, whose uses fall to the teams in
  // turns, has a barrier for each: block m's multiplications arrive at barrier m % EMPTIES, and the block B_STAGES behind,
  // always the same team's, waits there.
  static_assert(RAW_SLOTS % TEAMS == 0, "a slot of t is always the same team's");
  static_assert(EMPTIES % TEAMS == 0 && EMPTIES % B_STAGES == 0, "a free stage's barrier is always the same team's");
};
constexpr uint32_t SITE_ROUND = 0x500;
constexpr uint32_t kIdesc128 = (kIdesc8 & ~(0x1Fu << 24)) | ((ROWS >> 4) << 24);

__device__ __forceinline__ void mma_block_scaled(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t a_scale,
                                                 uint32_t b_scale, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(sdesc) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0),
               "r"(c1)
               : "memory");
}
// A box into L2 alone.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* m, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1) : "memory");
}

// Adds four fp32 numbers to those at `to`, on their way through L2.
__device__ __forceinline__ void add_to(float* to, const uint4& v) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to), "f"(__uint_as_float(v.x)), "f"(__uint_as_float(v.y)),
               "f"(__uint_as_float(v.z)), "f"(__uint_as_float(v.w))
               : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void st_shared8(uint32_t at, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t at, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }

// A thread's 64 numbers of a block.
struct Numbers {
  uint4 v[8];
};

__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// 16 bytes of a row of a tile of t: `chunk` of the row's sixteen (128-byte swizzle, 64 numbers a half).
__device__ __forceinline__ uint4 raw16(uint32_t slot, int row, int chunk) {
  return ld_shared16(slot + (chunk >> 3) * RAW_HALF + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

// ---- by rows: lane `lane8` of row group `group` (0..31) has numbers 8 lane8 .. + 7 and 64 + 8 lane8 .. of rows group +
// 32 u: v[2 u] and v[2 u + 1]; `left`: of the block's 128, those before the row's end (the others are not loaded)
__device__ __forceinline__ void load_rows(Numbers& x, uint32_t slot, int left, int group, int lane8) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x.v[2 * u + h] = make_uint4(0u, 0u, 0u, 0u);
      if (64 * h + 8 * lane8 < left) x.v[2 * u + h] = raw16(slot, group + 32 * u, 8 * h + lane8);
    }
}
template <typename Release>
__device__ __forceinline__ void round_rows(const Numbers& x, uint32_t codes, uint32_t scales, int group, int lane8, Release release) {
  uint32_t m[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) m[u] = max_magnitude(x.v[2 * u], x.v[2 * u + 1]);
  // two rows' largest in a word, over the row's eight lanes
  auto over_row = [&](uint32_t (&top)[4]) {
    uint32_t two[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      two[k] = max16x2(__byte_perm(top[2 * k], top[2 * k + 1], 0x5410), __byte_perm(top[2 * k], top[2 * k + 1], 0x7632));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      two[0] = max16x2(two[0], __shfl_xor_sync(0xffffffffu, two[0], o));
      two[1] = max16x2(two[1], __shfl_xor_sync(0xffffffffu, two[1], o));
    }
    top[0] = two[0] & 0xffffu, top[1] = two[0] >> 16, top[2] = two[1] & 0xffffu, top[3] = two[1] >> 16;
  };
  over_row(m);
  release();
  bool fine[4], all = true;
#pragma unroll
  for (int u = 0; u < 4; ++u) fine[u] = m[u] < 0x7f80u, all = all && fine[u];
  if (!__all_sync(0xffffffffu, all)) {  // rare
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = max16x2(max_of(finite(x.v[2 * u])), max_of(finite(x.v[2 * u + 1])));
    over_row(m);
  }
  uint32_t byte[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    byte[u] = scale_byte(m[u] << 16);
    const float inv = over_scale(byte[u]);
    const uint2 a = codes_of(x.v[2 * u], inv, fine[u]), b = codes_of(x.v[2 * u + 1], inv, fine[u]);
    const int row = group + 32 * u;
    st_shared8(codes + row * 128 + (((lane8 >> 1) ^ (row & 7)) << 4) + (lane8 & 1) * 8, a);
    st_shared8(codes + row * 128 + (((4 + (lane8 >> 1)) ^ (row & 7)) << 4) + (lane8 & 1) * 8, b);
  }
  if (lane8 == 0) st_shared16(scales + group * 16, byte[0], byte[1], byte[2], byte[3]);
}

// ---- by columns: warp `warp` of the team has columns 16 warp .. + 15, a lane the eight of its `chunk` (2 warp or 2 warp + 1) in
// rows `row0` + 16 u: v[u]; eight neighbouring lanes eight rows of a chunk, so that no two meet in a bank.  A column's
// numbers are all in one warp: no other is waited for.  `left`: of the tile's 128 columns, those before the last
__device__ __forceinline__ void load_cols(Numbers& x, uint32_t slot, int left, int row0, int chunk) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    x.v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (8 * chunk < left) x.v[u] = raw16(slot, row0 + 16 * u, chunk);
  }
}
template <bool kSums, typename Release>
__device__ __forceinline__ void round_cols(const Numbers& x, f2 (&sums)[4], uint32_t codes, uint32_t scales, int lane, int row0, int chunk,
                                           Release release) {
  auto join = [](uint4& a, const uint4& b) {
    a.x = max16x2(a.x, b.x), a.y = max16x2(a.y, b.y), a.z = max16x2(a.z, b.z), a.w = max16x2(a.w, b.w);
  };
  auto larger = [](uint4& a, const uint4& b) {
    a.x = max_signed(a.x, b.x), a.y = max_signed(a.y, b.y), a.z = max_signed(a.z, b.z), a.w = max_signed(a.w, b.w);
  };
  uint4 top = x.v[0];
#pragma unroll
  for (int u = 1; u < 8; ++u) larger(top, x.v[u]);
  top = magnitudes(top);
  const uint32_t all = max_of(top);
  const bool fine = (all & 0xffffu) < 0x7f80u && all < 0x7f800000u;
  if (!fine) {  // rare
    top = finite(x.v[0]);
#pragma unroll
    for (int u = 1; u < 8; ++u) join(top, finite(x.v[u]));
  }
  // Over the sixteen lanes of a chunk (all of a lane's bits but 8): by bit 16 a lane keeps two of its four words and gets the
  // other lane's, by bit 4 one of the two.  Then each lane has two columns, whose powers it works out, and the way back
  // brings those of all eight.
  const bool hi2 = lane & 16, hi1 = lane & 4;
  auto other = [](uint32_t v, int bit) { return __shfl_xor_sync(0xffffffffu, v, bit); };
  const uint32_t t0 = max16x2(hi2 ? top.z : top.x, other(hi2 ? top.x : top.z, 16));
  const uint32_t t1 = max16x2(hi2 ? top.w : top.y, other(hi2 ? top.y : top.w, 16));
  uint32_t m = max16x2(hi1 ? t1 : t0, other(hi1 ? t0 : t1, 4));
  m = max16x2(m, other(m, 2));
  m = max16x2(m, other(m, 1));
  release();
  const uint32_t two = scale_byte(m << 16) | scale_byte(m & 0xffff0000u) << 8;
  const uint32_t two1 = other(two, 4);
  const uint32_t four = __byte_perm(two, two1, hi1 ? 0x1054 : 0x5410), four1 = other(four, 16);
  const uint32_t lo = hi2 ? four1 : four, hi = hi2 ? four : four1;  // the bytes of columns 0 .. 3 and 4 .. 7
  f2 inv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = e < 2 ? lo : hi, at = 16 * (e & 1);
    inv[e] = pair2(over_scale(w >> at & 0xffu), over_scale(w >> (at + 8) & 0xffu));
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int row = row0 + 16 * u;
    if (kSums) add_row(sums, x.v[u]);
    st_shared8(codes + row * 128 + (((chunk >> 1) ^ (row & 7)) << 4) + (chunk & 1) * 8, codes_of(x.v[u], inv, fine));
  }
  if (!(lane & 2)) {  // a lane's two columns, by bit 1
    const int c = chunk * 8 + 4 * hi2 + 2 * hi1 + (lane & 1);
    st_shared4(scales + (c % 32) * 16 + (c / 32) * 4, two >> (8 * (lane & 1)) & 0xffu);
  }
}
}  // namespace

// kFew (by rows only): a run's tiles take the same codes of A, which wait in their slots until the last tile has had them.
// Else a slot of A's codes goes with a stage of B's, and is free when that is.
// kMore: with a bias; by columns, with the sums of t's columns (dbias), which the rounding warps take as they pass: a lane adds its
// eight rows of each of its team's blocks, the sixteen lanes of a column are joined, and every slice leaves two sums.
template <bool kCols, bool kFew, bool kMore>
__global__ void __launch_bounds__(Plan<kFew>::THREADS, 1)
    k13_fused8(const __grid_constant__ CUtensorMap tm_t, const __grid_constant__ CUtensorMap tm_b,
               const __grid_constant__ CUtensorMap tm_b_scale, const __grid_constant__ CUtensorMap tm_c, const Fused8Args p) {
  using P = Plan<kFew>;
  constexpr int A_SLOTS = P::A_SLOTS, B_STAGES = P::B_STAGES, RAW_SLOTS = P::RAW_SLOTS, TEAMS = P::TEAMS, EMPTIES = P::EMPTIES,
                RAW = P::RAW;
  constexpr uint32_t B0 = P::B0, RAW0 = P::RAW0, AS0 = P::AS0, BS0 = P::BS0, BARS = P::BARS;
  constexpr bool kBias = kMore && !kCols, kSums = kMore && kCols;
  let_next_begin();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bars = base + BARS;
  // bfull [B_STAGES] bempty [EMPTIES] afull aempty [A_SLOTS] rfull rempty [RAW_SLOTS] tfull tempty [2] over drain, then the TMEM base word
  const uint32_t bfull0 = bars, bempty0 = bfull0 + 8 * B_STAGES, afull0 = bempty0 + 8 * EMPTIES, aempty0 = kFew ? afull0 + 8 * A_SLOTS : bempty0;
  const uint32_t rfull0 = afull0 + 16 * A_SLOTS, rempty0 = rfull0 + 8 * RAW_SLOTS;
  const uint32_t tfull0 = rempty0 + 8 * RAW_SLOTS, tempty0 = tfull0 + 16, over = tempty0 + 16, drain = over + 8;
  const uint32_t tmem_slot = drain + 8;
  volatile uint32_t* tmem_slot_ptr = reinterpret_cast<volatile uint32_t*>(base_ptr + (tmem_slot - base));

  const KStatus st{p.g.status, p.g.timeout_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1;  // which half of a tile's rows

  // a first kernel has nobody before it to clear the status word: the first block does, and no other looks at it sooner
  // than a millisecond into a wait
  if (p.clear && blockIdx.x == 0 && threadIdx.x == 0) *p.g.status = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < B_STAGES; ++s) {
      mbar_init(bfull0 + 8 * s, 1);            // one expect_tx arrival
    }
    for (int s = 0; s < EMPTIES; ++s) mbar_init(bempty0 + 8 * s, 1);  // one commit
    for (int s = 0; s < A_SLOTS; ++s) {
      mbar_init(afull0 + 8 * s, TEAM_WARPS);
      if (kFew) mbar_init(aempty0 + 8 * s, 1);  // one commit
    }
    for (int r = 0; r < RAW_SLOTS; ++r) {
      mbar_init(rfull0 + 8 * r, 1);  // one expect_tx arrival
      mbar_init(rempty0 + 8 * r, TEAM_WARPS);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, EPI_WARPS);
    }
    mbar_init(over, 4);  // the warps that have read the columns that overlap
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  float* const bias_at = reinterpret_cast<float*>(base_ptr + BARS + BAR_BYTES);
  const bool all_bias = kBias && p.g.N <= ALL_BIAS;
  if (all_bias) {
    for (int i = threadIdx.x; i < ALL_BIAS; i += P::THREADS) bias_at[i] = i < p.g.N ? p.g.bias[i] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  after_previous();  // (the bias is older than the call)
  const uint32_t tmem_base = *tmem_slot_ptr;
  Walk w(p.g, blockIdx.x >> 1, gridDim.x >> 1);

  if (warp == 0) {
    // ------------------------------------------------------------ producer of B
    if (lane == 0 && !p.g.stall) {
      tma_prefetch_desc(&tm_b);
      tma_prefetch_desc(&tm_b_scale);
      const int groups = (p.g.blocks + 3) / 4, b_tiles = (p.g.N + ROWS - 1) / ROWS;
      int stage = 0, empty = EMPTIES - B_STAGES;
      uint32_t phase = 0, ephase = 1;  // (the first uses pass)
      long long issued = 0;
      bool ok = true;
      for (; w.more() && ok; w.next()) {
        // (a half wholly past N is not loaded: what is there instead makes columns that are not stored)
        const int bt = 2 * w.tn, halves = bt + 1 < b_tiles ? 2 : 1;
        for (int b = w.b0; b < w.b1; ++b) {
          if (!mbar_wait(bempty0 + 8 * empty, ephase, st, SITE_PRODUCER)) {
            ok = false;
            break;
          }
          if (++empty == EMPTIES) {
            empty = 0;
            ephase ^= 1u;
          }
          const uint32_t fb = bfull0 + 8 * stage;
          const bool scales = b % 4 == 0 || b == w.b0;
          mbar_arrive_expect_tx(fb, halves * (CODE_BYTES + (scales ? L8_SCALE_TILE : 0)));
          const int d = b * L8_BLOCK;
          for (int h = 0; h < halves; ++h) {
            const int rb = (bt + h) * ROWS;
            tma_load_2d(base + B0 + stage * B_BYTES + h * CODE_BYTES, &tm_b, fb, p.g.b_mn ? rb : d, p.g.b_mn ? d : rb);
            if (scales) tma_load_2d(base + BS0 + (2 * stage + h) * L8_SCALE_TILE, &tm_b_scale, fb, 0, (bt + h) * groups + b / 4);
          }
          ++issued;
          if (++stage == B_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {  // the copies on their way land before the CTA goes away
        int s = stage;
        uint32_t ph = phase;
        for (long long i = 0; i < issued && i < B_STAGES; ++i) {
          if (--s < 0) {
            s = B_STAGES - 1;
            ph ^= 1u;
          }
          mbar_wait_drain(bfull0 + 8 * s, ph, p.g.timeout_ns);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint64_t adesc0 = sdesc_sw128(base, kCols ? CODE_BYTES : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(base + B0, p.g.b_mn ? CODE_BYTES : 16, 1024);
      const uint64_t as0 = sdesc_scales(base + AS0), bs0 = sdesc_scales(base + BS0);
      const uint32_t astep = kCols ? 32 * 128 >> 4 : 32 >> 4, bstep = p.g.b_mn ? 32 * 128 >> 4 : 32 >> 4;
      const uint32_t majors = static_cast<uint32_t>(kCols) << 15 | static_cast<uint32_t>(p.g.b_mn) << 16;
      int stage = 0, empty = 0, acc = 0, slot = 0, run_slot = 0;
      uint32_t phase = 0, sphase = 0, run_phase = 0, aphase = 0, ophase = 1, a_set = 0, b_set = 0;
      bool ok = true;
      for (; w.more() && ok; w.next()) {
        if (!mbar_wait(tempty0 + 8 * acc, aphase ^ 1u, st, SITE_MMA) || !mbar_wait(over, ophase, st, SITE_MMA)) {
          ok = false;
          break;
        }
        ophase ^= 1u;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_STEP;
        uint32_t sfb = 0;
        if (kFew) slot = run_slot, sphase = run_phase;  // each tile of a run begins at its first slot
        const bool give_back = kFew && w.last_tile();
        for (int b = w.b0; b < w.b1; ++b) {
          if (!mbar_wait(bfull0 + 8 * stage, phase, st, SITE_MMA) || !mbar_wait(afull0 + 8 * slot, sphase, st, SITE_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t aoff = (slot * CODE_BYTES) >> 4, boff = (stage * B_BYTES) >> 4;
          const uint32_t sfa = tmem_base + A_COLS + a_set * 4;
          if (++a_set == A_SETS) a_set = 0;
          copy_scales(sfa, as0 + slot * (L8_SCALE_TILE >> 4));
          if (b % 4 == 0 || b == w.b0) {
            sfb = tmem_base + B_COLS + b_set * 8;
            if (++b_set == B_SETS) b_set = 0;
            copy_scales(sfb, bs0 + 2 * stage * (L8_SCALE_TILE >> 4));
            copy_scales(sfb + 4, bs0 + (2 * stage + 1) * (L8_SCALE_TILE >> 4));
          }
          const uint32_t idesc = kIdesc128 | majors | static_cast<uint32_t>(b % 4) << 4;  // A's power is the first byte of its word
#pragma unroll
          for (int kk = 0; kk < L8_BLOCK / 32; ++kk)
            mma_block_scaled(d_tmem, adesc0 + aoff + kk * astep, bdesc0 + boff + kk * bstep, idesc, sfa, sfb,
                                  (b != w.b0 || kk != 0) ? 1u : 0u);
          mma_commit(bempty0 + 8 * empty);
          if (++empty == EMPTIES) empty = 0;
          if (give_back) mma_commit(aempty0 + 8 * slot);
          if (++stage == B_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          if (++slot == A_SLOTS) {
            slot = 0;
            sphase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(tfull0 + 8 * acc);
        if (give_back) run_slot = slot, run_phase = sphase;
        if (++acc == 2) {
          acc = 0;
          aphase ^= 1u;
        }
      }
      if (!ok) {
        mma_commit(drain);
        mbar_wait_drain(drain, 0, p.g.timeout_ns);
      }
    }
  } else if (warp < ROUND0) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;               // TMEM lane quadrant of this warp
    // 0: the outer two of the 64-column blocks, 1: the inner two (an element has one thread, whichever accumulator it is in)
    const int sub = (warp - EPI0) >> 2;
    auto block_of = [&](int turn, int acc) { return (turn ^ acc) ? sub : 3 - sub; };
    const uint32_t gb = lane & 7, ga = lane >> 3;
    int acc = 0;
    uint32_t aphase = 0;
    bool ok = true;
    for (; w.more() && ok; w.next()) {
      if (kBias && !all_bias) {
        __syncwarp();  // the last tile's have been read
#pragma unroll
        for (int turn = 0; turn < TURNS; ++turn)
          stage_bias(bias_at + (TURNS * (warp - EPI0) + turn) * 64, p.g.bias, w.tn * L8_TILE + block_of(turn, acc) * 64, p.g.N, lane);
        __syncwarp();
      }
      ok = __all_sync(0xffffffffu, mbar_wait(tfull0 + 8 * acc, aphase, st, SITE_EPI));
      if (!ok) break;
      tc_fence_after();
      const int row0 = w.tm * L8_TILE + static_cast<int>(rank) * ROWS + q * 32 + static_cast<int>(ga) * 8;
#pragma unroll 1
      for (int turn = 0; turn < TURNS; ++turn) {
        const int cb = block_of(turn, acc);
        const bool shared = cb == (acc ? 0 : 3);  // the columns that both accumulators have
        const int c0 = w.tn * L8_TILE + cb * 64;
        const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * ACC_STEP + cb * 64;
        auto hand_back = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (shared) mbar_arrive(over);
            if (turn == TURNS - 1) mbar_arrive(tempty0 + 8 * acc);
          }
        };
        if constexpr (kFew) {
          if (c0 >= p.g.N) {  // nothing of C
            hand_back();
            continue;
          }
          // by way of shared memory, row by row as the tile's map has them (128-byte swizzle); TMA writes what lies in C
          const float* const bias = bias_at + (all_bias ? c0 : (TURNS * (warp - EPI0) + turn) * 64);
          const uint32_t out = base + P::OUT0 + (warp - EPI0) * OUT_BYTES;
          const int row = w.tm * L8_TILE + static_cast<int>(rank) * ROWS + q * 32;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            tmem_read32(t_addr + h * 32, r);
            if (h == 1) hand_back();
            if (kBias) add_bias(r, bias + h * 32);
            if (h == 0) {
              if (lane == 0) tma_store_wait_read<0>();  // the last one has been read
              __syncwarp();
            }
            auto pack = [](uint32_t lo, uint32_t hi) { return pack_bf162(__uint_as_float(lo), __uint_as_float(hi)); };
#pragma unroll
            for (int v = 0; v < 4; ++v)
              st_shared16(out + lane * 128 + (((4 * h + v) ^ gb) << 4), pack(r[v * 8 + 0], r[v * 8 + 1]), pack(r[v * 8 + 2], r[v * 8 + 3]),
                          pack(r[v * 8 + 4], r[v * 8 + 5]), pack(r[v * 8 + 6], r[v * 8 + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row < p.g.M) {
            tma_store_2d(&tm_c, out, c0, row);
            tma_store_commit();
          }
        } else if constexpr (!kCols) {
          // 32 columns at a time, and four rows' chunks among four lanes: few registers, as the rounding warps leave few
          const float* const bias = bias_at + (all_bias ? c0 : (TURNS * (warp - EPI0) + turn) * 64);
          const int row4 = w.tm * L8_TILE + static_cast<int>(rank) * ROWS + q * 32 + (lane & ~3);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 R[4];
            {
              uint32_t r[32];
              tmem_read32(t_addr + h * 32, r);
              if (h == 1) hand_back();
              if (kBias) add_bias(r, bias + h * 32);
              auto pack = [](uint32_t lo, uint32_t hi) { return pack_bf162(__uint_as_float(lo), __uint_as_float(hi)); };
#pragma unroll
              for (int v = 0; v < 4; ++v)
                R[v] = make_uint4(pack(r[v * 8 + 0], r[v * 8 + 1]), pack(r[v * 8 + 2], r[v * 8 + 3]), pack(r[v * 8 + 4], r[v * 8 + 5]),
                                  pack(r[v * 8 + 6], r[v * 8 + 7]));
            }
            transpose4(R, lane & 3);
            const int col = c0 + h * 32 + (lane & 3) * 8;
            if (col < p.g.N) {  // N is a multiple of 8: a chunk is all in or all out
#pragma unroll
              for (int s4 = 0; s4 < 4; ++s4) {
                const int row = row4 + s4;
                if (row < p.g.M) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.g.c) + static_cast<size_t>(row) * p.g.N + col) = R[s4];
              }
            }
          }
        } else {
          float* const cz = static_cast<float*>(p.g.c) + static_cast<size_t>(w.z) * p.g.M * p.g.N;
          const bool add = !w.first();
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 32 columns: 8 chunks of 4 fp32
            uint4 R[8];
            {
              uint32_t r[32];
              tmem_read32(t_addr + h * 32, r);
#pragma unroll
              for (int v = 0; v < 8; ++v) R[v] = make_uint4(r[v * 4], r[v * 4 + 1], r[v * 4 + 2], r[v * 4 + 3]);
            }
            if (h == 1) hand_back();
            transpose8(R, gb);
            const int col = c0 + h * 32 + static_cast<int>(gb) * 4;
            if (col < p.g.N) {
#pragma unroll
              for (int s8 = 0; s8 < 8; ++s8) {
                const int row = row0 + s8;
                if (row >= p.g.M) continue;
                float* const to = cz + static_cast<size_t>(row) * p.g.N + col;
                if (add)
                  add_to(to, R[s8]);
                else
                  *reinterpret_cast<uint4*>(to) = R[s8];
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
    if (kFew && lane == 0) tma_store_wait_all();
  } else if (warp < RAW) {
    // ------------------------------------------------------------ rounding of A
    // the teams take the blocks in turns: one block's way through shared memory, the maxima and the conversions is long, and the
    // other team's instructions fill it
    const int team = (warp - ROUND0) / TEAM_WARPS, t = threadIdx.x - 32 * (ROUND0 + team * TEAM_WARPS);
    // by columns: the chunk and the first row
    const int lanes = kCols ? t / 32 * 2 + (lane >> 3 & 1) : t % 8, group = kCols ? (lane & 7) + (lane >> 4) * 8 : t / 8;
    constexpr int kFrees = kFew ? A_SLOTS : EMPTIES;  // the barriers that say that a slot of A's is free
    int slot = 0, free = kFrees - A_SLOTS, raw_slot = 0, turn = 0;
    uint32_t fphase = 1, rphase = 0;
    bool ok = true;
    f2 sums[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
    int first_turn = 0;
    for (; w.more() && ok; kFew ? w.next_run() : w.next()) {
      const long long c0 = (static_cast<long long>(w.tm) * 2 + rank) * ROWS;
      for (int b = w.b0; b < w.b1; ++b) {
        if (turn == team) {
          ok = __all_sync(0xffffffffu, mbar_wait(rfull0 + 8 * raw_slot, rphase, st, SITE_ROUND) &&
                                           mbar_wait(aempty0 + 8 * free, fphase, st, SITE_ROUND));
          if (!ok) break;
          const uint32_t sr = base + RAW0 + raw_slot * RAW_BYTES, sa = base + slot * CODE_BYTES, ss = base + AS0 + slot * L8_SCALE_TILE;
          Numbers x;
          if (kCols) {
            const long long left = p.g.M - c0;
            load_cols(x, sr, left < ROWS ? static_cast<int>(left) : ROWS, group, lanes);
          } else {
            const long long left = p.depth - static_cast<long long>(b) * L8_BLOCK;
            load_rows(x, sr, left < L8_BLOCK ? static_cast<int>(left) : L8_BLOCK, group, lanes);
          }
          // The slot is free once the numbers are here, not once their loads have been issued: it is given back behind the
          // maxima, which need all of them.  (Given back right behind the loads, by columns one pass in two hundred took some
          // numbers from the next block's copy.)
          auto release = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(rempty0 + 8 * raw_slot);
          };
          if (kCols)
            round_cols<kSums>(x, sums, sa, ss, lane, group, lanes, release);
          else
            round_rows(x, sa, ss, group, lanes, release);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(afull0 + 8 * slot);
        }
        if (++turn == TEAMS) turn = 0;
        if (++slot == A_SLOTS) slot = 0;
        if (++free == kFrees) {
          free = 0;
          fphase ^= 1u;
        }
        if (++raw_slot == RAW_SLOTS) {
          raw_slot = 0;
          rphase ^= 1u;
        }
      }
      if (kSums && ok && w.last()) {  // a slice's end: the sums of every other of its blocks, from the first or the second on
        const int odd = team ^ first_turn;
        const long long c = c0 + 8 * lanes;
        if (w.tn == 0) join_columns(sums, p.sums + (static_cast<long long>(w.z) * TEAMS + odd) * p.g.M + c, c < p.g.M);
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[e] = both(0.f);
        first_turn = turn;
      }
    }
  } else {
    // ------------------------------------------------------------ producer of t
    if (lane == 0 && !p.g.stall) {
      tma_prefetch_desc(&tm_t);
      int slot = 0, lead = 0;
      uint32_t rphase = 0;
      long long issued = 0;
      bool ok = true;
      // (a box wholly past t may not complete its bytes: rows of C past M take those of row 0, and a half that has nothing
      // is not loaded)
      struct Box {
        int x, y, halves;
      };
      auto box = [&](const Walk& v, int b) {
        long long c0 = (static_cast<long long>(v.tm) * 2 + rank) * ROWS;
        if (c0 >= p.g.M) c0 = 0;
        const int d = b * L8_BLOCK, x = kCols ? static_cast<int>(c0) : d;
        return Box{x, kCols ? d : static_cast<int>(c0), x + 64 < (kCols ? p.g.M : p.depth) ? 2 : 1};
      };
      auto next = [](Walk& v) { kFew ? v.next_run() : v.next(); };
      const int ahead = p.g.run > 1 ? 0 : AHEAD;
      Walk far = w;
      int far_b = far.b0;
      for (; w.more() && ok; next(w)) {
        for (int b = w.b0; b < w.b1; ++b) {
          for (; lead < ahead && far.more(); ++lead) {
            const Box f = box(far, far_b);
            tma_prefetch_2d(&tm_t, f.x, f.y);
            if (f.halves == 2) tma_prefetch_2d(&tm_t, f.x + 64, f.y);
            if (++far_b == far.b1) {
              next(far);
              far_b = far.b0;
            }
          }
          if (ahead) --lead;
          if (!mbar_wait(rempty0 + 8 * slot, rphase ^ 1u, st, SITE_PRODUCER)) {
            ok = false;
            break;
          }
          const Box t = box(w, b);
          const uint32_t sr = base + RAW0 + slot * RAW_BYTES;
          mbar_arrive_expect_tx(rfull0 + 8 * slot, t.halves * RAW_HALF);
          tma_load_2d(sr, &tm_t, rfull0 + 8 * slot, t.x, t.y);
          if (t.halves == 2) tma_load_2d(sr + RAW_HALF, &tm_t, rfull0 + 8 * slot, t.x + 64, t.y);
          ++issued;
          if (++slot == RAW_SLOTS) {
            slot = 0;
            rphase ^= 1u;
          }
        }
      }
      if (!ok) {  // the copies on their way land before the CTA goes away
        int r = slot;
        uint32_t ph = rphase;
        for (long long i = 0; i < issued && i < RAW_SLOTS; ++i) {
          if (--r < 0) {
            r = RAW_SLOTS - 1;
            ph ^= 1u;
          }
          mbar_wait_drain(rfull0 + 8 * r, ph, p.g.timeout_ns);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

cudaError_t launch_fused8(const Fused8Args& a, const Fused8Maps& m, bool cols, int pairs, cudaStream_t s) {
  const bool few = !cols && a.g.blocks <= FUSED8_FEW_BLOCKS;
  auto kernel = cols  ? (a.sums ? k13_fused8<true, false, true> : k13_fused8<true, false, false>)
                : few ? (a.g.bias ? k13_fused8<false, true, true> : k13_fused8<false, true, false>)
                      : (a.g.bias ? k13_fused8<false, false, true> : k13_fused8<false, false, false>);
  const size_t smem = few ? Plan<true>::SMEM : Plan<false>::SMEM;
  const int threads = few ? Plan<true>::THREADS : Plan<false>::THREADS;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const long long runs = static_cast<long long>(a.g.tiles_m) * ((a.g.tiles_n + a.g.run - 1) / a.g.run) * a.g.n_z;
  const int grid = 2 * static_cast<int>(runs < pairs ? runs : pairs);
  return launch8(kernel, grid, threads, smem, !a.clear, s, m.t, m.b, m.b_scale, m.c, a);
}

}  // namespace trimul
