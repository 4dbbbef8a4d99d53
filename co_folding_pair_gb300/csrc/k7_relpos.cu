// k7_relpos.cu -- relative position bias by buckets, and its table's gradient.
//
//   out[b,i,j,:] = base[b,i,j,:] + table[bucket(q_pos[b,i] - k_pos[b,j])]
//   dtable[n,:]  = sum of dout[b,i,j,:] over the pairs of bucket n
//
// Distances are clipped to [-M, M] (one-sided: [0, M]); LINEAR buckets are that,
// LOG buckets a table of 16-bit numbers over it, made when the plan is made.
// Both directions are one pass over B I J D elements (the forward writes them,
// and reads them if there is a base; the gradient reads them), so both are
// bound by memory.
#include <algorithm>

#include "pair_ops.cuh"

namespace trimul {

namespace {

template <typename T>
struct Vec;  // 16 bytes of T
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4 v, float (&f)[8]) { unpack8(v, f); }
  static __device__ __forceinline__ void unpack(const uint4 v, f2 (&f)[4]) {
    f[0] = unpack_bf162(v.x), f[1] = unpack_bf162(v.y), f[2] = unpack_bf162(v.z), f[3] = unpack_bf162(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) { return pack8(f); }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void unpack(const uint4 v, f2 (&f)[2]) {
    f[0] = pair2(__uint_as_float(v.x), __uint_as_float(v.y)), f[1] = pair2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// V elements of a table's row as fp32.
template <int V>
__device__ __forceinline__ void row_of(const float* p, float (&f)[V]) {
#pragma unroll
  for (int q = 0; q < V / 4; ++q) {
    const float4 v = reinterpret_cast<const float4*>(p)[q];
    f[4 * q] = v.x, f[4 * q + 1] = v.y, f[4 * q + 2] = v.z, f[4 * q + 3] = v.w;
  }
}
template <int V>
__device__ __forceinline__ void row_of(const __nv_bfloat16* p, float (&f)[V]) {
#pragma unroll
  for (int q = 0; q < V / 4; ++q) {
    const uint2 v = reinterpret_cast<const uint2*>(p)[q];
    f[4 * q] = bf16_lo(v.x), f[4 * q + 1] = bf16_hi(v.x), f[4 * q + 2] = bf16_lo(v.y), f[4 * q + 3] = bf16_hi(v.y);
  }
}

// PAIR layout: a thread has one place of 16 bytes in a pair and goes over pairs,
// kUnroll at a time, so that a warp's loads and stores are whole lines; the
// table comes from L1.  With a base it runs at a copy's rate (2 x 1024^2 x 128:
// 165 us, 0.97 of the copy), without one at that of a fill, which is less here
// (2048^2 x 256: 480 us, 4.47 TB/s; torch's fill of as much reaches 4.05).
template <typename T, typename Tab, int kUnroll>
__global__ void __launch_bounds__(256)
    k7_relpos_pair(RelposArgs a, const Tab* __restrict__ table, const T* base, T* out, uint32_t pairs, int per_pair) {
  constexpr int V = Vec<T>::n;
  const uint32_t at_once = blockDim.x / per_pair, c = threadIdx.x % per_pair;
  const uint32_t step = gridDim.x * at_once * kUnroll;
  // (pairs are below 2^31, and a step is at most 8 x 1024 of them an SM: p0 stays within 32 bits)
  for (uint32_t p0 = blockIdx.x * at_once * kUnroll + threadIdx.x / per_pair; p0 < pairs; p0 += step) {
    uint4 z[kUnroll];
    RelposPair at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t p = p0 + u * at_once;
      at[u].none();
      if (p >= pairs) continue;
      if (base) z[u] = __ldcs(reinterpret_cast<const uint4*>(base) + (static_cast<size_t>(p) * per_pair + c));
      uint32_t row, j;
      a.by_J.divmod(p, row, j);
      at[u].load(a, row, a.by_I.div(row) * a.J + j);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t p = p0 + u * at_once;
      if (p >= pairs) continue;
      const int k = at[u].bucket(a);
      float v[V] = {}, w[V];
      if (k >= 0) row_of<V>(table + static_cast<size_t>(k) * a.D + c * V, v);
      if (base) {
        Vec<T>::unpack(z[u], w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += w[e];
      }
      __stcs(reinterpret_cast<uint4*>(out) + (static_cast<size_t>(p) * per_pair + c), Vec<T>::pack(v));
    }
  }
}

// V buckets (16 bits each) that begin at word-aligned `ids` + V - m, from the two aligned groups of V around them.
template <int V>
__device__ __forceinline__ void shifted_ids(const uint16_t* ids, int m, uint32_t (&w)[V / 2]);
template <>
__device__ __forceinline__ void shifted_ids<8>(const uint16_t* ids, int m, uint32_t (&w)[4]) {
  const uint4 hi = *reinterpret_cast<const uint4*>(ids + 8);
  w[0] = hi.x, w[1] = hi.y, w[2] = hi.z, w[3] = hi.w;
  if (m == 0) return;
  const uint4 lo = *reinterpret_cast<const uint4*>(ids);
  uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  // by whole words first, m / 2 of them, then by half a word
  if (m & 4) {
#pragma unroll
    for (int i = 7; i >= 2; --i) x[i] = x[i - 2];
  }
  if (m & 2) {
#pragma unroll
    for (int i = 7; i >= 1; --i) x[i] = x[i - 1];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (m & 1) ? __funnelshift_l(x[i + 3], x[i + 4], 16) : x[i + 4];
}
template <>
__device__ __forceinline__ void shifted_ids<4>(const uint16_t* ids, int m, uint32_t (&w)[2]) {
  const uint2 hi = *reinterpret_cast<const uint2*>(ids + 4);
  w[0] = hi.x, w[1] = hi.y;
  if (m == 0) return;
  const uint2 lo = *reinterpret_cast<const uint2*>(ids);
  uint32_t x[4] = {lo.x, lo.y, hi.x, hi.y};
  if (m & 2) {
#pragma unroll
    for (int i = 3; i >= 1; --i) x[i] = x[i - 1];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = (m & 1) ? __funnelshift_l(x[i + 1], x[i + 2], 16) : x[i + 2];
}

// The buckets of plane positions [f0 - V, f0 + 32 V n) of batch b, in order:
// a tile of n segments, 16 bytes of elements a lane each.  `none` stands for
// what has no bucket: padding, and positions outside the plane.  The warps take
// pieces of 32 H positions, H = V or half of it.  Where all of a piece, early
// ones of a shifted plane among them, is in one bucket, as most are,
// whole[piece] is that bucket, else kMixed.
constexpr uint32_t kMixed = 0xffffffff;
template <int V, int H>
struct Piece {
  RelposPair pair[H + 1];
  __device__ __forceinline__ void load(const RelposArgs& a, uint32_t b, uint32_t f0, int piece, uint32_t plane) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int q = 0; q <= H; ++q) {
      const uint32_t f = f0 - V + (piece * H + q) * 32 + lane;  // what is before the plane comes out beyond its end
      pair[q].none();
      if (f < plane && (q < H || lane < V)) {
        uint32_t row, j;
        a.by_J.divmod(f, row, j);
        pair[q].load(a, b * a.I + row, b * a.J + j);
      }
    }
  }
  __device__ __forceinline__ void finish(const RelposArgs& a, int piece, int pieces, uint16_t none, uint16_t* ids,
                                         uint32_t* whole) const {
    const int lane = threadIdx.x % 32;
    uint32_t first = 0;
    bool same = true;
#pragma unroll
    for (int q = 0; q <= H; ++q) {
      const int k = pair[q].bucket(a);
      const uint32_t id = k < 0 ? none : k;
      if (q == 0) first = __shfl_sync(0xffffffffu, id, 0);
      same = same && (id == first || (q == H && lane >= V));
      if (q < H || (piece == pieces - 1 && lane < V)) ids[(piece * H + q) * 32 + lane] = static_cast<uint16_t>(id);
    }
    same = __all_sync(0xffffffffu, same);
    if (lane == 0) whole[piece] = same ? first : kMixed;
  }
};

// HEADS layout.  A block goes over tiles of a plane [I][J] of 16 bytes a
// thread: the buckets of a tile are worked out once, in shared memory, and
// every head of the block looks its values up by them, in its column of the
// table, in shared memory too; a segment of one bucket takes one look.  Planes
// of odd sizes begin anywhere within 16 bytes: a head's tile then begins up to
// V - 1 elements early, on a boundary, its buckets shifted alike, and only a
// plane's ends are written one by one.  4 x 8 x 515 x 1030 fp32: 15.4 us, 4.4
// TB/s; bf16, 2 x 16 x 1000^2: 16.9 us, 3.8 TB/s.  Both outputs fit L2, and DRAM
// is idle: what bounds them is the issue of the look-ups' instructions (three
// quarters of the slots in fp32, 0.71 in bf16) and the last, partial wave of blocks
// (1.3 waves).
constexpr int kHeadThreads = 256;
constexpr int kTableBytes = 64 * 1024;

template <typename T, typename Tab>
__global__ void __launch_bounds__(kHeadThreads)
    k7_relpos_heads(RelposArgs a, const Tab* __restrict__ table, const T* base, T* out, uint32_t plane,
                    FastDiv by_tiles, int heads) {
  constexpr int V = Vec<T>::n, kTile = kHeadThreads * V, kSegments = kHeadThreads / 32;
  extern __shared__ float tab[];  // [heads][rows + 1], the last of each 0
  __shared__ alignas(16) uint16_t ids[2][kTile + V];
  __shared__ uint32_t whole[2][kSegments];
  const int h0 = blockIdx.y * heads, n_heads = min(heads, a.D - h0), rows = a.rows + 1;
  const uint16_t none = static_cast<uint16_t>(a.rows);
  for (int n = threadIdx.x; n < rows * n_heads; n += kHeadThreads) {
    const int r = n / n_heads, q = n - r * n_heads;
    tab[q * rows + r] = r < a.rows ? to_f32(table[static_cast<size_t>(r) * a.D + h0 + q]) : 0.f;
  }
  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < by_tiles.d * a.B; tile += gridDim.x, turn ^= 1) {
    uint32_t b, t;
    by_tiles.divmod(tile, b, t);
    // two buffers: a warp that still works on the last tile reads the other one
    Piece<V, V> piece;  // one a warp
    piece.load(a, b, t * kTile, threadIdx.x / 32, plane);
    piece.finish(a, threadIdx.x / 32, kSegments, none, ids[turn], whole[turn]);
    __syncthreads();
    const uint32_t one = whole[turn][threadIdx.x / 32];
    const uint32_t first = t * kTile + threadIdx.x * V;
    const long long begin0 = (static_cast<long long>(b) * a.D + h0) * plane;
    int m = static_cast<int>(begin0 % V);
    const int m_step = static_cast<int>(plane % V);
    const T* z0 = base + begin0;
    T* o0 = out + begin0;
    const float* col = tab;
    const uint32_t whole_ends = plane < V ? 0u : plane - V + 1;  // all V of those that begin before it are in the plane
#pragma unroll 2
    for (int q = 0; q < n_heads; ++q, m = (m + m_step) % V, z0 += plane, o0 += plane, col += rows) {
      // the position in the plane of the first of V elements; what is before the plane is beyond its end without a sign
      const uint32_t n = first - m;
      if (first >= plane + m) continue;
      float v[V];
      if (one != kMixed) {
        v[0] = col[one];
#pragma unroll
        for (int e = 1; e < V; ++e) v[e] = v[0];
      } else {
        uint32_t w[V / 2];
        shifted_ids<V>(ids[turn] + threadIdx.x * V, m, w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = col[(e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu];
      }
      if (n < whole_ends) {
        if (base) {
          float z[V];
          Vec<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(z0 + n)), z);
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] += z[e];
        }
        __stcs(reinterpret_cast<uint4*>(o0 + n), Vec<T>::pack(v));
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (n + e < plane) o0[n + e] = from_f32<T>(base ? v[e] + to_f32(z0[n + e]) : v[e]);
      }
    }
  }
}

// ------------------------------------------------------------------ gradient
// Sums are kept in shared memory and written to global memory once a block;
// k7_relpos_sum adds the blocks' sums in order.  No atomics: every sum has one
// owner, so results do not depend on the order in which warps run.
//
// What makes these sums cheap is that neighbours share a bucket: all pairs
// farther than M, and in LOG buckets runs of near ones.  A run is added up in
// registers and goes to shared memory when it ends.

// Shared memory for a block's sums.  With the 1 KB that every block has besides
// it is one of the sizes that an SM can split its 256 KB by, and leaves 60 KB
// for L1, through which the loads on their way go: the next size leaves 28 KB,
// and cost the pair gradient a fifth of its rate when the two were compared
// (2048^2 x 256 with 66 rows: 415 us to 340, before the present order of its sums).
constexpr int kSumBytes = 195 * 1024;

// PAIR layout.  A warp has sums of its own, [rows][W channels], for one slice
// of at most W channels.  G lanes (16 bytes each) share a pair, so the warp
// takes 32 / G neighbouring pairs at a time, its slots, and kSteps of these
// make a batch.  One batch is worked on while the next one is on its way.
// A batch of one bucket is added up in registers, and joins the run of batches
// before it, as does a step of one bucket in a mixed batch; the pairs of other
// steps go to shared memory at once.  The buckets are worked out one pair a
// lane and handed round by shuffles.  2048^2 x 256 with four chains: 370 us, 5.8
// TB/s, bound by DRAM; 256^2 x 128: 12.7 us, most of it the sums' way through
// shared and global memory.  Every pair in a bucket of its own choosing, the
// worst there is, takes three times as long.
constexpr int kSteps = 8;
// Warps of a block: few lanes a pair means many pairs a lane, and registers for them.
constexpr int pair_warps(int G) { return G >= 4 ? 16 : 8; }

template <typename T, int G>
__global__ void __launch_bounds__(pair_warps(G) * 32)
    k7_relpos_grad_pair(RelposArgs a, const T* __restrict__ dout, float* part, uint32_t pairs, int slice, int S) {
  constexpr int V = Vec<T>::n, W = G * V, P = 32 / G, kBatch = P * kSteps, kPerLane = (kBatch + 31) / 32;
  constexpr int kBuffers = 2;
  extern __shared__ float4 smem4[];
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int slot = lane / G, c = (lane % G) * V;
  float* const sums = reinterpret_cast<float*>(smem4) + static_cast<size_t>(warp) * a.rows * W;
  for (int n = lane; n < a.rows * W / 4; n += 32) reinterpret_cast<float4*>(sums)[n] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
  // this warp's channels, and its block's range of batches
  const int c0 = (blockIdx.y * S + warp % S) * slice, width = min(slice, a.D - c0);
  const bool live = c < width;
  const uint32_t batches = (pairs + kBatch - 1) / kBatch;
  const uint32_t b0 = static_cast<uint32_t>(static_cast<unsigned long long>(batches) * blockIdx.x / gridDim.x);
  const uint32_t b1 = static_cast<uint32_t>(static_cast<unsigned long long>(batches) * (blockIdx.x + 1) / gridDim.x);
  const int streams = warps / S;

  uint4 buf[kBuffers][kSteps];
  RelposPair pos[kBuffers][kPerLane];
  // lanes past the slice read its first channels, into columns that nobody looks at
  const T* const mine = dout + c0 + (live ? c : 0);
  auto load = [&](uint32_t batch, uint4 (&to)[kSteps], RelposPair (&at)[kPerLane]) {
    if (batch >= b1) return;
    const uint32_t p0 = batch * kBatch;
    if (p0 + kBatch <= pairs) {
      const T* from = mine + static_cast<size_t>(p0 + slot) * a.D;
#pragma unroll
      for (int u = 0; u < kSteps; ++u, from += P * a.D) to[u] = __ldcs(reinterpret_cast<const uint4*>(from));
    } else {  // pairs past the end: the last one, without a bucket
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
        to[u] = *reinterpret_cast<const uint4*>(mine + static_cast<size_t>(min(p0 + u * P + slot, pairs - 1)) * a.D);
    }
#pragma unroll
    for (int q = 0; q < kPerLane; ++q) {
      const uint32_t p = p0 + (q * 32 + lane) % kBatch;
      at[q].none();
      if (p < pairs) {
        uint32_t row, j;
        a.by_J.divmod(p, row, j);
        at[q].load(a, row, a.by_I.div(row) * a.J + j);
      }
    }
  };
  // v joins the sums of bucket k, for the slots that say `on`
  auto add = [&](int k, const f2 (&v)[V / 2], bool on) {
    ulonglong2* const to = reinterpret_cast<ulonglong2*>(sums + k * W + c);
    if (on) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const ulonglong2 t = to[q];
        to[q] = make_ulonglong2(add2(t.x, v[2 * q]), add2(t.y, v[2 * q + 1]));
      }
    }
    __syncwarp();
  };
  int at = -1;  // the bucket of the run of batches
  f2 run[V / 2] = {};
  auto flush = [&] {
    if (at < 0) return;
#pragma unroll 1
    for (int k = 0; k < P; ++k) add(at, run, slot == k);
  };
  auto join = [&](int k, const f2 (&v)[V / 2]) {  // k and what it leads to is the same in all lanes
    if (k != at) {
      flush();
      at = k;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) run[e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) run[e] = add2(run[e], v[e]);
    }
  };
  auto take = [&](const uint4 (&from)[kSteps], const RelposPair (&pair)[kPerLane]) {
    int k_of[kPerLane];
#pragma unroll
    for (int q = 0; q < kPerLane; ++q) k_of[q] = pair[q].bucket(a);
    const int k0 = __shfl_sync(0xffffffffu, k_of[0], 0);
    bool one = k0 >= 0;
#pragma unroll
    for (int q = 0; q < kPerLane; ++q) one = one && k_of[q] == k0;
    f2 v[V / 2];
    if (__all_sync(0xffffffffu, one)) {
      f2 t[V / 2];
      Vec<T>::unpack(from[0], t);
#pragma unroll
      for (int u = 1; u < kSteps; ++u) {
        Vec<T>::unpack(from[u], v);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) t[e] = add2(t[e], v[e]);
      }
      join(k0, t);
      return;
    }
    // Pairs that share their step's bucket take turns, by their rank among
    // these (in bits 16 on); steps of one bucket join the run.
    constexpr unsigned step = P == 32 ? 0xffffffffu : (1u << (P % 32)) - 1;
    unsigned some[kPerLane], all[kPerLane];
#pragma unroll
    for (int q = 0; q < kPerLane; ++q) {
      const unsigned like = (__match_any_sync(0xffffffffu, k_of[q]) >> (lane / P * P)) & step;
      const int rank = __popc(like & ((1u << (lane % P)) - 1));
      some[q] = __ballot_sync(0xffffffffu, rank > 0 && k_of[q] >= 0);
      all[q] = __ballot_sync(0xffffffffu, like == step && k_of[q] >= 0);
      if (k_of[q] >= 0) k_of[q] |= rank << 16;
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int k = __shfl_sync(0xffffffffu, k_of[u * P / 32], (u * P + slot) % 32);
      Vec<T>::unpack(from[u], v);
      const int at_bit = u * P % 32;
      if ((all[u * P / 32] >> at_bit) & 1) {
        join(k & 0xffff, v);
      } else if (some[u * P / 32] & (step << at_bit)) {
#pragma unroll 1
        for (int turn = 0; __any_sync(0xffffffffu, k >> 16 >= turn); ++turn) add(k & 0xffff, v, k >> 16 == turn);
      } else {
        add(k, v, k >= 0);
      }
    }
  };

  uint32_t batch = b0 + warp / S;
#pragma unroll
  for (int q = 0; q < kBuffers; ++q) load(batch + q * streams, buf[q], pos[q]);
  while (batch < b1) {
#pragma unroll
    for (int q = 0; q < kBuffers; ++q) {
      if (batch < b1) {
        take(buf[q], pos[q]);
        load(batch + kBuffers * streams, buf[q], pos[q]);
        batch += streams;
      }
    }
  }
  flush();
  __syncthreads();
  const float* const all = reinterpret_cast<const float*>(smem4);
  float* const out = part + static_cast<size_t>(blockIdx.x) * a.rows * a.D;
  for (int q = 0; q < S; ++q) {
    const int from = (blockIdx.y * S + q) * slice, n_here = min(slice, a.D - from);
    for (int n = threadIdx.x; n < a.rows * W / 4; n += blockDim.x) {
      const int r = n * 4 / W, w = n * 4 % W;
      if (w >= n_here) continue;
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < streams; ++k) {
        const float4 v = reinterpret_cast<const float4*>(all + static_cast<size_t>(k * S + q) * a.rows * W)[n];
        t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
      }
      *reinterpret_cast<float4*>(out + static_cast<size_t>(r) * a.D + from + w) = t;
    }
  }
}

// HEADS layout.  A block goes over tiles of a plane [I][J]; the buckets of a
// tile are worked out once, in shared memory, and every warp adds up one
// head's part of the tile.  Each lane has sums of its own ([rows + 1][32
// lanes], the last row for what has no bucket), 16 bytes of neighbouring
// elements at a time; a segment of one bucket joins a run in registers, the
// elements of others go to shared memory at once.  Planes of odd sizes as in the
// forward.  2 x 16 x 1001^2 bf16: 28.8 us, 2.2 TB/s; bound by the instructions
// around each tile (its buckets, loads and the meeting of the warps), which take
// as long for any pattern of buckets.  (The same sums as a product with tiles of
// ones on the tensor cores took 24 to 29 us here and more for few heads.)
constexpr int kTileSteps = 8;
constexpr int kHeadsBytes = 218 * 1024;  // shared memory for a block's sums and buckets

template <typename T>
struct HeadTile {
  static constexpr int V = Vec<T>::n;
  static constexpr int part = kTileSteps * 32 * V;  // elements of a warp's part of a tile
};

template <typename T>
__global__ void __launch_bounds__(512)
    k7_relpos_grad_heads(RelposArgs a, const T* __restrict__ dout, float* partial, uint32_t plane, FastDiv by_tiles,
                         int heads) {
  constexpr int V = Vec<T>::n, kPart = HeadTile<T>::part;
  extern __shared__ float4 smem4[];
  let_next_begin();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int parts = warps / heads, tile_n = parts * kPart, own = (a.rows + 1) * 32;
  const int h = blockIdx.y * heads + warp % heads, my_part = warp / heads;
  const bool live = h < a.D;
  float* const sums = reinterpret_cast<float*>(smem4) + static_cast<size_t>(warp) * own;
  uint16_t* const ids0 = reinterpret_cast<uint16_t*>(reinterpret_cast<float*>(smem4) + static_cast<size_t>(warps) * own);
  __shared__ alignas(8) uint32_t whole0[2][2 * 16 * kTileSteps];
  for (int r = 0; r <= a.rows; ++r) sums[r * 32 + lane] = 0.f;
  const uint32_t tiles = by_tiles.d * a.B;
  const uint16_t none = static_cast<uint16_t>(a.rows);

  auto plane_of = [&](uint32_t b) { return HeadPlane(b, h, a.B, a.D, plane, V); };
  uint4 buf[kTileSteps];
  auto load = [&](uint32_t tile) {
    uint32_t b, t;
    by_tiles.divmod(tile, b, t);
    const HeadPlane p = plane_of(b);
    const T* const from = dout + p.at;
    const uint32_t first = t * tile_n + my_part * kPart + lane * V;
#pragma unroll
    for (int u = 0; u < kTileSteps; ++u) {
      const uint32_t n = first + u * 32 * V;
      buf[u] = make_uint4(0u, 0u, 0u, 0u);
      if (!live || n >= p.end) continue;
      if (n + V <= p.whole) {
        buf[u] = __ldcs(reinterpret_cast<const uint4*>(from + n));
      } else {
        alignas(16) T last[V] = {};
        for (int e = 0; e < V; ++e)
          if (n + e < p.end) last[e] = from[n + e];
        buf[u] = *reinterpret_cast<const uint4*>(last);
      }
    }
  };

  uint32_t at = none;
  float run = 0.f;
  int turn = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    uint32_t b, t;
    by_tiles.divmod(tile, b, t);
    load(tile);  // on its way while the buckets are worked out
    uint16_t* const ids = ids0 + turn * (tile_n + V);
    // two buffers: a warp that is still adding the last tile reads the other one
    for (int k = warp; k < 2 * parts * kTileSteps; k += warps) {
      Piece<V, V / 2> piece;
      piece.load(a, b, t * tile_n, k, plane);
      piece.finish(a, k, 2 * parts * kTileSteps, none, ids, whole0[turn]);
    }
    __syncthreads();
    if (!live) continue;
    const int m = plane_of(b).early;
#pragma unroll
    for (int u = 0; u < kTileSteps; ++u) {
      const uint2 halves = reinterpret_cast<const uint2*>(whole0[turn])[my_part * kTileSteps + u];
      const uint32_t one = halves.x == halves.y ? halves.x : kMixed;
      if (one != kMixed) {  // of the whole warp's elements
        f2 v[V / 2];
        Vec<T>::unpack(buf[u], v);
#pragma unroll
        for (int i = 1; i < V / 2; ++i) v[0] = add2(v[0], v[i]);
        const float2 s = split2(v[0]);
        if (one != at) {
          sums[at * 32 + lane] += run;
          at = one;
          run = 0.f;
        }
        run += s.x + s.y;
      } else {
        uint32_t w[V / 2];
        shifted_ids<V>(ids + my_part * kPart + u * 32 * V + lane * V, m, w);
        float v[V];
        Vec<T>::unpack(buf[u], v);
#pragma unroll
        for (int e = 0; e < V; ++e) sums[((e & 1) ? w[e / 2] >> 16 : w[e / 2] & 0xffffu) * 32 + lane] += v[e];
      }
    }
  }
  sums[at * 32 + lane] += run;
  __syncwarp();
  // the lanes' sums, added in a fixed order into lane 0's column; then the parts'
  for (int r = lane; r < a.rows; r += 32) {
    float t = 0.f;
    for (int l = 0; l < 32; ++l) t += sums[r * 32 + ((l + lane) & 31)];
    sums[r * 32] = t;
  }
  __syncthreads();
  for (int n = threadIdx.x; n < a.rows * heads; n += blockDim.x) {
    const int r = n / heads, q = n % heads, head = blockIdx.y * heads + q;
    if (head >= a.D) continue;
    float t = 0.f;
    for (int k = 0; k < parts; ++k)
      t += reinterpret_cast<const float*>(smem4)[static_cast<size_t>(k * heads + q) * own + r * 32];
    partial[(static_cast<size_t>(blockIdx.x) * a.rows + r) * a.D + head] = t;
  }
}

// The blocks' sums: 32 columns a block, eight groups of parts side by side.
__global__ void __launch_bounds__(256)
    k7_relpos_sum(const float* __restrict__ part, float* dtable, int n, int parts, int accumulate) {
  __shared__ float s[8][32];
  const int e = blockIdx.x * 32 + threadIdx.x % 32, g = threadIdx.x / 32;
  float t = 0.f;
  after_previous();
  if (e < n) {
#pragma unroll 8
    for (int k = g; k < parts; k += 8) t += part[static_cast<size_t>(k) * n + e];
  }
  s[g][threadIdx.x % 32] = t;
  __syncthreads();
  if (g != 0 || e >= n) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) t += s[k][threadIdx.x];
  dtable[e] = accumulate ? dtable[e] + t : t;
}

// How a gradient is split over blocks.
struct GradSplit {
  int warps, lanes, slice, slices, ranges, smem;
  int S;  // PAIR: slices of a block
};

// PAIR: a warp's slice is 64 channels where these divide D and ten warps' sums
// have room, else 32: more warps, and more pairs that meet in a bucket
// (1024^2 x 256, us, 64 to 32: 65 rows 101 to 100, LOG 32 rows 99 to 138, 66
// rows with eight warps 128 to 114; 2048^2 x 96: 170 to 141).  Narrower for long tables, whose sums
// leave room for few warps.  Slices are as even as 16-byte groups allow.
template <typename T>
GradSplit split_pair(int rows, long long pairs, int D, int num_sms) {
  constexpr int V = Vec<T>::n;
  GradSplit g;
  int W = V;
  while (W < D && W < 32 && rows * 2 * W * 4 * 6 <= kSumBytes) W *= 2;
  const int fit64 = std::min(pair_warps(64 / V), kSumBytes / (rows * 64 * 4));
  if (D % 64 == 0 && fit64 / (D / 64) * (D / 64) >= 10) W = 64;
  g.lanes = W / V;
  const int groups = D / V;  // of 16 bytes
  g.slices = (groups + g.lanes - 1) / g.lanes;
  g.slice = (groups + g.slices - 1) / g.slices * V;
  g.slices = (D + g.slice - 1) / g.slice;
  g.warps = std::min(pair_warps(g.lanes), kSumBytes / (rows * W * 4));
  g.S = 1;
  const long long batches = (pairs + 32 / g.lanes * kSteps - 1) / (32 / g.lanes * kSteps);
  // One block for all of a pair's slices reads whole rows, which DRAM serves
  // better, but writes sums of all channels a block: worth it once a warp has
  // some sixteen batches (when written, 2048^2 x 256: 479 us against 559; 256^2
  // x 128, with two batches a warp: 19.2 against 16.3).
  if (g.slices <= g.warps && batches >= 16ll * (g.warps / g.slices) * num_sms) {
    g.S = g.slices;
    g.slices = 1;
    g.warps = g.warps / g.S * g.S;
  }
  g.smem = g.warps * rows * W * 4;
  g.ranges = static_cast<int>(std::max<long long>(1, std::min<long long>((batches + g.warps / g.S - 1) / (g.warps / g.S), num_sms / g.slices)));
  return g;
}

// HEADS: one warp a head, several for a head's parts of a tile where there are few heads.
template <typename T>
GradSplit split_heads(int rows, int B, long long plane, int H, int num_sms) {
  constexpr int V = Vec<T>::n, kPart = HeadTile<T>::part;
  GradSplit g;
  constexpr int kMost = kHeadsBytes, kIds = 2 * (kPart + V) * 2;  // two buffers of a part's buckets
  const int own = (rows + 1) * 32 * 4;
  const int warps = std::max(1, std::min(16, (kMost - kIds) / own));
  g.slices = (H + warps - 1) / warps;
  g.lanes = (H + g.slices - 1) / g.slices;  // heads of a block
  int parts = static_cast<int>(std::max<long long>(1, std::min<long long>(warps / g.lanes, (plane + kPart - 1) / kPart)));
  while (parts > 1 && parts * (g.lanes * own + kIds) > kMost) --parts;
  g.warps = g.lanes * parts;
  g.slice = parts * kPart;
  g.smem = g.warps * own + 2 * (g.slice + V) * 2;
  const long long tiles = B * ((plane + V - 1 + g.slice - 1) / g.slice);
  g.ranges = static_cast<int>(std::max<long long>(1, std::min<long long>(tiles, num_sms / g.slices)));
  return g;
}

template <typename T>
GradSplit split(int rows, int B, int I, int J, int D, trimul_layout layout, int num_sms) {
  const long long plane = static_cast<long long>(I) * J;
  return layout == TRIMUL_LAYOUT_PAIR ? split_pair<T>(rows, B * plane, D, num_sms)
                                      : split_heads<T>(rows, B, plane, D, num_sms);
}

template <typename T, typename Tab>
cudaError_t forward(const RelposArgs& a, const void* table, const void* base, void* out, trimul_layout layout,
                    int num_sms, cudaStream_t s) {
  if (layout == TRIMUL_LAYOUT_PAIR) {
    const int per_pair = a.D / Vec<T>::n, at_once = 256 / per_pair;  // per_pair is at most 64
    const uint32_t pairs = static_cast<uint32_t>(a.B) * a.I * a.J;
    auto launch = [&](auto kernel, int unroll) {
      const long long blocks = (static_cast<long long>(pairs) + at_once * unroll - 1) / (at_once * unroll);
      kernel<<<static_cast<int>(std::min<long long>(blocks, 8ll * num_sms)), at_once * per_pair, 0, s>>>(
          a, static_cast<const Tab*>(table), static_cast<const T*>(base), static_cast<T*>(out), pairs, per_pair);
    };
    // four pairs a thread at a time where that leaves two blocks an SM (64^2 x 32: 1.9 us with one, 2.6 with four)
    if (pairs >= 8ll * at_once * num_sms)
      launch(k7_relpos_pair<T, Tab, 4>, 4);
    else
      launch(k7_relpos_pair<T, Tab, 1>, 1);
    return cudaGetLastError();
  }
  constexpr int V = Vec<T>::n, kTile = kHeadThreads * V;
  const uint32_t plane = static_cast<uint32_t>(a.I) * a.J;
  const long long tiles = (static_cast<long long>(plane) + V - 1 + kTile - 1) / kTile;
  // heads of a block: as many as have room for their columns of the table, fewer where that leaves SMs without work
  const int most = std::min(a.D, kTableBytes / ((a.rows + 1) * 4));
  int groups = static_cast<int>(std::max<long long>((a.D + most - 1) / most,
                                                    std::min<long long>(a.D, 4 * num_sms / (tiles * a.B))));
  const int heads = (a.D + groups - 1) / groups;
  groups = (a.D + heads - 1) / heads;
  const int grid = static_cast<int>(std::min<long long>(tiles * a.B, std::max(1, 8 * num_sms / groups)));
  cudaError_t e = allow_smem<k7_relpos_heads<T, Tab>>(kTableBytes);
  if (e != cudaSuccess) return e;
  k7_relpos_heads<T, Tab><<<dim3(grid, groups), kHeadThreads, heads * (a.rows + 1) * 4, s>>>(
      a, static_cast<const Tab*>(table), static_cast<const T*>(base), static_cast<T*>(out), plane,
      FastDiv(static_cast<uint32_t>(tiles)), heads);
  return cudaGetLastError();
}

template <typename T, int G>
cudaError_t grad_pair(const RelposArgs& a, const T* dout, const GradSplit& g, float* ws, cudaStream_t s) {
  cudaError_t e = allow_smem<k7_relpos_grad_pair<T, G>>(kSumBytes);
  if (e != cudaSuccess) return e;
  k7_relpos_grad_pair<T, G><<<dim3(g.ranges, g.slices), g.warps * 32, g.smem, s>>>(
      a, dout, ws, static_cast<uint32_t>(a.B) * a.I * a.J, g.slice, g.S);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const RelposArgs& a, const void* grad, trimul_layout layout, float* dtable, bool accumulate,
                     float* ws, int num_sms, cudaStream_t s) {
  const GradSplit g = split<T>(a.rows, a.B, a.I, a.J, a.D, layout, num_sms);
  const T* const dout = static_cast<const T*>(grad);
  cudaError_t e = cudaSuccess;
  if (layout == TRIMUL_LAYOUT_PAIR) {
    switch (g.lanes) {
      case 1: e = grad_pair<T, 1>(a, dout, g, ws, s); break;
      case 2: e = grad_pair<T, 2>(a, dout, g, ws, s); break;
      case 4: e = grad_pair<T, 4>(a, dout, g, ws, s); break;
      case 8: e = grad_pair<T, 8>(a, dout, g, ws, s); break;
      default: e = grad_pair<T, 16>(a, dout, g, ws, s); break;
    }
  } else {
    e = allow_smem<k7_relpos_grad_heads<T>>(kHeadsBytes);
    if (e != cudaSuccess) return e;
    const uint32_t plane = static_cast<uint32_t>(a.I) * a.J;
    const uint32_t tiles = static_cast<uint32_t>((plane + static_cast<long long>(Vec<T>::n) - 1 + g.slice - 1) / g.slice);
    k7_relpos_grad_heads<T><<<dim3(g.ranges, g.slices), g.warps * 32, g.smem, s>>>(a, dout, ws, plane, FastDiv(tiles), g.lanes);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const int n = a.rows * a.D;
  return launch_early(k7_relpos_sum, (n + 31) / 32, 256, s, ws, dtable, n, g.ranges, accumulate);
}

}  // namespace

cudaError_t launch_relpos_forward(const RelposArgs& a, const void* table, bool table_f32, const void* base, void* out,
                                  bool f32, trimul_layout layout, int num_sms, cudaStream_t s) {
  if (f32)
    return table_f32 ? forward<float, float>(a, table, base, out, layout, num_sms, s)
                     : forward<float, __nv_bfloat16>(a, table, base, out, layout, num_sms, s);
  return table_f32 ? forward<__nv_bfloat16, float>(a, table, base, out, layout, num_sms, s)
                   : forward<__nv_bfloat16, __nv_bfloat16>(a, table, base, out, layout, num_sms, s);
}

size_t relpos_backward_workspace(int rows, int B, int I, int J, int D, trimul_layout layout, bool f32, int num_sms) {
  const GradSplit g = f32 ? split<float>(rows, B, I, J, D, layout, num_sms) : split<__nv_bfloat16>(rows, B, I, J, D, layout, num_sms);
  return static_cast<size_t>(g.ranges) * rows * D * sizeof(float);
}

cudaError_t launch_relpos_backward(const RelposArgs& a, const void* dout, bool f32, trimul_layout layout,
                                   float* dtable, bool accumulate, float* ws, int num_sms, cudaStream_t s) {
  return f32 ? backward<float>(a, dout, layout, dtable, accumulate, ws, num_sms, s)
             : backward<__nv_bfloat16>(a, dout, layout, dtable, accumulate, ws, num_sms, s);
}

}  // namespace trimul
