// attention.cu — attention of one new token of each sequence over the paged key-value cache.
//
// For query head h over the positions j that it sees: s_j = scale (q . k_j) (capped when asked),
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m). The formula takes 2 G flops
// for each element of the cache (G query heads to a key head), so while the cache is read once the bound
// is HBM, and everything is arranged to keep enough bytes in flight. It is read once for each block of 8
// query heads to a key head (16 where G > 8 and heads are up to 128 wide), so again for the next block.
//
// Work: a row is one (sequence, key head, block of up to 8 NT query heads). Its positions are cut
// into units of 64, and the units of all rows are dealt to the CTAs of one wave in nearly equal runs,
// so ragged batches and single long sequences both fill the GPU. A CTA's run covers a part of a row,
// or parts of several (segments); a row that several CTAs share is joined by the last of them to
// arrive, in the order of the CTAs, so the result does not depend on who that is. No CTA waits for
// another.
//
// Within a segment the CTA's warps take tiles of 16 or 32 positions in turn; each streams its own
// through its own ring in shared memory with 16-byte asynchronous copies, and keeps its own running
// maximum, sum and outputs; the warps meet once, at the segment's end.
//
// Products run on the m16n8k16 matrix instructions, transposed: S^T = K Q^T and O^T = V^T P^T, so
// that the 16-row side is always positions or entries of the cache and the 8-column side the query
// heads. The 128 rows of tcgen05 would be full that way as well; up to 8 heads to a key head, where HBM
// is the bound, its rate would gain nothing. With more heads, and with 256-wide ones, the outputs'
// registers leave 8 to 12 warps on an SM, which tensor memory would free: not built.
// The order of a head's entries along the contraction is free, so a lane takes the 16 bytes that
// lie together in the cache as the fragment's entries and the query is laid out to match; for V the
// pairs of positions that a fragment wants are woven from two rows by byte permutes.
//
// Precision: cache elements are exact in bf16 (8-bit ones in fp16). fp32 queries and probabilities
// enter as three parts of 8 bits, which hold them, or in fp16 as two of 11. A remainder of 12 bits can
// meet the second of these, which then leaves 2^-23 of the value (a unit in fp32's last place; a third
// part of the queries cost 5 to 10% of the time). fp16 ends at 2^-24, so a head's largest query is
// brought below 2^15, probabilities are lifted by 2^12, and the second parts by another 2^12, in sums
// of their own: entries down to 2^-28 of the head's largest, and probabilities down to 2^-26 of the
// largest, are within 2^-23 of themselves, and smaller ones within 2^-51 and 2^-49 of the largest (0 to
// 1.5% of the time, 33 x 4099 positions 51.3 -> 52.0 us; without the second lift entries from 2^-17 of
// the largest on lose bits). The matrix instructions add with truncation, so sums over many tiles are
// kept outside of them. Against 64 bits the outputs are 2e-7 to 7e-7 off (2-norm), less than elementary
// fp32 operations.
//
// Measured on B200 (6.55 TB/s is a copy's rate): 131071 positions of 8 key heads 87 to 90 us, 6.0 to 6.2
// TB/s; a ragged batch of 64 up to 8192 113 to 116 us, 6.2 to 6.4 TB/s; 33 x 4099 positions of an 8-bit
// cache 52 to 53 us, 5.3 TB/s: there its products and their latency bound it, and the start and end of a
// CTA, about 3 and 1 us. One token of 32 heads over 517 positions 8.2 us: launch 2, start-up 2 (lengths, dealing, page
// table), copies and tiles 2, the join of nine parts 1. The ragged batch with 16 heads to a key head 156
// us (8-bit 114); with 71 heads on one key head, 64-wide, 56 us, eight times what one read would take.
#include <type_traits>

#include "layer.cuh"

namespace spax {

constexpr int kUnit = 64;  // positions in a unit of work, starting at a multiple of 64
constexpr int kJoin = 16;  // parts that are joined in one step (32 of 256-wide heads: 15.7 us, in two 13.1)
constexpr float kLow = 4096.0f;  // of the fp16 parts
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shapes of one instance: head_dim padded to DP, NT blocks of 8 query heads, tiles of 16 MT positions,
// WARPS warps with rings of SLOTS pieces (a tile's keys or its values; an odd number, so that the
// piece that is started before keys are used is keys again), CTAS resident on an SM.
template <int DP_, bool E4M3_, int NT_, int MT_, int WARPS_, int SLOTS_, int CTAS_>
struct AttnShape {
  static constexpr int DP = DP_, NT = NT_, HB = 8 * NT_, MT = MT_, TILE = 16 * MT_, SLOTS = SLOTS_, CTAS = CTAS_;
  static constexpr int WARPS = WARPS_, THREADS = WARPS * 32;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int PARTS = E4M3 ? 2 : 3;      // of a query entry, of a probability
  static constexpr float LOW = E4M3 ? kLow : 1.0f;  // the lower parts are held times this
  static constexpr int ROW = DP * ES;             // bytes of a row of a tile
  static constexpr int CH = ROW / 16;             // 16-byte chunks of a row
  static constexpr int PIECE = TILE * ROW;       // bytes of a tile's keys (or values)
  static constexpr int AHEAD = (SLOTS - 1) / 2;   // tiles between a copy's start and its use
  static constexpr int RING = WARPS * SLOTS * PIECE;
  static_assert(SLOTS % 2 == 1 && SLOTS >= 3);
  static constexpr int KS = DP / 16;              // k steps of a score
  // Units of the shortest run, which has a tile for each warp (8-bit 128-wide, 512 positions: 8.0 us in
  // runs of 2 units, 9.2 in runs of 1, whose second pair of warps had nothing).
  static constexpr int LEAST = (WARPS * TILE + kUnit - 1) / kUnit;
  // Units of the dealing that a row counts for beside its own: the start-up and the end of a segment
  // take about as long as the copies of 64 KB at a CTA's share of the bandwidth.
  static constexpr int EXTRA = 512 / ROW > 1 ? 512 / ROW : 1;
  static constexpr int SMEM = RING + KS / 2 * PARTS * NT * 512;  // and the query's parts
  static constexpr int OS = DP + 4;               // row stride of the warps' outputs at the join
  static_assert(WARPS * HB * OS * 4 <= RING, "the join's buffer overlays the ring");
  static_assert(CTAS * (SMEM + 3 * 1024) <= 228 * 1024, "shared memory of the resident CTAs");
};

// d = a b + c on the matrix unit; ZERO: d = a b.
template <bool E4M3, bool ZERO>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t* a, uint32_t b0,
                                         uint32_t b1) {
  const float c0 = ZERO ? 0.0f : d[0], c1 = ZERO ? 0.0f : d[1], c2 = ZERO ? 0.0f : d[2],
              c3 = ZERO ? 0.0f : d[3];
  if constexpr (E4M3)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
}

// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// Four 8-bit elements as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t* low, uint32_t* high) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(*low), "=r"(*high)
      : "r"(w));
}

__device__ __forceinline__ void scale_pair(float& x, float& y, float by) {
  const f2 r = ffma2(f2{x, y}, f2{by, by}, f2{0.0f, 0.0f});
  x = r.x, y = r.y;
}

// (x, y) as a pair in the matrix type, and what the pair leaves of them (times kLow for fp16).
template <bool E4M3>
__device__ __forceinline__ uint32_t take_part(float& x, float& y) {
  uint32_t d;
  if constexpr (E4M3) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    const __half2 h = *reinterpret_cast<const __half2*>(&d);
    scale_pair(x, y, kLow);
    const f2 left = ffma2(f2{__low2float(h), __high2float(h)}, f2{-kLow, -kLow}, f2{x, y});
    x = left.x, y = left.y;
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    x -= __uint_as_float(d << 16);
    y -= __uint_as_float(d & 0xFFFF0000u);
  }
  return d;
}

// A token's reads of the cache are the first to leave L2 again. Else 67 MB of it push out what the
// projections around the call keep there (their code, the activations, their workspaces): a
// Llama-2-7B layer at a context of 4096 takes 109 us a token then and 96 so, the attention alone
// 116 and 113 (ragged batch of 64 up to 8192). Where blocks of heads read it again the mark costs
// nothing on the whole (-4 to +5% without it over nine batches of 2 to 8 blocks).
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0), "l"(policy));
}

// Pairs of bf16 elements with 0 in place of an infinity: what the lower parts of a query or probability
// multiply in a careful pass. Such a part can be zero or of the other sign, and an infinity times it
// would turn the infinity that the first part gives into NaN (so would sums of the largest finite value).
__device__ __forceinline__ void finite_pairs(const uint32_t (&a)[4], uint32_t (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = a[k] & ~__vcmpeq2(a[k] & 0x7FFF7FFFu, 0x7F807F80u);
}

// tanh without branches, within a few ulp: (1 - u) / (1 + u) with u = e^(-2|x|), and below 0.4, where
// that difference cancels, the odd Taylor series to x^13 (the next term is below 2^-25 of x there).
__device__ __forceinline__ float tanh_flat(float x) {
  const float a = fabsf(x), u = exp2_ftz(-2.0f * kLog2e * a);
  const float big = copysignf(__fdividef(1.0f - u, 1.0f + u), x);
  const float y = x * x;
  float p = 21844.0f / 6081075.0f;
  p = fmaf(p, y, -1382.0f / 155925.0f);
  p = fmaf(p, y, 62.0f / 2835.0f);
  p = fmaf(p, y, -17.0f / 315.0f);
  p = fmaf(p, y, 2.0f / 15.0f);
  p = fmaf(p, y, -1.0f / 3.0f);
  return a < 0.4f ? fmaf(x * y, p, x) : big;
}

struct AttnArgs {
  AttnLaunch a;
  uint32_t page_mul;  // position / page_size = page_size == 1 ? position : umulhi(position, mul) >> shift
  int page_shift;
  int row_heads;      // query heads to a key head
  int blocks;         // blocks of HB query heads to a key head
  bool page16;        // 16 positions from a multiple of 16 are on one page
  float* part;        // [2 CTAs][HB][DP] outputs of shared rows
  float2 *part_ml, *part_ml2;  // [2 CTAs][HB] their maxima and sums, and those of joined groups
  uint32_t *tickets, *tickets2;  // [2 CTAs] each, zero at rest
};

template <class S>
struct Attn {
  // Positions [lo, len) of a sequence, by the window.
  static __device__ __forceinline__ int clipped_len(const AttnArgs& g, int seq, bool* bad) {
    const int len = g.a.lens[seq];
    *bad = len < 0 || len > g.a.max_pages * g.a.cache.page_size;
    return *bad ? 0 : len;
  }
  static __device__ __forceinline__ int first_seen(const AttnArgs& g, int len) {
    return g.a.prm.window > 0 ? max(0, len - g.a.prm.window) : 0;
  }
  static __device__ __forceinline__ int units_of(const AttnArgs& g, int len) {
    return (len + kUnit - 1) / kUnit - first_seen(g, len) / kUnit;
  }

  static __device__ __forceinline__ int page_of(const AttnArgs& g, int pos) {
    return g.page_shift < 0 ? pos : (int)(__umulhi((uint32_t)pos, g.page_mul) >> g.page_shift);
  }
};

// Counts this CTA in: true for the last of n, which also readies the ticket for the next call. The
// parts that the others wrote before are visible to every thread of it.
__device__ __forceinline__ bool arrive(uint32_t* ticket, int n, bool* is_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    // releases what the barrier has gathered of this CTA, acquires what the others released
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
    *is_last = before == (uint32_t)(n - 1);
    if (*is_last) *ticket = 0;
  }
  __syncthreads();
  return *is_last;
}

// One head's entries of a row, joined: written as they are to a slot (the maximum and sum to ml), or
// divided to the output.
template <class S>
__device__ __forceinline__ void put_row(const AttnArgs& g, float2* ml, int slot, long long at, int h, int d,
                                        float4 v, float M, float L) {
  if (slot >= 0) {
    __stcg(reinterpret_cast<float4*>(g.part + ((long long)slot * S::HB + h) * S::DP + d), v);
    if (d == 0) __stcg(ml + slot * S::HB + h, make_float2(M, L));
  } else {
    const float inv = L == 0.0f ? 0.0f : g.a.cache.v_scale / L;
    if (L == 0.0f) v = make_float4(0, 0, 0, 0);
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    *reinterpret_cast<float4*>(g.a.out + (at + h) * g.a.cache.head_dim + d) = v;
    if (d == 0 && g.a.lse) g.a.lse[at + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

// The slots of a row's parts in their order.
struct Parts {
  int first, next, step;
  __device__ __forceinline__ long long slot(int k) const { return k == 0 ? first : next + k * step; }
};

// Joins n parts of a row in their order: a thread takes the maxima, sums and entries of N parts for E
// of its quads at a time, all in flight at once, since each go costs a round trip to L2. A slot that is
// joined to may be one of the parts: an entry is read and written by one thread alone, while the
// maximum and sum, which several threads read, go to another array (the second step's).
template <class S, int N, int E>
__device__ __forceinline__ void join(const AttnArgs& g, const float2* from_ml, int heads, int n, Parts parts,
                                     int to, long long at) {
  const int quads = g.a.cache.head_dim / 4, all = heads * quads;
  for (int e0 = threadIdx.x; e0 < all; e0 += E * S::THREADS) {
    int h[E], d[E];
    float4 v[E];
    float M[E], L[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int e = e0 + j * S::THREADS < all ? e0 + j * S::THREADS : e0;  // past the end: its first again
      h[j] = e / quads, d[j] = (e - h[j] * quads) * 4;
      v[j] = make_float4(0, 0, 0, 0);
      M[j] = -INFINITY, L[j] = 0.0f;
    }
    for (int k = 0; k < n; k += N) {
      float4 t[E][N];
      float2 ml[E][N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const long long slot = parts.slot(k + i);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          ml[j][i] = make_float2(-INFINITY, 0.0f);
          t[j][i] = make_float4(0, 0, 0, 0);
          if (k + i < n) {
            ml[j][i] = __ldcg(from_ml + slot * S::HB + h[j]);
            t[j][i] = __ldcg(reinterpret_cast<const float4*>(g.part + (slot * S::HB + h[j]) * S::DP + d[j]));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float top = M[j];
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, ml[j][i].x);  // drops a NaN: its sum is NaN too
        const float fade = M[j] == -INFINITY ? 0.0f : exp2_ftz(M[j] - top);
        L[j] *= fade;
        v[j].x *= fade, v[j].y *= fade, v[j].z *= fade, v[j].w *= fade;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float f = ml[j][i].x == -INFINITY ? 0.0f : exp2_ftz(ml[j][i].x - top);
          L[j] += f * ml[j][i].y;
          v[j].x += f * t[j][i].x, v[j].y += f * t[j][i].y, v[j].z += f * t[j][i].z, v[j].w += f * t[j][i].w;
        }
        M[j] = top;
      }
    }
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (e0 + j * S::THREADS < all) put_row<S>(g, g.part_ml2, to, at, h[j], d[j], v[j], M[j], L[j]);
  }
}
template <class S>
__device__ __forceinline__ void join(const AttnArgs& g, const float2* from_ml, int heads, int n, Parts parts, int to,
                                     long long at) {
  // Two quads at a time where a row has more than one for each thread; 16 parts of one fill the
  // registers. Measured on B200, 8 query heads, 512 positions (8 parts): 256-wide 10.6 us, 11.7 with
  // 16 places for parts and one quad at a time; 128-wide 7.6 and 9.1.
  constexpr int E = S::HB * S::DP / 4 > S::THREADS ? 2 : 1;
  if (n <= 4)
    join<S, 4, E>(g, from_ml, heads, n, parts, to, at);
  else if (n <= 8)
    join<S, 8, E>(g, from_ml, heads, n, parts, to, at);
  else
    join<S, 16, 1>(g, from_ml, heads, n, parts, to, at);
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS) attention_kernel(const AttnArgs g) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int prefix[S::WARPS], start_base, start_seq;
  __shared__ float2 warp_ml[S::WARPS][S::HB];
  __shared__ bool is_last;
  using A = Attn<S>;
  constexpr int DP = S::DP, NT = S::NT, HB = S::HB, T = S::THREADS, W = S::WARPS,
                MT = S::MT, TILE = S::TILE;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int r = lane >> 2, c = lane & 3;
  const int b = blockIdx.x;
  const spax_kv_cache& C = g.a.cache;
  const int D = C.head_dim, n_seq = g.a.n_seq;
  const int chunks = D * S::ES / 16;
  const int rows_of_seq = C.n_kv_heads * g.blocks;

  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share ------------------------------------------------------------------------
  // Where a run length gives every row whole CTAs of its own within the wave (runs start at row
  // starts, the last of a row may be shorter), that is taken: one segment, one start-up and one
  // join for each CTA. Else all units are dealt in equal runs across row ends.
  auto len_at = [&](int s) {
    bool bad;
    return s < n_seq ? A::clipped_len(g, s, &bad) : 0;
  };
  // Up to 128 sequences: every warp for itself, 1 or kOwn to a lane, in registers, without barriers.
  constexpr int kOwn = 4;
  const bool few = n_seq <= 32 * kOwn;
  const int per = n_seq <= 32 ? 1 : few ? kOwn : (n_seq + T - 1) / T, s0 = (few ? lane : tid) * per;
  int own_len[kOwn], own_units[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    own_len[k] = few && k < per ? len_at(n_seq == 1 ? 0 : s0 + k) : 0;
    own_units[k] = A::units_of(g, own_len[k]);
  }
  auto units_at = [&](int s) { return A::units_of(g, len_at(s)); };
  auto total = [&](auto f) -> int {  // sum of f(units) over the sequences
    unsigned x = 0;
    if (n_seq == 1) return f(own_units[0]);  // every lane has it
    if (few) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k)
        if (k < per) x += f(own_units[k]);
      return (int)__reduce_add_sync(~0u, x);
    }
    for (int k = 0; k < per; ++k) x += f(units_at(s0 + k));
    x = __reduce_add_sync(~0u, x);
    __syncthreads();
    if (lane == 0) prefix[warp] = (int)x;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < W; ++w) all += prefix[w];
    return all;
  };
  int U = rows_of_seq * total([](int u) { return u; });
  int B = min((int)gridDim.x, U);
  int extra = 0;
  int run = 0;  // units in a run of the first kind
  if (U > 0) {
    const int rows = rows_of_seq * total([](int u) { return u > 0; });
    if (2 * rows <= (int)gridDim.x) {
      run = max(S::LEAST, (U + B - 1) / B);
      // a run may be this much longer than equal runs before their row ends cost less
      const int most = run + max(6, run / 16);
      const int more = few ? max(1, run / 16) : (most - run) / 2;
      for (;; run += more) {
        const int n = rows_of_seq * total([run](int u) { return run == 1 ? u : (u + run - 1) / run; });
        if (n <= (int)gridDim.x) {
          B = n;
          break;
        }
        if (run >= most) {
          run = 0;
          break;
        }
      }
    }
    if (!run) {
      extra = S::EXTRA;
      U += rows * extra;
    }
  }
  // Rows that see nothing, and lengths to report: after this CTA's share.
  auto leftovers = [&] {
    if (b == 0) {
      bool any_bad = false;
      for (int k = tid; k < n_seq; k += T) {
        bool bad;
        A::clipped_len(g, k, &bad);
        any_bad |= bad;
      }
      if (any_bad) record_status(g.a.status, SPAX_ERR_INDEX);
    }
    for (int s = b; s < n_seq; s += gridDim.x) {
      if (units_at(s) != 0) continue;
      for (int i = tid; i < g.a.n_heads * D; i += T) g.a.out[(long long)s * g.a.n_heads * D + i] = 0.0f;
      if (g.a.lse)
        for (int i = tid; i < g.a.n_heads; i += T) g.a.lse[(long long)s * g.a.n_heads + i] = -INFINITY;
    }
  };
  if (b >= B) {
    leftovers();
    return;
  }

  // CTA k's share is [start_of(k), start_of(k + 1)) of the units, floor(U k / B), or run k; the
  // sequence of its first unit (run), and the units (runs) before that sequence
  auto start_of = [&](int k) { return run ? k : U / B * k + U % B * k / B; };
  const int begin = start_of(b), end = start_of(b + 1);
  auto weight = [&](int u) { return rows_of_seq * (run ? (u + run - 1) / run : u ? u + extra : 0); };
  int seq = 0, base = 0, len = own_len[0];
  if (n_seq > 1) {
    int sum = 0;
    if (few) {
#pragma unroll
      for (int k = 0; k < kOwn; ++k)
        if (k < per) sum += weight(own_units[k]);
    } else {
      for (int k = 0; k < per; ++k) sum += weight(units_at(s0 + k));
    }
    int x = sum;  // inclusive scan
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (few) {
      const int there = __popc(__ballot_sync(~0u, x <= begin));  // the lane that has it
      int at = x - sum, k = 0, own = own_len[0];
#pragma unroll
      for (int i = 0; i + 1 < kOwn; ++i) {
        if (per == 1) break;
        const int w = weight(own_units[i]);
        if (k == i && begin >= at + w) {
          at += w;
          ++k;
          own = own_len[i + 1];
        }
      }
      seq = __shfl_sync(~0u, s0 + k, there);
      base = __shfl_sync(~0u, at, there);
      len = __shfl_sync(~0u, own, there);
    } else {
      __syncthreads();
      if (lane == 31) prefix[warp] = x;
      __syncthreads();
      for (int w = 0; w < warp; ++w) x += prefix[w];
      if (x - sum <= begin && begin < x) {
        int at = x - sum, s = s0;
        for (; s + 1 < n_seq; ++s) {
          const int n = weight(units_at(s));
          if (begin < at + n) break;
          at += n;
        }
        start_seq = s;
        start_base = at;
      }
      __syncthreads();
      seq = start_seq;
      base = start_base;
      len = len_at(seq);
    }
  }

  const uint32_t ring = smem_u32(smem) + warp * (S::SLOTS * S::PIECE);
  const uint32_t qsm = smem_u32(smem) + S::RING;

  for (int x = begin; x < end;) {
    const int units = A::units_of(g, len);
    if (units == 0) {  // an empty sequence between two others
      if (++seq >= n_seq) break;  // (only if lengths change under the call)
      len = len_at(seq);
      continue;
    }
    const int y = x - base;
    // what the row counts for
    const int runs = run == 1 ? units : run ? (units + run - 1) / run : units + extra;
    const int row = runs == 1 ? y : y / runs, r0 = y - row * runs;
    const int u0 = run ? r0 * run : max(0, r0 - extra);
    const int u1 = run ? min(units, u0 + run) : min(units, r0 - extra + (end - x));
    const int row_begin = base + row * runs + extra;  // the first unit's place
    // the share ends before the row's first unit (or lengths change under the call)
    if (u1 <= u0 || row >= rows_of_seq) break;
    const int kvh = g.blocks == 1 ? row : row / g.blocks, hb = row - kvh * g.blocks;
    const int heads = min(HB, g.row_heads - hb * HB);   // real query heads of this block
    const int head0 = kvh * g.row_heads + hb * HB;
    const int lo = A::first_seen(g, len);  // positions [t0, t1), of which those from lo are seen
    const int t0 = (lo / kUnit + u0) * kUnit;
    const int t1 = min(len, t0 + (u1 - u0) * kUnit);
    const int32_t* table = g.a.table + (long long)seq * g.a.max_pages;
    const uint8_t* kpool = static_cast<const uint8_t*>(C.d_k) + kvh * C.head_stride * S::ES;
    const uint8_t* vpool = static_cast<const uint8_t*>(C.d_v) + kvh * C.head_stride * S::ES;

    // ---- the query's parts, and the factors from a product to an exponent of two -----------------
    // k steps 2 i and 2 i + 1 of part p, block nt lie together: lane l's two fragments in 16 bytes.
    float f1[NT][2], f2;
    // entries of this lane's head for k step ks
    auto query = [&](int nt, int ks) {
      const int h = nt * 8 + r;
      const int d = S::E4M3 ? 64 * (ks / 4) + 16 * c + 4 * (ks % 4) : 32 * (ks / 2) + 8 * c + 4 * (ks % 2);
      return h < heads && d < D ? *reinterpret_cast<const float4*>(g.a.q + seq * g.a.q_stride + (head0 + h) * D + d)
                                : make_float4(0, 0, 0, 0);
    };
    constexpr int PAIRS = (S::KS / 2 + W - 1) / W;  // this warp prepares pairs warp, warp + W, ...
    constexpr int HELD = S::E4M3 ? S::KS : 2 * PAIRS;  // 8-bit caches need a head's largest entry
    float4 held[NT][HELD];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < HELD; ++k) held[nt][k] = query(nt, S::E4M3 ? k : 2 * (k / 2 * W + warp) + k % 2);
    auto prepare_query = [&] {
      const float cap = g.a.prm.softcap;
      f2 = cap * kLog2e;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float up = 1.0f, down = 1.0f;
        if constexpr (S::E4M3) {
          // fp16 parts: the head's largest entry is brought to [2^14, 2^15) (from 2^-86 on)
          float top = 0.0f;
#pragma unroll
          for (int ks = 0; ks < S::KS; ++ks) {
            const float4 v = held[nt][ks];
            top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const int e = (int)(__float_as_uint(top) >> 23) - 127;  // -127: zero or subnormal, 128: inf
          if (e < 128) {
            const int k = min(100, 14 - e);
            up = __uint_as_float((uint32_t)(k + 127) << 23);
            down = __uint_as_float((uint32_t)(127 - k) << 23);
          }
        }
        auto put = [&](int pair, float4 v, float4 w) {
          v.x *= up, v.y *= up, v.z *= up, v.w *= up;
          w.x *= up, w.y *= up, w.z *= up, w.w *= up;
#pragma unroll
          for (int p = 0; p < S::PARTS; ++p) {
            const uint32_t x0 = take_part<S::E4M3>(v.x, v.y), x1 = take_part<S::E4M3>(v.z, v.w);
            const uint32_t y0 = take_part<S::E4M3>(w.x, w.y), y1 = take_part<S::E4M3>(w.z, w.w);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             qsm + ((pair * S::PARTS + p) * NT + nt) * 512 + lane * 16),
                         "r"(x0), "r"(x1), "r"(y0), "r"(y1));
          }
        };
        if constexpr (S::E4M3) {
#pragma unroll
          for (int pair = 0; pair < S::KS / 2; ++pair)
            if (pair % W == warp) put(pair, held[nt][2 * pair], held[nt][2 * pair + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < PAIRS; ++i)
            if (i * W + warp < S::KS / 2) put(i * W + warp, held[nt][2 * i], held[nt][2 * i + 1]);
        }
        // the columns of a score fragment are heads 2c, 2c + 1
        const float f = g.a.prm.scale * C.k_scale * down * (cap > 0.0f ? 1.0f / cap : kLog2e);
        f1[nt][0] = __shfl_sync(~0u, f, (2 * c) * 4);
        f1[nt][1] = __shfl_sync(~0u, f, (2 * c + 1) * 4);
      }
      __syncthreads();
    };

    // ---- this warp's tiles: tile i starts at t0 + (i * W + warp) * TILE ---------------------------
    // Exponents are taken from a base that trails the maximum by up to kSlack powers of two (it moves
    // only when a score passes it by more), and fp16 probabilities are lifted by 2^12 so that their
    // parts stay normal numbers (and their sums are lowered again, exactly, at the end).
    constexpr float kSlack = S::E4M3 ? 3.0f : 8.0f, kLift = S::E4M3 ? 12.0f : 0.0f,
                    kDrop = S::E4M3 ? 1.0f / 4096.0f : 1.0f;
    const int tiles = (t1 - t0 + TILE - 1) / TILE;
    const int mine = tiles > warp ? (tiles - warp + W - 1) / W : 0;
    const int first = t0 + warp * TILE;
    float m[NT][2], l[NT][2], o[NT][DP / 16][4];

    auto stream = [&](auto careful) {
      constexpr bool CAREFUL = decltype(careful)::value;
      const int mine_at = lane & (TILE - 1);  // this lane's position in a tile
      auto page_entry = [&](int i) {  // the table's entry for the lane's position of tile i
        int pos = first + i * (W * TILE) + (g.page16 ? mine_at & 16 : mine_at);
        return i < mine ? table[A::page_of(g, min(pos, t1 - 1))] : 0;
      };
      // Where the rows of tile i are, and which of its positions are seen.
      struct Place {
        long long off[MT];  // one page for each 16: pool offset of this lane's chunk of its first row;
                            // else off[0]: of this lane's position, or -1
        uint32_t bits;
        bool plain;
      };
      constexpr uint32_t kAll = TILE == 32 ? ~0u : (1u << TILE) - 1;
      constexpr int RPI = 32 / S::CH;  // rows of a copy step
      const int row0 = lane / S::CH, ch = lane % S::CH;
      auto place = [&](int i, int page) {
        Place at;
        at.off[0] = -1;
        at.bits = 0;
        at.plain = false;
        if (i >= mine) return at;
        const int pos0 = first + i * (W * TILE), pos = pos0 + (g.page16 ? mine_at & 16 : mine_at);
        const bool real_page = (uint32_t)page < (uint32_t)C.n_pages;
        long long off = (page * C.page_stride +
                         (long long)(pos - A::page_of(g, pos) * C.page_size) * C.token_stride) * S::ES;
        if (g.page16 && D == DP && pos0 >= lo && pos0 + TILE <= t1 && __all_sync(~0u, real_page)) {
          const long long own = (row0 * C.token_stride) * S::ES + ch * 16;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) at.off[mt] = (MT == 1 ? off : __shfl_sync(~0u, off, 16 * mt)) + own;
          at.bits = kAll;
          at.plain = true;
        } else {
          const int me = pos0 + mine_at;
          if (g.page16) off += (long long)(mine_at & 15) * C.token_stride * S::ES;
          const bool seen = me >= lo && me < t1;
          if (seen && !real_page) record_status(g.a.status, SPAX_ERR_INDEX);
          at.off[0] = seen && real_page ? off : -1;
          at.bits = __ballot_sync(~0u, at.off[0] >= 0) & kAll;
        }
        return at;
      };
      // Starts the copies of a tile's keys or values. Rows are 16-byte chunks, placed so that the
      // fragments' loads spread over the banks: keys with rows of unlike parity in different halves,
      // values with pairs of rows apart.
      const long long step = RPI * C.token_stride * S::ES;
      const uint64_t policy = evict_first();
      auto issue = [&](const Place& at, bool real_tile, bool keys, int slot) {
        if (real_tile) {
          const uint32_t piece = ring + slot * S::PIECE;
          const uint8_t* pool = keys ? kpool : vpool;
          auto spot = [&](int row_) {
            const int to = S::CH >= 8 ? (keys ? ch ^ ((row_ & 1) << 2) : ch ^ (((row_ >> 1) & 3) << 1))
                                      : (keys ? ch : ch ^ (((row_ >> 1) & 1) << 1));
            return piece + row_ * S::ROW + to * 16;
          };
          if (at.plain) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint8_t* src = pool + at.off[mt];
#pragma unroll
              for (int k = 0; k < 16 / RPI; ++k) {
                cp16(spot(mt * 16 + k * RPI + row0), src, true, policy);
                src += step;
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < TILE / RPI; ++k) {
              const long long row_off = __shfl_sync(~0u, at.off[0], k * RPI + row0);
              const bool real = row_off >= 0 && ch < chunks;
              cp16(spot(k * RPI + row0), pool + (real ? row_off + ch * 16 : 0), real, policy);
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      auto next_slot = [](int slot) { return slot + 1 == S::SLOTS ? 0 : slot + 1; };

      uint32_t seen[S::AHEAD];
      int page = page_entry(0), fill = 0, use = 0;
#pragma unroll
      for (int i = 0; i < S::AHEAD; ++i) {
        const int next = page_entry(i + 1);
        const Place at = place(i, page);
        seen[i] = at.bits;
        issue(at, i < mine, true, 2 * i);
        issue(at, i < mine, false, 2 * i + 1);
        page = next;
      }
      fill = 2 * S::AHEAD;
      if constexpr (!CAREFUL) prepare_query();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
      }
      for (int i = 0; i < mine; ++i) {
        const int next = page_entry(i + S::AHEAD + 1);
        const Place ahead = place(i + S::AHEAD, page);
        page = next;
        const uint32_t here = seen[0];
#pragma unroll
        for (int k = 0; k + 1 < S::AHEAD; ++k) seen[k] = seen[k + 1];
        seen[S::AHEAD - 1] = ahead.bits;
        issue(ahead, i + S::AHEAD < mine, true, fill);
        fill = next_slot(fill);
        asm volatile("cp.async.wait_group %0;" ::"n"(S::SLOTS - 1) : "memory");
        __syncwarp();
        const uint32_t ks_at = ring + use * S::PIECE;
        use = next_slot(use);

        // scores: one chain for the first part of the query, one for the others
        float acc[MT][NT][2][4];
        auto step = [&](int pair, const uint32_t(&x)[MT][2][4]) {
          uint32_t fin[MT][2][4];
          if constexpr (CAREFUL) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              finite_pairs(x[mt][0], fin[mt][0]);
              finite_pairs(x[mt][1], fin[mt][1]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = S::PARTS - 1; p >= 0; --p) {
              const uint4 v = lds128(qsm + ((pair * S::PARTS + p) * NT + nt) * 512 + lane * 16);
              const bool low = CAREFUL && p > 0;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float(&d)[4] = acc[mt][nt][p == 0 ? 0 : 1];
                if (pair == 0 && (p == 0 || p == S::PARTS - 1))
                  mma16816<S::E4M3, true>(d, low ? fin[mt][0] : x[mt][0], v.x, v.y);
                else
                  mma16816<S::E4M3, false>(d, low ? fin[mt][0] : x[mt][0], v.x, v.y);
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma16816<S::E4M3, false>(acc[mt][nt][p == 0 ? 0 : 1], low ? fin[mt][1] : x[mt][1], v.z, v.w);
            }
        };
#pragma unroll
        for (int j = 0; j < S::CH / 4; ++j) {
          const int kc = S::CH >= 8 ? (c + 4 * j) ^ ((r & 1) << 2) : c + 4 * j;
          uint4 top[MT], low[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            top[mt] = lds128(ks_at + (mt * 16 + r) * S::ROW + kc * 16);
            low[mt] = lds128(ks_at + (mt * 16 + r + 8) * S::ROW + kc * 16);
          }
          if constexpr (S::E4M3) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t x[MT][2][4];
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                e4m3x4_to_f16(k ? top[mt].z : top[mt].x, &x[mt][0][0], &x[mt][0][2]);
                e4m3x4_to_f16(k ? low[mt].z : low[mt].x, &x[mt][0][1], &x[mt][0][3]);
                e4m3x4_to_f16(k ? top[mt].w : top[mt].y, &x[mt][1][0], &x[mt][1][2]);
                e4m3x4_to_f16(k ? low[mt].w : low[mt].y, &x[mt][1][1], &x[mt][1][3]);
              }
              step(2 * j + k, x);
            }
          } else {
            uint32_t x[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              x[mt][0][0] = top[mt].x, x[mt][0][1] = low[mt].x, x[mt][0][2] = top[mt].y, x[mt][0][3] = low[mt].y;
              x[mt][1][0] = top[mt].z, x[mt][1][1] = low[mt].z, x[mt][1][2] = top[mt].w, x[mt][1][3] = low[mt].w;
            }
            step(j, x);
          }
        }

        uint32_t pb[MT][NT][S::PARTS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[MT][4], n0 = m[nt][0], n1 = m[nt][1];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              s[mt][k] = fmaf(acc[mt][nt][1][k], 1.0f / S::LOW, acc[mt][nt][0][k]) * f1[nt][k & 1];
            if (f2 > 0.0f) {
#pragma unroll
              for (int k = 0; k < 4; ++k) s[mt][k] = tanh_flat(s[mt][k]) * f2;
            }
          }
          if (here != kAll) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if (!(here >> (mt * 16 + r) & 1)) s[mt][0] = s[mt][1] = -INFINITY;
              if (!(here >> (mt * 16 + r + 8) & 1)) s[mt][2] = s[mt][3] = -INFINITY;
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            n0 = fmaxf(n0, fmaxf(s[mt][0], s[mt][2]));
            n1 = fmaxf(n1, fmaxf(s[mt][1], s[mt][3]));
          }
          if (__any_sync(~0u, n0 > m[nt][0] + kSlack || n1 > m[nt][1] + kSlack)) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
              n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, k));
              n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, k));
            }
            // a column that has seen only -inf keeps its zero sum
            const float f0 = n0 == -INFINITY ? 1.0f : exp2_ftz(m[nt][0] - n0);
            const float f1_ = n1 == -INFINITY ? 1.0f : exp2_ftz(m[nt][1] - n1);
            m[nt][0] = n0;
            m[nt][1] = n1;
            l[nt][0] *= f0;
            l[nt][1] *= f1_;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
              o[nt][k][0] *= f0;
              o[nt][k][1] *= f1_;
              o[nt][k][2] *= f0;
              o[nt][k][3] *= f1_;
            }
          }
          const float base0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0] - kLift;
          const float base1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1] - kLift;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float p[4];
            p[0] = exp2_ftz(s[mt][0] - base0);
            p[1] = exp2_ftz(s[mt][1] - base1);
            p[2] = exp2_ftz(s[mt][2] - base0);
            p[3] = exp2_ftz(s[mt][3] - base1);
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
#pragma unroll
            for (int k = 0; k < S::PARTS; ++k) {
              pb[mt][nt][k][0] = transpose8x8(take_part<S::E4M3>(p[0], p[1]));
              pb[mt][nt][k][1] = transpose8x8(take_part<S::E4M3>(p[2], p[3]));
            }
          }
        }

        __syncwarp();  // every lane is done with the keys before their slot is filled again
        issue(ahead, i + S::AHEAD < mine, false, fill);
        fill = next_slot(fill);
        asm volatile("cp.async.wait_group %0;" ::"n"(S::SLOTS - 1) : "memory");
        __syncwarp();
        const uint32_t vs_at = ring + use * S::PIECE;
        use = next_slot(use);

        // outputs: 64 entries at a time; this lane's 8 are 64 j + 8 r + (0..7)
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          uint32_t w[MT][4][4];  // [position 2c, 2c + 1, 2c + 8, 2c + 9][words of 8 entries]
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row_ = mt * 16 + 2 * c + (k & 1) + (k >> 1) * 8;
              const int sw = S::CH >= 8 ? ((row_ >> 1) & 3) << 1 : ((row_ >> 1) & 1) << 1;
              if constexpr (S::E4M3) {
                const int unit = 8 * j + r;  // of 8 bytes
                const uint2 v = lds64(vs_at + row_ * S::ROW + ((unit >> 1) ^ sw) * 16 + (unit & 1) * 8);
                w[mt][k][0] = v.x;
                w[mt][k][1] = v.y;
              } else {
                const uint4 v = lds128(vs_at + row_ * S::ROW + ((8 * j + r) ^ sw) * 16);
                w[mt][k][0] = v.x;
                w[mt][k][1] = v.y;
                w[mt][k][2] = v.z;
                w[mt][k][3] = v.w;
              }
            }
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // entries 8 r + 2 q and 8 r + 2 q + 1
            uint32_t x[MT][4], fin[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if constexpr (S::E4M3) {
                const uint32_t sel = q & 1 ? 0x7362 : 0x5140;
                e4m3x4_to_f16(__byte_perm(w[mt][0][q / 2], w[mt][1][q / 2], sel), &x[mt][0], &x[mt][1]);
                e4m3x4_to_f16(__byte_perm(w[mt][2][q / 2], w[mt][3][q / 2], sel), &x[mt][2], &x[mt][3]);
              } else {
                x[mt][0] = __byte_perm(w[mt][0][q], w[mt][1][q], 0x5410);
                x[mt][1] = __byte_perm(w[mt][0][q], w[mt][1][q], 0x7632);
                x[mt][2] = __byte_perm(w[mt][2][q], w[mt][3][q], 0x5410);
                x[mt][3] = __byte_perm(w[mt][2][q], w[mt][3][q], 0x7632);
              }
              if constexpr (CAREFUL) finite_pairs(x[mt], fin[mt]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float t[4];
#pragma unroll
              for (int k = S::PARTS - 1; k >= 0; --k) {
                if (S::E4M3 && k == 0) {  // the lower parts' sum, back to its size
                  scale_pair(t[0], t[1], 1.0f / S::LOW);
                  scale_pair(t[2], t[3], 1.0f / S::LOW);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  const uint32_t* a = CAREFUL && k > 0 ? fin[mt] : x[mt];
                  if (k == S::PARTS - 1 && mt == 0)
                    mma16816<S::E4M3, true>(t, a, pb[mt][nt][k][0], pb[mt][nt][k][1]);
                  else
                    mma16816<S::E4M3, false>(t, a, pb[mt][nt][k][0], pb[mt][nt][k][1]);
                }
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) o[nt][4 * j + q][k] += t[k];
            }
          }
        }
        __syncwarp();
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    };
    stream(std::false_type{});
    if constexpr (!S::E4M3) {
      // a NaN may stem from an infinity of the cache times a zero or negative lower part: then the
      // tiles are taken again with the lower parts kept from it
      bool nan = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        nan |= isnan(l[nt][0]) || isnan(l[nt][1]);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) nan |= isnan(o[nt][k][q]);
      }
      if (__any_sync(~0u, nan)) stream(std::true_type{});
    }

    // ---- the warps meet -----------------------------------------------------------------------------
    __syncthreads();  // the rings are drained
    float* os = reinterpret_cast<float*>(smem);  // [warp][head][OS]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float s = l[nt][k] * kDrop;
        for (int q = 4; q < 32; q <<= 1) s += __shfl_xor_sync(~0u, s, q);
        const int h = nt * 8 + 2 * c + k;
        if (r == 0) warp_ml[warp][h] = make_float2(m[nt][k], s);
        if (h < heads) {
#pragma unroll
          for (int j = 0; j < DP / 64; ++j) {
            float4* dst = reinterpret_cast<float4*>(os + (warp * HB + h) * S::OS + 64 * j + 8 * r);
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = o[nt][4 * j + q / 2][k + 2 * (q & 1)] * kDrop;
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == units;
    const int slot = 2 * b + (row_begin <= begin ? 0 : 1);
    const int quads = D / 4;
    for (int e = tid; e < heads * quads; e += T) {
      const int h = e / quads, d = (e - h * quads) * 4;
      float2 ml[W];
      float4 t[W], v = make_float4(0, 0, 0, 0);
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        ml[w] = warp_ml[w][h];
        t[w] = *reinterpret_cast<const float4*>(os + (w * HB + h) * S::OS + d);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, ml[w].x);  // drops a NaN: its sum is NaN too
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ml[w].x == -INFINITY ? 0.0f : exp2_ftz(ml[w].x - M);
        L += f * ml[w].y;
        v.x += f * t[w].x, v.y += f * t[w].y, v.z += f * t[w].z, v.w += f * t[w].w;
      }
      put_row<S>(g, g.part_ml, whole ? -1 : slot, (long long)seq * g.a.n_heads + head0, h, d, v, M, L);
    }

    // ---- a shared row: the last CTA to arrive joins its parts ----------------------------------------
    if (!whole) {
      auto owner = [&](int unit) { return (int)(((unit + 1ll) * B - 1) / U); };  // start_of's inverse
      const int b0 = run ? row_begin : owner(row_begin);
      const int n = run ? runs : owner(row_begin + units - 1) - b0 + 1;
      // the first CTA's slot: its first segment if its run starts in this row
      const int slot0 = 2 * b0 + (run || row_begin <= start_of(b0) ? 0 : 1);
      const long long at = (long long)seq * g.a.n_heads + head0;
      auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (b0 + k); };
      // In one step up to kJoin parts; else groups first, each by its own last CTA, into the slot of
      // the group's first: two short reads in place of a long one. A group of 8 or 16 is read in one
      // go, and so are the up to 16 groups (8 query heads: 128 parts 12.6 us, 13.9 in groups of 12; 444
      // parts 16.2 in groups of 32, 17.5 in groups of 22).
      const int group = n <= kJoin ? n : n <= 128 ? 8 : n <= 256 ? 16 : 32;
      const int k0 = (b - b0) / group * group, groups = (n + group - 1) / group;
      bool last = arrive(g.tickets + slot_of(k0), min(group, n - k0), &is_last);
      if (last) {
        join<S>(g, g.part_ml, heads, min(group, n - k0), {slot_of(k0), 2 * (b0 + k0), 2},
                groups == 1 ? -1 : slot_of(k0), at);
        if (groups > 1) {
          last = arrive(g.tickets2 + slot0, groups, &is_last);
          if (last) join<S>(g, g.part_ml2, heads, groups, {slot0, 2 * b0, 2 * group}, -1, at);
        }
      }
    }
    __syncthreads();  // the join's buffer is read before the next segment fills the ring
    if (run) break;
    x += runs - r0;
    if (x == base + rows_of_seq * runs) {
      base = x;
      len = len_at(++seq);
    }
  }
  leftovers();
}

constexpr int kMaxCtas = 4;  // CTAs on an SM, over all shapes

// Blocks of query heads: 16 at a time where a key head has more than 8 and the outputs fit the
// registers (head_dim up to 128), else 8.
static int head_blocks(int row_heads, int head_dim) { return row_heads > 8 && head_dim <= 128 ? 2 : 1; }

static int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

size_t attention_ws_bytes(int n_heads, int n_kv_heads, int head_dim, int sm_count) {
  const size_t hb = 8 * head_blocks(n_heads / n_kv_heads, head_dim);
  const size_t slots = 2 * kMaxCtas * (size_t)sm_count;  // two for each CTA
  return slots * hb * (padded_dim(head_dim) * 4 + 16) + ((slots * 8 + 255) & ~size_t(255));
}

// CTAs of a call whose tables hold max_pos positions a sequence: a wave, or fewer where the units that
// there can be are fewer. In 64 bits: a window of 2^31 - 1 is a common way to ask for none.
static int grid_ctas(long long rows, long long max_pos, int window, int wave) {
  const long long seen = (long long)window + kUnit;
  const long long longest = window > 0 && seen < max_pos ? seen : max_pos;
  const long long units = rows * ((longest + kUnit - 1) / kUnit);
  return (int)(units < wave ? units : wave);
}

template <class S>
static int shape_ctas(int n_seq, int n_kv_heads, int row_heads, long long max_pos, int window, int sm_count) {
  static_assert(S::CTAS <= kMaxCtas, "workspace slots");
  const int blocks = (row_heads + S::HB - 1) / S::HB;
  return grid_ctas((long long)n_seq * n_kv_heads * blocks, max_pos, window, S::CTAS * sm_count);
}

template <class S>
static cudaError_t launch_shape(AttnArgs g, int sm_count, cudaStream_t stream) {
  const void* f = reinterpret_cast<const void*>(attention_kernel<S>);
  cudaError_t e = ensure_smem_limit(f, S::SMEM);
  if (e != cudaSuccess) return e;
  g.blocks = (g.row_heads + S::HB - 1) / S::HB;
  const long long slots = 2ll * kMaxCtas * sm_count;
  g.tickets = static_cast<uint32_t*>(g.a.ws);
  g.tickets2 = g.tickets + slots;
  g.part = reinterpret_cast<float*>(static_cast<uint8_t*>(g.a.ws) + ((slots * 8 + 255) & ~255ll));
  g.part_ml = reinterpret_cast<float2*>(g.part + slots * S::HB * S::DP);
  g.part_ml2 = g.part_ml + slots * S::HB;
  const int ctas = shape_ctas<S>(g.a.n_seq, g.a.cache.n_kv_heads, g.row_heads,
                                 (long long)g.a.max_pages * g.a.cache.page_size, g.a.prm.window, sm_count);
  return launch_pdl(attention_kernel<S>, dim3(ctas), dim3(S::THREADS), (size_t)S::SMEM, stream, g);
}

// Calls f with the shape by head_dim (padded), type and query heads to a key head; tiles, warps, slots
// and CTAs are what was fastest of what fits 227 KB and 65536 registers an SM. Measured on B200, before
// the copies left L2 first (1 to 3% less with it):
// - 128-wide bf16, 131071 positions of 8 key heads: 88.9 us; 16 warps an SM (128 registers a
//   thread) 96 to 98, tiles of 32 positions with 8 warps 94.5;
// - 128-wide 8-bit, 33 x 4099 positions: 53 us (56.5 with three query parts, where tiles of 16
//   positions took 68 and 16 warps 62 to 63);
// - 256-wide bf16: 8 warps of 3 slots 37.6 us on 48 windows of 2048, 6 warps 63, tiles of 32
//   positions 72; 8-bit, 33 x 4099: tiles of 32 positions 102, of 16 113;
// - 16 query heads to a key head, ragged batch of 64 up to 8192: bf16 with 12 warps 153, 8 warps 166
//   (one sequence alone prefers 8: 40 to 48); 8-bit tiles of 32 positions 89, of 16 99.
template <class F>
static auto with_shape(int head_dim, int row_heads, bool e4m3, F f) {
  const int dp = padded_dim(head_dim), nt = head_blocks(row_heads, head_dim);
  if (dp == 64 && nt == 1)
    return e4m3 ? f(AttnShape<64, true, 1, 2, 4, 5, 3>()) : f(AttnShape<64, false, 1, 2, 4, 3, 3>());
  if (dp == 64) return e4m3 ? f(AttnShape<64, true, 2, 2, 4, 3, 3>()) : f(AttnShape<64, false, 2, 2, 4, 3, 3>());
  if (dp == 128 && nt == 1)
    return e4m3 ? f(AttnShape<128, true, 1, 2, 4, 3, 3>()) : f(AttnShape<128, false, 1, 1, 4, 3, 3>());
  if (dp == 128)
    return e4m3 ? f(AttnShape<128, true, 2, 2, 4, 3, 2>()) : f(AttnShape<128, false, 2, 1, 4, 3, 3>());
  return e4m3 ? f(AttnShape<256, true, 1, 2, 4, 3, 2>()) : f(AttnShape<256, false, 1, 1, 4, 3, 2>());
}

int attention_ctas(int n_seq, int n_heads, int n_kv_heads, int head_dim, bool e4m3, long long max_pos,
                   int window, int sm_count) {
  const int row_heads = n_heads / n_kv_heads;
  return with_shape(head_dim, row_heads, e4m3, [&](auto shape) {
    return shape_ctas<decltype(shape)>(n_seq, n_kv_heads, row_heads, max_pos, window, sm_count);
  });
}

cudaError_t launch_paged_attention(const AttnLaunch& a, int sm_count, cudaStream_t stream) {
  AttnArgs g = {};
  g.a = a;
  g.row_heads = a.n_heads / a.cache.n_kv_heads;
  // position / page_size for positions below 2^31 by a multiplication: with s = ceil(log2 d) and
  // mul = floor(2^(31 + s) / d) + 1, mul * d exceeds 2^(31 + s) by at most d <= 2^s
  const uint32_t d = (uint32_t)a.cache.page_size;
  int s = 0;
  while ((1ull << s) < d) ++s;
  g.page_shift = s - 1;
  g.page_mul = d == 1 ? 0 : (uint32_t)((1ull << (31 + s)) / d + 1);
  g.page16 = d % 16 == 0;
  return with_shape(a.cache.head_dim, g.row_heads, a.cache.dtype == SPAX_KV_E4M3,
                    [&](auto shape) { return launch_shape<decltype(shape)>(g, sm_count, stream); });
}

}  // namespace spax
