// attention.cu — attention of one new token of each sequence over the paged key-value cache.
//
// For query head h over the positions j that it sees: s_j = scale (q . k_j) (capped when asked),
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m). The cache is read once, 4 G flops for each of its
// elements (G query heads to a key head), so the bound is HBM; everything else is arranged to keep
// enough bytes in flight.
//
// Work: a row is one (sequence, key head, block of up to 8 NT query heads). Its positions are cut
// into units of 64; the units of all rows, laid end to end, are dealt to the CTAs of one wave in
// equal contiguous runs, so ragged batches and single long sequences both fill the GPU. A CTA's run
// covers parts of rows (segments); a row that several CTAs share is joined by the last of them to
// arrive, in the order of the CTAs, so the result does not depend on who that is. No CTA waits for
// another.
//
// Within a segment the CTA's warps take tiles of 16 positions in turn; each streams its own
// through its own ring in shared memory with 16-byte asynchronous copies, and keeps its own running
// maximum, sum and outputs; the warps meet once, at the segment's end.
//
// Products run on the m16n8k16 matrix instructions, transposed: S^T = K Q^T and O^T = V^T P^T, so
// that the 16-row side is always positions or entries of the cache and the 8-column side the query
// heads (a decode step has 1 to 16 heads to a key head; the 128-row tiles of tcgen05 would be idle
// for the most part, and at 16 flops a byte the smaller instructions are nowhere near their rate).
// The order of a head's entries along the contraction is free, so a lane takes the 16 bytes that
// lie together in the cache as the fragment's entries and the query is laid out to match; for V the
// pairs of positions that a fragment wants are woven from two rows by byte permutes.
//
// Precision: cache elements are exact in bf16 (8-bit ones in fp16); fp32 queries and probabilities
// enter as three parts of 8 (11) bits each, which together hold the value, smallest part first. The
// matrix instructions add with truncation, so sums over many tiles are kept outside of them.
#include <type_traits>

#include "layer.cuh"

namespace spax {

constexpr int kTile = 16;  // positions in a warp's tile, starting at a multiple of 16
constexpr int kUnit = 64;  // positions in a unit of work, starting at a multiple of 64
constexpr int kJoin = 16;  // parts that are joined in one step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shapes of one instance: head_dim padded to DP, NT blocks of 8 query heads, WARPS warps with rings
// of STAGES tiles, CTAS resident on an SM.
template <int DP_, bool E4M3_, int NT_, int WARPS_, int STAGES_, int CTAS_>
struct AttnShape {
  static constexpr int DP = DP_, NT = NT_, HB = 8 * NT_, STAGES = STAGES_, CTAS = CTAS_;
  static constexpr int WARPS = WARPS_, THREADS = WARPS * 32;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int QP = 3, PP = E4M3 ? 2 : 3;  // parts of a query entry, of a probability
  static constexpr int ROW = DP * ES;             // bytes of a row of a tile
  static constexpr int CH = ROW / 16;             // 16-byte chunks of a row
  static constexpr int HALF = kTile * ROW;        // bytes of a tile's keys (or values)
  static constexpr int STAGE = 2 * HALF;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int KS = DP / 16;              // k steps of a score
  static constexpr int SMEM = RING + KS / 2 * QP * NT * 512;  // and the query's parts
  static constexpr int OS = DP + 4;               // row stride of the warps' outputs at the join
  static_assert(WARPS * HB * OS * 4 <= RING, "the join's buffer overlays the ring");
  static_assert(CTAS * (SMEM + 3072) <= 228 * 1024, "shared memory of the resident CTAs");
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

// (x, y) as a pair in the matrix type, and what the pair leaves of them.
template <bool E4M3>
__device__ __forceinline__ uint32_t take_part(float& x, float& y) {
  uint32_t d;
  if constexpr (E4M3) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    const __half2 h = *reinterpret_cast<const __half2*>(&d);
    x -= __low2float(h);
    y -= __high2float(h);
  } else {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    x -= __uint_as_float(d << 16);
    y -= __uint_as_float(d & 0xFFFF0000u);
  }
  return d;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0));
}

// Pairs of bf16 elements with an infinity replaced by the largest finite value: what the lower parts
// of a query or probability multiply in a careful pass. Such a part can be zero or negative, and an
// infinity times it would turn the product's own infinity into NaN.
__device__ __forceinline__ void finite_pairs(const uint32_t (&a)[4], uint32_t (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(f[k]) : "r"(a[k]), "r"(0x7F7F7F7Fu));
}

struct AttnArgs {
  AttnLaunch a;
  uint32_t page_mul;  // position / page_size = page_size == 1 ? position : umulhi(position, mul) >> shift
  int page_shift;
  int row_heads;      // query heads to a key head
  int blocks;         // blocks of HB query heads to a key head
  bool page16;        // a tile's positions are on one page
  float* part;        // [2 CTAs][HB][DP] outputs of shared rows
  float2* part_ml;    // [2 CTAs][HB] their maxima and sums
  uint32_t *tickets, *tickets2;  // [2 CTAs] each, zero at rest
};

template <class S>
struct Attn {
  // Positions [lo, len) of a sequence, by the window.
  static __device__ __forceinline__ int clipped_len(const AttnArgs& g, int seq, bool* bad) {
    const int len = __ldg(g.a.lens + seq);
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
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    *is_last = atomicAdd(ticket, 1u) == (uint32_t)(n - 1);
    if (*is_last) *ticket = 0;
    __threadfence();
  }
  __syncthreads();
  return *is_last;
}

// One head's entries of a row, joined: written as they are to a slot, or divided to the output.
template <class S>
__device__ __forceinline__ void put_row(const AttnArgs& g, int slot, long long at, int h, int d, float4 v,
                                        float M, float L) {
  if (slot >= 0) {
    __stcg(reinterpret_cast<float4*>(g.part + ((long long)slot * S::HB + h) * S::DP + d), v);
    if (d == 0) __stcg(g.part_ml + slot * S::HB + h, make_float2(M, L));
  } else {
    const float inv = L == 0.0f ? 0.0f : g.a.cache.v_scale / L;
    if (L == 0.0f) v = make_float4(0, 0, 0, 0);
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    *reinterpret_cast<float4*>(g.a.out + (at + h) * g.a.cache.head_dim + d) = v;
    if (d == 0 && g.a.lse) g.a.lse[at + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

// Joins n parts of a row, the slots of which slot_of gives, in their order.
template <class S, class F>
__device__ __forceinline__ void join(const AttnArgs& g, uint8_t* smem, int heads, int n, F slot_of,
                                     int to, long long at) {
  float2* ml = reinterpret_cast<float2*>(smem);  // [n][HB]: maximum and sum, then weight and sum
  __shared__ float2 total[S::HB];
  const int tid = threadIdx.x;
  for (int e = tid; e < n * S::HB; e += S::THREADS)
    if (e % S::HB < heads) ml[e] = __ldcg(g.part_ml + slot_of(e / S::HB) * S::HB + e % S::HB);
  __syncthreads();
  if (tid < heads) {
    float M = -INFINITY, L = 0.0f;
    for (int k = 0; k < n; ++k) M = fmaxf(M, ml[k * S::HB + tid].x);  // drops NaN: its sum has it too
    for (int k = 0; k < n; ++k) {
      const float2 v = ml[k * S::HB + tid];
      const float f = v.x == -INFINITY ? 0.0f : exp2_ftz(v.x - M);
      L += f * v.y;
      ml[k * S::HB + tid].x = f;
    }
    total[tid] = make_float2(M, L);
  }
  __syncthreads();
  const int quads = g.a.cache.head_dim / 4;
  for (int e = tid; e < heads * quads; e += S::THREADS) {
    const int h = e / quads, d = (e - h * quads) * 4;
    const float4* src = reinterpret_cast<const float4*>(g.part + (long long)h * S::DP + d);
    float4 v = make_float4(0, 0, 0, 0);
    int k = 0;
    auto take = [&](auto count) {
      constexpr int N = decltype(count)::value;
      for (; k + N <= n; k += N) {
        float4 t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = __ldcg(src + (long long)slot_of(k + i) * (S::HB * S::DP / 4));
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float f = ml[(k + i) * S::HB + h].x;
          v.x += f * t[i].x, v.y += f * t[i].y, v.z += f * t[i].z, v.w += f * t[i].w;
        }
      }
    };
    take(std::integral_constant<int, 8>{});
    take(std::integral_constant<int, 4>{});
    take(std::integral_constant<int, 1>{});
    put_row<S>(g, to, at, h, d, v, total[h].x, total[h].y);
  }
  __syncthreads();  // the buffers may be used again
}

template <class S>
__global__ void __launch_bounds__(S::THREADS, S::CTAS) attention_kernel(const AttnArgs g) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long prefix[S::THREADS + 1];
  __shared__ long long start_base;
  __shared__ int start_seq;
  __shared__ float2 warp_ml[S::WARPS][S::HB];
  __shared__ bool is_last;
  using A = Attn<S>;
  constexpr int DP = S::DP, NT = S::NT, HB = S::HB, T = S::THREADS, W = S::WARPS;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int r = lane >> 2, c = lane & 3;
  const int b = blockIdx.x;
  const spax_kv_cache& C = g.a.cache;
  const int D = C.head_dim, n_seq = g.a.n_seq;
  const int chunks = D * S::ES / 16;
  const long long rows_of_seq = (long long)C.n_kv_heads * g.blocks;

  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's run of units -----------------------------------------------------------------
  const int per = (n_seq + T - 1) / T;
  {
    long long sum = 0;
    bool any_bad = false;
    for (int s = tid * per; s < min(n_seq, (tid + 1) * per); ++s) {
      bool bad;
      sum += rows_of_seq * A::units_of(g, A::clipped_len(g, s, &bad));
      any_bad |= bad;
    }
    if (any_bad && b == 0) record_status(g.a.status, SPAX_ERR_INDEX);
    long long x = sum;  // inclusive scan
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) prefix[warp] = x;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += prefix[w];
    __syncthreads();
    prefix[tid + 1] = before + x;
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
  }
  const long long U = prefix[T];
  const long long B = min((long long)gridDim.x, U);

  // rows that see nothing
  for (int s = b; s < n_seq; s += gridDim.x) {
    bool bad;
    if (A::units_of(g, A::clipped_len(g, s, &bad)) != 0) continue;
    for (int i = tid; i < g.a.n_heads * D; i += T)
      g.a.out[(long long)s * g.a.n_heads * D + i] = 0.0f;
    if (g.a.lse)
      for (int i = tid; i < g.a.n_heads; i += T)
        g.a.lse[(long long)s * g.a.n_heads + i] = -INFINITY;
  }
  if (b >= B) return;

  const long long begin = U * b / B, end = U * (b + 1) / B;
  if (prefix[tid] <= begin && begin < prefix[tid + 1]) {
    long long base = prefix[tid];
    int s = tid * per;
    for (;; ++s) {
      bool bad;
      const long long n = rows_of_seq * A::units_of(g, A::clipped_len(g, s, &bad));
      if (begin < base + n) break;
      base += n;
    }
    start_seq = s;
    start_base = base;
  }
  __syncthreads();
  int seq = start_seq;
  long long base = start_base;

  const uint32_t ring = smem_u32(smem) + warp * (S::STAGES * S::STAGE);
  const uint32_t qsm = smem_u32(smem) + S::RING;

  for (long long x = begin; x < end;) {
    bool bad;
    const int len = A::clipped_len(g, seq, &bad);
    const int units = A::units_of(g, len);
    if (units == 0) {  // an empty sequence between two others
      ++seq;
      continue;
    }
    const long long y = x - base;
    const int row = (int)(y / units), u0 = (int)(y - (long long)row * units);
    const int u1 = (int)min((long long)units, u0 + (end - x));
    const long long row_begin = base + (long long)row * units, row_end = row_begin + units;
    const int kvh = row / g.blocks, hb = row - kvh * g.blocks;
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
    {
      const float cap = g.a.prm.softcap;
      f2 = cap * kLog2e;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + r;
        const float* q = g.a.q + seq * g.a.q_stride + (long long)(head0 + min(h, heads - 1)) * D;
        auto entries = [&](int ks) {  // entries of this lane's head for k step ks
          const int d = S::E4M3 ? 64 * (ks / 4) + 16 * c + 4 * (ks % 4) : 32 * (ks / 2) + 8 * c + 4 * (ks % 2);
          return h < heads && d < D ? *reinterpret_cast<const float4*>(q + d) : make_float4(0, 0, 0, 0);
        };
        float up = 1.0f, down = 1.0f;
        if constexpr (S::E4M3) {
          // fp16 parts: the head's largest entry is brought to [2^9, 2^10)
          float top = 0.0f;
#pragma unroll
          for (int ks = 0; ks < S::KS; ++ks) {
            const float4 v = entries(ks);
            top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const int e = (int)(__float_as_uint(top) >> 23) - 127;  // -127: zero or subnormal, 128: inf
          if (e < 128) {
            const int k = min(100, 9 - e);
            up = __uint_as_float((uint32_t)(k + 127) << 23);
            down = __uint_as_float((uint32_t)(127 - k) << 23);
          }
        }
#pragma unroll
        for (int i = 0; i < (S::KS / 2 + W - 1) / W; ++i) {
          const int pair = i * W + warp;
          if (pair >= S::KS / 2) break;
          float4 v = entries(2 * pair), w = entries(2 * pair + 1);
          v.x *= up, v.y *= up, v.z *= up, v.w *= up;
          w.x *= up, w.y *= up, w.z *= up, w.w *= up;
#pragma unroll
          for (int p = 0; p < S::QP; ++p) {
            const uint32_t x0 = take_part<S::E4M3>(v.x, v.y), x1 = take_part<S::E4M3>(v.z, v.w);
            const uint32_t y0 = take_part<S::E4M3>(w.x, w.y), y1 = take_part<S::E4M3>(w.z, w.w);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             qsm + ((pair * S::QP + p) * NT + nt) * 512 + lane * 16),
                         "r"(x0), "r"(x1), "r"(y0), "r"(y1));
          }
        }
        // the columns of a score fragment are heads 2c, 2c + 1
        const float f = g.a.prm.scale * C.k_scale * down * (cap > 0.0f ? 1.0f / cap : kLog2e);
        f1[nt][0] = __shfl_sync(~0u, f, (2 * c) * 4);
        f1[nt][1] = __shfl_sync(~0u, f, (2 * c + 1) * 4);
      }
    }
    __syncthreads();

    // ---- this warp's tiles: tile i starts at t0 + (i * W + warp) * 16 ------------------------------
    // Exponents are taken from a base that trails the maximum by up to kSlack powers of two (it moves
    // only when a score passes it by more), and fp16 probabilities are lifted by 2^12 so that their
    // parts stay normal numbers (and their sums are lowered again, exactly, at the end).
    constexpr float kSlack = S::E4M3 ? 3.0f : 8.0f, kLift = S::E4M3 ? 12.0f : 0.0f,
                    kDrop = S::E4M3 ? 1.0f / 4096.0f : 1.0f;
    const int tiles = (t1 - t0 + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + W - 1) / W : 0;
    const int first = t0 + warp * kTile;
    float m[NT][2], l[NT][2], o[NT][DP / 16][4];

    auto stream = [&](auto careful) {
      constexpr bool CAREFUL = decltype(careful)::value;
      auto page_entry = [&](int i) {  // the table's entry for the lane's position of tile i
        int pos = first + i * (W * kTile);
        if (!g.page16) pos = min(pos + (lane & 15), t1 - 1);
        return i < mine ? __ldg(table + A::page_of(g, pos)) : 0;
      };
      // Starts the copies of tile i; returns which of its positions are seen.
      auto issue = [&](int i, int page) -> uint32_t {
        uint32_t bits = 0;
        if (i < mine) {
          const int pos0 = first + i * (W * kTile);
          const uint32_t stage = ring + (uint32_t)i % S::STAGES * S::STAGE;
          constexpr int RPI = 32 / S::CH >= 1 ? 32 / S::CH : 1;  // rows of a step
          const int row0 = lane / S::CH, ch = lane % S::CH;
          auto put = [&](int k, const uint8_t* ks, const uint8_t* vs, bool real) {
            const int row_ = k * RPI + row0;
            // keys: rows of unlike parity in different halves of the banks; values: pairs of rows
            const int kc = S::CH >= 8 ? ch ^ ((row_ & 1) << 2) : ch;
            const int vc = S::CH >= 8 ? ch ^ (((row_ >> 1) & 3) << 1) : ch ^ (((row_ >> 1) & 1) << 1);
            cp16(stage + row_ * S::ROW + kc * 16, ks, real);
            cp16(stage + S::HALF + row_ * S::ROW + vc * 16, vs, real);
          };
          if (g.page16 && pos0 >= lo && pos0 + kTile <= t1 && (uint32_t)page < (uint32_t)C.n_pages &&
              D == DP) {
            // the whole tile on one page: rows at one stride
            const long long at = (page * C.page_stride +
                                  (long long)(pos0 - A::page_of(g, pos0) * C.page_size + row0) * C.token_stride) * S::ES + ch * 16;
            const uint8_t* ks = kpool + at;
            const uint8_t* vs = vpool + at;
            const long long step = RPI * C.token_stride * S::ES;
            bits = 0xFFFFu;
#pragma unroll
            for (int k = 0; k < kTile / RPI; ++k) {
              put(k, ks, vs, true);
              ks += step;
              vs += step;
            }
          } else {
            const int pos = pos0 + (lane & 15);
            long long off = -1;
            if (pos >= lo && pos < t1) {
              if ((uint32_t)page < (uint32_t)C.n_pages)
                off = (page * C.page_stride +
                       (long long)(pos - A::page_of(g, pos) * C.page_size) * C.token_stride) * S::ES;
              else
                record_status(g.a.status, SPAX_ERR_INDEX);
            }
            bits = __ballot_sync(~0u, off >= 0) & 0xFFFFu;
#pragma unroll
            for (int k = 0; k < kTile / RPI; ++k) {
              const long long row_off = __shfl_sync(~0u, off, k * RPI + row0);
              const bool real = row_off >= 0 && ch < chunks;
              const long long at = real ? row_off + ch * 16 : 0;
              put(k, kpool + at, vpool + at, real);
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return bits;
      };

      uint32_t seen[S::STAGES - 1];
      int page = page_entry(0);
#pragma unroll
      for (int i = 0; i < S::STAGES - 1; ++i) {
        const int next = page_entry(i + 1);
        seen[i] = issue(i, page);
        page = next;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
      }
      for (int i = 0; i < mine; ++i) {
        const int next = page_entry(i + S::STAGES);
        const uint32_t now = issue(i + S::STAGES - 1, page);
        page = next;
        const uint32_t here = seen[0];
#pragma unroll
        for (int k = 0; k + 1 < S::STAGES - 1; ++k) seen[k] = seen[k + 1];
        seen[S::STAGES - 2] = now;
        asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
        __syncwarp();
        const uint32_t ks_at = ring + (uint32_t)i % S::STAGES * S::STAGE, vs_at = ks_at + S::HALF;

        // scores: one chain for the first part of the query, one for the others
        float acc[NT][2][4];
        auto step = [&](int pair, const uint32_t(&a)[4], const uint32_t(&b)[4]) {
          uint32_t fa[4], fb[4];
          if constexpr (CAREFUL) {
            finite_pairs(a, fa);
            finite_pairs(b, fb);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = S::QP - 1; p >= 0; --p) {
              const uint4 v = lds128(qsm + ((pair * S::QP + p) * NT + nt) * 512 + lane * 16);
              float(&d)[4] = acc[nt][p == 0 ? 0 : 1];
              const bool low = CAREFUL && p > 0;
              if (pair == 0 && (p == 0 || p == S::QP - 1))
                mma16816<S::E4M3, true>(d, low ? fa : a, v.x, v.y);
              else
                mma16816<S::E4M3, false>(d, low ? fa : a, v.x, v.y);
              mma16816<S::E4M3, false>(d, low ? fb : b, v.z, v.w);
            }
        };
#pragma unroll
        for (int j = 0; j < S::CH / 4; ++j) {
          const int kc = S::CH >= 8 ? (c + 4 * j) ^ ((r & 1) << 2) : c + 4 * j;
          const uint4 top = lds128(ks_at + r * S::ROW + kc * 16);
          const uint4 low = lds128(ks_at + (r + 8) * S::ROW + kc * 16);
          if constexpr (S::E4M3) {
            const uint32_t tw[4] = {top.x, top.y, top.z, top.w}, lw[4] = {low.x, low.y, low.z, low.w};
            uint32_t a[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              e4m3x4_to_f16(tw[k], &a[k][0], &a[k][2]);
              e4m3x4_to_f16(lw[k], &a[k][1], &a[k][3]);
            }
            step(2 * j, a[0], a[1]);
            step(2 * j + 1, a[2], a[3]);
          } else {
            const uint32_t a0[4] = {top.x, low.x, top.y, low.y}, a1[4] = {top.z, low.z, top.w, low.w};
            step(j, a0, a1);
          }
        }

        uint32_t pb[NT][S::PP][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float s[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) s[k] = (acc[nt][1][k] + acc[nt][0][k]) * f1[nt][k & 1];
          if (f2 > 0.0f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] = tanhf(s[k]) * f2;
          }
          if (here != 0xFFFFu) {
            if (!(here >> r & 1)) s[0] = s[1] = -INFINITY;
            if (!(here >> (r + 8) & 1)) s[2] = s[3] = -INFINITY;
          }
          const bool up = fmaxf(s[0], s[2]) > m[nt][0] + kSlack || fmaxf(s[1], s[3]) > m[nt][1] + kSlack;
          if (__any_sync(~0u, up)) {
            float n0 = fmaxf(m[nt][0], fmaxf(s[0], s[2])), n1 = fmaxf(m[nt][1], fmaxf(s[1], s[3]));
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
          float p[4];
          const float base0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0] - kLift;
          const float base1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1] - kLift;
          p[0] = exp2_ftz(s[0] - base0);
          p[1] = exp2_ftz(s[1] - base1);
          p[2] = exp2_ftz(s[2] - base0);
          p[3] = exp2_ftz(s[3] - base1);
          l[nt][0] += p[0] + p[2];
          l[nt][1] += p[1] + p[3];
#pragma unroll
          for (int k = 0; k < S::PP; ++k) {
            pb[nt][k][0] = transpose8x8(take_part<S::E4M3>(p[0], p[1]));
            pb[nt][k][1] = transpose8x8(take_part<S::E4M3>(p[2], p[3]));
          }
        }

        // outputs: 64 entries at a time; this lane's 8 are 64 j + 8 r + (0..7)
#pragma unroll
        for (int j = 0; j < DP / 64; ++j) {
          uint32_t w[4][4];  // [position 2c, 2c + 1, 2c + 8, 2c + 9][words of 8 entries]
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row_ = 2 * c + (k & 1) + (k >> 1) * 8;
            const int sw = S::CH >= 8 ? ((row_ >> 1) & 3) << 1 : ((row_ >> 1) & 1) << 1;
            if constexpr (S::E4M3) {
              const int unit = 8 * j + r;  // of 8 bytes
              const uint2 v = lds64(vs_at + row_ * S::ROW + ((unit >> 1) ^ sw) * 16 + (unit & 1) * 8);
              w[k][0] = v.x;
              w[k][1] = v.y;
            } else {
              const uint4 v = lds128(vs_at + row_ * S::ROW + ((8 * j + r) ^ sw) * 16);
              w[k][0] = v.x;
              w[k][1] = v.y;
              w[k][2] = v.z;
              w[k][3] = v.w;
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // entries 8 r + 2 q and 8 r + 2 q + 1
            uint32_t a[4];
            if constexpr (S::E4M3) {
              const uint32_t sel = q & 1 ? 0x7362 : 0x5140;
              e4m3x4_to_f16(__byte_perm(w[0][q / 2], w[1][q / 2], sel), &a[0], &a[1]);
              e4m3x4_to_f16(__byte_perm(w[2][q / 2], w[3][q / 2], sel), &a[2], &a[3]);
            } else {
              a[0] = __byte_perm(w[0][q], w[1][q], 0x5410);
              a[1] = __byte_perm(w[0][q], w[1][q], 0x7632);
              a[2] = __byte_perm(w[2][q], w[3][q], 0x5410);
              a[3] = __byte_perm(w[2][q], w[3][q], 0x7632);
            }
            uint32_t fa[4];
            if constexpr (CAREFUL) finite_pairs(a, fa);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float t[4];
#pragma unroll
              for (int k = S::PP - 1; k >= 0; --k) {
                const bool low = CAREFUL && k > 0;
                if (k == S::PP - 1)
                  mma16816<S::E4M3, true>(t, low ? fa : a, pb[nt][k][0], pb[nt][k][1]);
                else
                  mma16816<S::E4M3, false>(t, low ? fa : a, pb[nt][k][0], pb[nt][k][1]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) o[nt][4 * j + q][k] += t[k];
            }
          }
        }
        __syncwarp();  // every lane is done with the stage before it is filled again
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
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, warp_ml[w][h].x);
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // fmaxf drops a NaN maximum; its warp's sum is NaN and brings it back
        const float f = warp_ml[w][h].x == -INFINITY ? 0.0f : exp2_ftz(warp_ml[w][h].x - M);
        if (f == 0.0f && warp_ml[w][h].y == 0.0f) continue;
        const float4 t = *reinterpret_cast<const float4*>(os + (w * HB + h) * S::OS + d);
        L += f * warp_ml[w][h].y;
        v.x += f * t.x, v.y += f * t.y, v.z += f * t.z, v.w += f * t.w;
      }
      put_row<S>(g, whole ? -1 : slot, (long long)seq * g.a.n_heads + head0, h, d, v, M, L);
    }

    // ---- a shared row: the last CTA to arrive joins its parts ----------------------------------------
    if (!whole) {
      const int b0 = (int)(((row_begin + 1) * B - 1) / U), b1 = (int)((row_end * B - 1) / U);
      const int n = b1 - b0 + 1;
      // the first CTA's slot: its first segment if its run starts in this row
      const int slot0 = 2 * b0 + (row_begin <= U * b0 / B ? 0 : 1);
      const long long at = (long long)seq * g.a.n_heads + head0;
      auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (b0 + k); };
      // In one step up to kJoin parts; else groups of about sqrt(n) first, each by its own last CTA,
      // into the slot of the group's first: two short reads in place of one long one.
      int group = n;
      if (n > kJoin)
        for (group = kJoin / 2; group * group < n;) ++group;
      const int k0 = (b - b0) / group * group, groups = (n + group - 1) / group;
      bool last = arrive(g.tickets + slot_of(k0), min(group, n - k0), &is_last);
      if (last) {
        join<S>(g, smem, heads, min(group, n - k0), [&](int i) { return slot_of(k0 + i); },
                groups == 1 ? -1 : slot_of(k0), at);
        if (groups > 1) {
          last = arrive(g.tickets2 + slot0, groups, &is_last);
          if (last) join<S>(g, smem, heads, groups, [&](int i) { return slot_of(i * group); }, -1, at);
        }
      }
    }
    __syncthreads();  // the join's buffer is read before the next segment fills the ring
    x += u1 - u0;
    if (x == base + rows_of_seq * units) {
      base = x;
      ++seq;
    }
  }
}

constexpr int kMaxCtas = 4;  // CTAs on an SM, over all shapes

// Blocks of query heads: 16 at a time where a key head has more than 8 and the outputs fit the
// registers (head_dim up to 128), else 8.
static int head_blocks(int row_heads, int head_dim) { return row_heads > 8 && head_dim <= 128 ? 2 : 1; }

static int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

size_t attention_ws_bytes(int n_heads, int n_kv_heads, int head_dim, int sm_count) {
  const size_t hb = 8 * head_blocks(n_heads / n_kv_heads, head_dim);
  const size_t slots = 2 * kMaxCtas * (size_t)sm_count;  // two for each CTA
  return slots * hb * (padded_dim(head_dim) * 4 + 8) + ((slots * 8 + 255) & ~size_t(255));
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
  long long longest = (long long)g.a.max_pages * g.a.cache.page_size;
  if (g.a.prm.window > 0 && g.a.prm.window + kUnit < longest) longest = g.a.prm.window + kUnit;
  const long long units = (long long)g.a.n_seq * g.a.cache.n_kv_heads * g.blocks *
                          ((longest + kUnit - 1) / kUnit);
  static_assert(S::CTAS <= kMaxCtas, "workspace slots");
  const long long wave = (long long)S::CTAS * sm_count;
  return launch_pdl(attention_kernel<S>, dim3((unsigned)(units < wave ? units : wave)),
                    dim3(S::THREADS), (size_t)S::SMEM, stream, g);
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
  g.page16 = d % kTile == 0;
  const int dp = padded_dim(a.cache.head_dim), nt = head_blocks(g.row_heads, a.cache.head_dim);
  const bool e = a.cache.dtype == SPAX_KV_E4M3;
  // warps, stages and CTAs by what fits 227 KB and 65536 registers an SM
  if (dp == 64 && nt == 1)
    return e ? launch_shape<AttnShape<64, true, 1, 4, 4, 4>>(g, sm_count, stream)
             : launch_shape<AttnShape<64, false, 1, 4, 3, 4>>(g, sm_count, stream);
  if (dp == 64)
    return e ? launch_shape<AttnShape<64, true, 2, 4, 4, 3>>(g, sm_count, stream)
             : launch_shape<AttnShape<64, false, 2, 4, 3, 3>>(g, sm_count, stream);
  if (dp == 128 && nt == 1)
    return e ? launch_shape<AttnShape<128, true, 1, 4, 4, 3>>(g, sm_count, stream)
             : launch_shape<AttnShape<128, false, 1, 4, 2, 3>>(g, sm_count, stream);
  if (dp == 128)
    return e ? launch_shape<AttnShape<128, true, 2, 4, 4, 2>>(g, sm_count, stream)
             : launch_shape<AttnShape<128, false, 2, 4, 3, 2>>(g, sm_count, stream);
  return e ? launch_shape<AttnShape<256, true, 1, 4, 3, 2>>(g, sm_count, stream)
           : launch_shape<AttnShape<256, false, 1, 6, 2, 1>>(g, sm_count, stream);
}

}  // namespace spax
