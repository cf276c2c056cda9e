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
// Within a segment each of the CTA's 4 warps takes every fourth tile of 16 positions, streams it
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
#include "layer.cuh"

namespace spax {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kTile = 16;                       // positions in a warp's tile
constexpr int kUnit = kTile * kAttnWarps;       // positions in a unit of work
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Shapes of one instance: head_dim padded to DP, NT blocks of 8 query heads.
template <int DP_, bool E4M3_, int NT_>
struct AttnShape {
  static constexpr int DP = DP_, NT = NT_, HB = 8 * NT_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int ROW = DP * ES;             // bytes of a row of a tile
  static constexpr int CH = ROW / 16;             // 16-byte chunks of a row
  static constexpr int HALF = kTile * ROW;        // bytes of a tile's keys (or values)
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = STAGE >= 8192 ? 3 : 4;
  static constexpr int RING = kAttnWarps * STAGES * STAGE;
  static constexpr int KS = DP / 16;              // k steps of a score
  static constexpr bool QREG = KS * 2 * 3 * NT <= 48;  // the query's parts fit in registers
  static constexpr int QBYTES = QREG ? 0 : KS * 3 * NT * 256;
  static constexpr int OS = DP + 4;               // row stride of the warps' outputs at the join
  static constexpr int SMEM = RING + QBYTES;
  static constexpr int CTAS = SMEM <= 112 * 1024 ? 2 : 1;  // resident on an SM
  static_assert(kAttnWarps * HB * OS * 4 <= RING, "the join's buffer overlays the ring");
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, bool e4m3) {
  if (e4m3)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_bytes) {
  uint32_t d;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(two_bytes));
  return d;
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

// A pair of cache elements with an infinity replaced by the largest finite value: what the lower
// parts of a query or probability multiply. Such a part can be zero or negative, and an infinity
// times it would turn the product's own infinity into NaN. (8-bit elements have no infinity.)
template <bool E4M3>
__device__ __forceinline__ void finite_pairs(const uint32_t (&a)[4], uint32_t (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (E4M3)
      f[k] = a[k];
    else
      asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(f[k]) : "r"(a[k]), "r"(0x7F7F7F7Fu));
  }
}

struct AttnArgs {
  AttnLaunch a;
  uint32_t page_mul;  // position / page_size = page_size == 1 ? position : umulhi(position, mul) >> shift
  int page_shift;
  int row_heads;      // query heads to a key head
  int blocks;         // blocks of HB query heads to a key head
  float* part;        // [2 CTAs][HB][DP] outputs of shared rows
  float2* part_ml;    // [2 CTAs][HB] their maxima and sums
  uint32_t* tickets;  // [2 CTAs], zero at rest
};

// What one warp knows of a tile: lane l < 16 holds the pool offset of position l, or -1.
struct TilePlace {
  long long off;
  uint32_t seen;  // bit l: position l is seen
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
    return (len - first_seen(g, len) + kUnit - 1) / kUnit;
  }

  static __device__ __forceinline__ int page_of(const AttnArgs& g, int pos) {
    return g.page_shift < 0 ? pos : (int)(__umulhi((uint32_t)pos, g.page_mul) >> g.page_shift);
  }
};

template <class S>
__global__ void __launch_bounds__(kAttnThreads, S::CTAS) attention_kernel(const AttnArgs g) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long prefix[kAttnThreads + 1];
  __shared__ long long start_base;
  __shared__ int start_seq;
  __shared__ float2 warp_ml[kAttnWarps][S::HB];
  __shared__ bool is_last;
  using A = Attn<S>;
  constexpr int DP = S::DP, NT = S::NT, HB = S::HB;

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
  const int per = (n_seq + kAttnThreads - 1) / kAttnThreads;
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
  const long long U = prefix[kAttnThreads];
  const long long B = min((long long)gridDim.x, U);

  // rows that see nothing
  for (int s = b; s < n_seq; s += gridDim.x) {
    bool bad;
    if (A::units_of(g, A::clipped_len(g, s, &bad)) != 0) continue;
    for (int i = tid; i < g.a.n_heads * D; i += kAttnThreads)
      g.a.out[(long long)s * g.a.n_heads * D + i] = 0.0f;
    if (g.a.lse)
      for (int i = tid; i < g.a.n_heads; i += kAttnThreads)
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
    const int t0 = A::first_seen(g, len) + u0 * kUnit;
    const int t1 = min(len, t0 + (u1 - u0) * kUnit);
    const int32_t* table = g.a.table + (long long)seq * g.a.max_pages;
    const uint8_t* kpool = static_cast<const uint8_t*>(C.d_k) + kvh * C.head_stride * S::ES;
    const uint8_t* vpool = static_cast<const uint8_t*>(C.d_v) + kvh * C.head_stride * S::ES;

    // ---- the ring: tile i of this warp starts at t0 + (i * warps + warp) * 16 --------------------
    const int tiles = (t1 - t0 + kTile - 1) / kTile;
    const int mine = tiles > warp ? (tiles - warp + kAttnWarps - 1) / kAttnWarps : 0;
    auto page_entry = [&](int i) {  // lane l < 16: the table's entry for position l of tile i
      const int pos = t0 + (i * kAttnWarps + warp) * kTile + lane;
      return i < mine && lane < kTile && pos < t1 ? __ldg(table + A::page_of(g, pos)) : 0;
    };
    auto issue = [&](int i, int page, uint32_t* seen) {
      if (i < mine) {
        const int pos = t0 + (i * kAttnWarps + warp) * kTile + lane;
        long long off = -1;
        if (lane < kTile && pos < t1) {
          if (page >= 0 && page < C.n_pages)
            off = (page * C.page_stride +
                   (long long)(pos - A::page_of(g, pos) * C.page_size) * C.token_stride) * S::ES;
          else
            record_status(g.a.status, SPAX_ERR_INDEX);
        }
        *seen = __ballot_sync(~0u, off >= 0);
        const uint32_t stage = ring + (i % S::STAGES) * S::STAGE;
#pragma unroll
        for (int k = 0; k < kTile * S::CH / 32; ++k) {
          const int e = k * 32 + lane, row_ = e / S::CH, ch = e % S::CH;
          const long long o = __shfl_sync(~0u, off, row_);
          const bool real = o >= 0 && ch < chunks;
          const long long at = real ? o + ch * 16 : 0;
          // keys: rows of unlike parity in different halves of the banks; values: pairs of rows
          const int kc = S::CH >= 8 ? ch ^ ((row_ & 1) << 2) : ch;
          const int vc = S::CH >= 8 ? ch ^ (((row_ >> 1) & 3) << 1) : ch ^ (((row_ >> 1) & 1) << 1);
          cp16(stage + row_ * S::ROW + kc * 16, kpool + at, real);
          cp16(stage + S::HALF + row_ * S::ROW + vc * 16, vpool + at, real);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t seen[S::STAGES] = {};
    int page = page_entry(0);
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; ++i) {
      const int next = page_entry(i + 1);
      issue(i, page, &seen[i]);
      page = next;
    }

    // ---- the query's parts, and the factor from a product to a score in powers of two ------------
    uint32_t qr[S::QREG ? S::KS * 3 * NT * 2 : 1];
    float factor[NT][2];
    if (!S::QREG) __syncthreads();  // the last segment's readers are done
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
      for (int ks = 0; ks < S::KS; ++ks) {
        float4 v = entries(ks);
        v.x *= up, v.y *= up, v.z *= up, v.w *= up;
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          const uint32_t b0 = take_part<S::E4M3>(v.x, v.y), b1 = take_part<S::E4M3>(v.z, v.w);
          const int at = (ks * 3 + p) * NT + nt;
          if constexpr (S::QREG) {
            qr[at * 2] = b0;
            qr[at * 2 + 1] = b1;
          } else if (warp == 0) {
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qsm + at * 256 + lane * 8), "r"(b0), "r"(b1));
          }
        }
      }
      // the columns of a score fragment are heads 2c, 2c + 1
      const float f = g.a.prm.scale * C.k_scale * down;
      factor[nt][0] = __shfl_sync(~0u, f, (2 * c) * 4);
      factor[nt][1] = __shfl_sync(~0u, f, (2 * c + 1) * 4);
    }
    if (!S::QREG) __syncthreads();
    const float cap = g.a.prm.softcap, cap_inv = cap > 0.0f ? 1.0f / cap : 0.0f;

    // ---- tiles ------------------------------------------------------------------------------------
    // Exponents are taken from a base that trails the maximum by up to kSlack powers of two (it moves
    // only when a score passes it by more), and fp16 probabilities are lifted by 2^12 so that their
    // parts stay normal numbers (and their sums are lowered again, exactly, at the end).
    constexpr float kSlack = S::E4M3 ? 3.0f : 8.0f, kLift = S::E4M3 ? 12.0f : 0.0f,
                    kDrop = S::E4M3 ? 1.0f / 4096.0f : 1.0f;
    float m[NT][2], l[NT][2], o[NT][DP / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
    }
    for (int i = 0; i < mine; ++i) {
      {
        const int next = page_entry(i + S::STAGES);
        uint32_t now = 0;
        issue(i + S::STAGES - 1, page, &now);
        page = next;
#pragma unroll
        for (int k = 0; k < S::STAGES; ++k)
          if ((i + S::STAGES - 1) % S::STAGES == k) seen[k] = now;
      }
      asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t ks_at = ring + (i % S::STAGES) * S::STAGE, vs_at = ks_at + S::HALF;
      uint32_t here = 0;
#pragma unroll
      for (int k = 0; k < S::STAGES; ++k)
        if (i % S::STAGES == k) here = seen[k];

      // scores: four chains (even and odd steps of the first part, the second, the third)
      float acc[NT][4][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][k][0] = acc[nt][k][1] = acc[nt][k][2] = acc[nt][k][3] = 0.0f;
      auto step = [&](int ks, const uint32_t(&a)[4]) {
        uint32_t fin[4];
        finite_pairs<S::E4M3>(a, fin);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int p = 2; p >= 0; --p) {
            const int at = (ks * 3 + p) * NT + nt;
            uint32_t b0, b1;
            if constexpr (S::QREG) {
              b0 = qr[at * 2];
              b1 = qr[at * 2 + 1];
            } else {
              const uint2 v = lds64(qsm + at * 256 + lane * 8);
              b0 = v.x;
              b1 = v.y;
            }
            if (p == 0)
              mma16816(acc[nt][ks & 1], a, b0, b1, S::E4M3);
            else
              mma16816(acc[nt][p + 1], fin, b0, b1, S::E4M3);
          }
      };
#pragma unroll
      for (int j = 0; j < S::CH / 4; ++j) {
        const int kc = S::CH >= 8 ? (c + 4 * j) ^ ((r & 1) << 2) : c + 4 * j;
        const uint4 top = lds128(ks_at + r * S::ROW + kc * 16);
        const uint4 low = lds128(ks_at + (r + 8) * S::ROW + kc * 16);
        if constexpr (S::E4M3) {
          const uint32_t tw[4] = {top.x, top.y, top.z, top.w}, lw[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a[4] = {e4m3x2_to_f16x2(tw[k] & 0xFFFF), e4m3x2_to_f16x2(lw[k] & 0xFFFF),
                                   e4m3x2_to_f16x2(tw[k] >> 16), e4m3x2_to_f16x2(lw[k] >> 16)};
            step(4 * j + k, a);
          }
        } else {
          const uint32_t a0[4] = {top.x, low.x, top.y, low.y}, a1[4] = {top.z, low.z, top.w, low.w};
          step(2 * j, a0);
          step(2 * j + 1, a1);
        }
      }

      uint32_t pb[NT][3][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[k] = ((acc[nt][3][k] + acc[nt][2][k]) + acc[nt][1][k]) + acc[nt][0][k];
          s[k] *= factor[nt][k & 1];
          if (cap > 0.0f) s[k] = cap * tanhf(s[k] * cap_inv);
          s[k] *= kLog2e;
        }
        if (here != 0xFFFFu) {
          if (!(here >> r & 1)) s[0] = s[1] = -INFINITY;
          if (!(here >> (r + 8) & 1)) s[2] = s[3] = -INFINITY;
        }
        const bool up = s[0] > m[nt][0] + kSlack || s[2] > m[nt][0] + kSlack ||
                        s[1] > m[nt][1] + kSlack || s[3] > m[nt][1] + kSlack;
        if (__any_sync(~0u, up)) {
          float n0 = fmaxf(m[nt][0], fmaxf(s[0], s[2])), n1 = fmaxf(m[nt][1], fmaxf(s[1], s[3]));
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(~0u, n0, k));
            n1 = fmaxf(n1, __shfl_xor_sync(~0u, n1, k));
          }
          // a column that has seen only -inf keeps its zero sum
          const float f0 = n0 == -INFINITY ? 1.0f : exp2f(m[nt][0] - n0);
          const float f1 = n1 == -INFINITY ? 1.0f : exp2f(m[nt][1] - n1);
          m[nt][0] = n0;
          m[nt][1] = n1;
          l[nt][0] *= f0;
          l[nt][1] *= f1;
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            o[nt][k][0] *= f0;
            o[nt][k][1] *= f1;
            o[nt][k][2] *= f0;
            o[nt][k][3] *= f1;
          }
        }
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float base_ = m[nt][k & 1] == -INFINITY ? 0.0f : m[nt][k & 1] - kLift;
          p[k] = exp2f(s[k] - base_);
        }
        l[nt][0] += p[0] + p[2];
        l[nt][1] += p[1] + p[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
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
            const uint32_t x0 = __byte_perm(w[0][q / 2], w[1][q / 2], sel);
            const uint32_t x1 = __byte_perm(w[2][q / 2], w[3][q / 2], sel);
            a[0] = e4m3x2_to_f16x2(x0 & 0xFFFF);
            a[1] = e4m3x2_to_f16x2(x0 >> 16);
            a[2] = e4m3x2_to_f16x2(x1 & 0xFFFF);
            a[3] = e4m3x2_to_f16x2(x1 >> 16);
          } else {
            a[0] = __byte_perm(w[0][q], w[1][q], 0x5410);
            a[1] = __byte_perm(w[0][q], w[1][q], 0x7632);
            a[2] = __byte_perm(w[2][q], w[3][q], 0x5410);
            a[3] = __byte_perm(w[2][q], w[3][q], 0x7632);
          }
          uint32_t fin[4];
          finite_pairs<S::E4M3>(a, fin);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 2; k > 0; --k) mma16816(t, fin, pb[nt][k][0], pb[nt][k][1], S::E4M3);
            mma16816(t, a, pb[nt][0][0], pb[nt][0][1], S::E4M3);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][4 * j + q][k] += t[k];
          }
        }
      }
      __syncwarp();  // every lane is done with the stage before it is filled again
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

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
    for (int e = tid; e < heads * quads; e += kAttnThreads) {
      const int h = e / quads, d = (e - h * quads) * 4;
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, warp_ml[w][h].x);
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        // fmaxf drops a NaN maximum; its warp's sum is NaN and brings it back
        const float f = warp_ml[w][h].x == -INFINITY ? 0.0f : exp2f(warp_ml[w][h].x - M);
        if (f == 0.0f && warp_ml[w][h].y == 0.0f) continue;
        const float4 t = *reinterpret_cast<const float4*>(os + (w * HB + h) * S::OS + d);
        L += f * warp_ml[w][h].y;
        v.x += f * t.x, v.y += f * t.y, v.z += f * t.z, v.w += f * t.w;
      }
      const long long at = (long long)seq * g.a.n_heads + head0 + h;
      if (whole) {
        const float inv = L == 0.0f ? 0.0f : C.v_scale / L;
        if (L == 0.0f) v = make_float4(0, 0, 0, 0);
        v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
        *reinterpret_cast<float4*>(g.a.out + at * D + d) = v;
        if (d == 0 && g.a.lse) g.a.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(g.part + ((long long)slot * HB + h) * DP + d) = v;
        if (d == 0) g.part_ml[slot * HB + h] = make_float2(M, L);
      }
    }

    // ---- a shared row: the last CTA to arrive joins its parts ----------------------------------------
    if (!whole) {
      const int b0 = (int)(((row_begin + 1) * B - 1) / U), b1 = (int)((row_end * B - 1) / U);
      const int n = b1 - b0 + 1;
      // the first CTA's slot: its first segment if its run starts in this row
      const int slot0 = 2 * b0 + (row_begin <= U * b0 / B ? 0 : 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        is_last = atomicAdd(g.tickets + slot0, 1u) == (uint32_t)(n - 1);
        if (is_last) g.tickets[slot0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (is_last) {
        auto slot_of = [&](int k) { return k == 0 ? slot0 : 2 * (b0 + k); };
        for (int e = tid; e < heads * quads; e += kAttnThreads) {
          const int h = e / quads, d = (e - h * quads) * 4;
          float M = -INFINITY, L = 0.0f;
          for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(g.part_ml + slot_of(k) * HB + h).x);
          float4 v = make_float4(0, 0, 0, 0);
          for (int k = 0; k < n; ++k) {
            const float2 ml = __ldcg(g.part_ml + slot_of(k) * HB + h);
            const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
            if (f == 0.0f && ml.y == 0.0f) continue;
            const float4 t = __ldcg(reinterpret_cast<const float4*>(
                g.part + ((long long)slot_of(k) * HB + h) * DP + d));
            L += f * ml.y;
            v.x += f * t.x, v.y += f * t.y, v.z += f * t.z, v.w += f * t.w;
          }
          const float inv = L == 0.0f ? 0.0f : C.v_scale / L;
          if (L == 0.0f) v = make_float4(0, 0, 0, 0);
          v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
          const long long at = (long long)seq * g.a.n_heads + head0 + h;
          *reinterpret_cast<float4*>(g.a.out + at * D + d) = v;
          if (d == 0 && g.a.lse) g.a.lse[at] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
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

// Blocks of query heads: 16 at a time where a key head has more than 8 and the outputs fit the
// registers (head_dim up to 128), else 8.
static int head_blocks(int row_heads, int head_dim) { return row_heads > 8 && head_dim <= 128 ? 2 : 1; }

static int padded_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

size_t attention_ws_bytes(int n_heads, int n_kv_heads, int head_dim, int sm_count) {
  const size_t hb = 8 * head_blocks(n_heads / n_kv_heads, head_dim);
  const size_t slots = 2 * 2 * (size_t)sm_count;  // two for each CTA, at most two CTAs on an SM
  return slots * hb * (padded_dim(head_dim) * 4 + 8) + ((slots * 4 + 255) & ~size_t(255));
}

template <int DP, bool E4M3, int NT>
static cudaError_t launch_shape(AttnArgs g, int sm_count, cudaStream_t stream) {
  using S = AttnShape<DP, E4M3, NT>;
  const void* f = reinterpret_cast<const void*>(attention_kernel<S>);
  cudaError_t e = ensure_smem_limit(f, S::SMEM);
  if (e != cudaSuccess) return e;
  g.blocks = (g.row_heads + S::HB - 1) / S::HB;
  const long long slots = 4ll * sm_count;
  g.tickets = static_cast<uint32_t*>(g.a.ws);
  g.part = reinterpret_cast<float*>(static_cast<uint8_t*>(g.a.ws) + ((slots * 4 + 255) & ~255ll));
  g.part_ml = reinterpret_cast<float2*>(g.part + slots * S::HB * DP);
  long long longest = (long long)g.a.max_pages * g.a.cache.page_size;
  if (g.a.prm.window > 0 && g.a.prm.window < longest) longest = g.a.prm.window;
  const long long units = (long long)g.a.n_seq * g.a.cache.n_kv_heads * g.blocks *
                          ((longest + kUnit - 1) / kUnit);
  const long long wave = (long long)S::CTAS * sm_count;
  return launch_pdl(attention_kernel<S>, dim3((unsigned)(units < wave ? units : wave)),
                    dim3(kAttnThreads), (size_t)S::SMEM, stream, g);
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
  const int dp = padded_dim(a.cache.head_dim), nt = head_blocks(g.row_heads, a.cache.head_dim);
  const bool e = a.cache.dtype == SPAX_KV_E4M3;
  if (dp == 64 && nt == 1) return e ? launch_shape<64, true, 1>(g, sm_count, stream) : launch_shape<64, false, 1>(g, sm_count, stream);
  if (dp == 64) return e ? launch_shape<64, true, 2>(g, sm_count, stream) : launch_shape<64, false, 2>(g, sm_count, stream);
  if (dp == 128 && nt == 1) return e ? launch_shape<128, true, 1>(g, sm_count, stream) : launch_shape<128, false, 1>(g, sm_count, stream);
  if (dp == 128) return e ? launch_shape<128, true, 2>(g, sm_count, stream) : launch_shape<128, false, 2>(g, sm_count, stream);
  return e ? launch_shape<256, true, 1>(g, sm_count, stream) : launch_shape<256, false, 1>(g, sm_count, stream);
}

}  // namespace spax
