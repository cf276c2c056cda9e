// residual_norm.cu — r = res_scale * h + out_scale * gate * N_post(y), x = N_pre(r), by rows.
//
// One CTA for each row (a cluster for a wide one), which stays in registers from its load to its last
// store: h and y are read once, r and x written once, so many rows are bound by HBM and one row by
// the latency of its loads and of one block sum for each norm (two with a mean: the deviations are
// taken from the rounded mean itself, in a second sum, not from a difference of squares).
//
// Measured on B200 (a copy's rate is 6.55 TB/s): 8192 rows of 4096, RMS, 81 us (6.63 TB/s); 4001 rows
// of 5004 with both LAYER norms, biases and a gate of each token 71 us (5.65 TB/s), and of 5003, whose
// rows start off the 16-byte boundary, 88 us (4.55 TB/s; 132 with single values: the instructions of
// addresses and checks bound it); 2000 rows of 16384 with the same 155 us (4.2 TB/s) and 600 of 28672 97
// us (3.6 TB/s), bound by four block sums in turn, each a cluster's barrier there. One row of 4096 2.3
// us, of 28672 3.2 us (a cluster of 8; 16 us in one CTA, whose registers it overflows).
#include "layer.cuh"

namespace spax {

// A thread's values of a row: N pieces of W neighbours, 32 W apart, so that a warp covers 32 N W values
// in a row and all of a thread's addresses are one base plus constants. Rows that start off a 16-byte
// boundary (an odd d) take W = 4 with SHIFT: every piece then starts `shift` values early, on the
// boundary before, and the first and the last piece of a row, and the weights, are taken value by
// value.
// Loads of a thread's pieces go out together; where all of them lie in the row (full), unchecked.
template <int W, int N, bool SHIFT>
struct Row {
  int at;  // index in the row of the thread's first value (negative where that lies before the row)
  int d;
  bool full;

  __device__ __forceinline__ bool whole(int i) const {
    const int e = at + i * 32 * W;
    return full || (SHIFT ? e >= 0 && e + 4 <= d : e < d);  // without a shift d is a multiple of W
  }
  __device__ __forceinline__ bool real(int i, int k) const {
    return full || (unsigned)(at + i * 32 * W + k) < (unsigned)d;
  }

  template <bool CHECK>
  __device__ __forceinline__ void load_as(const float* p, float (&v)[N][W]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!CHECK || whole(i)) {
        if constexpr (W == 4) {
          const float4 t = *reinterpret_cast<const float4*>(p + i * 128);
          v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
        } else {
          v[i][0] = p[i * 32];
        }
      } else if constexpr (SHIFT) {
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (real(i, k)) v[i][k] = p[i * 32 * W + k];
      }
    }
  }
  // The row's values from p (the row's first) on; those outside the row are left as they are.
  __device__ __forceinline__ void load(const float* p, float (&v)[N][W]) const {
    if (full)
      load_as<false>(p + at, v);
    else
      load_as<true>(p + at, v);
  }
  __device__ __forceinline__ void store(float* p, const float (&v)[N][W]) const {
    p += at;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (whole(i)) {
        if constexpr (W == 4)
          *reinterpret_cast<float4*>(p + i * 128) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        else
          p[i * 32] = v[i][0];
      } else if constexpr (SHIFT) {
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (real(i, k)) p[i * 32 * W + k] = v[i][k];
      }
    }
  }

  static __device__ __forceinline__ float4 four(const float* w) { return *reinterpret_cast<const float4*>(w); }
  static __device__ __forceinline__ float4 four(const uint16_t* w) {
    const uint2 t = *reinterpret_cast<const uint2*>(w);
    return make_float4(__uint_as_float(t.x << 16), __uint_as_float(t.x & 0xFFFF0000u),
                       __uint_as_float(t.y << 16), __uint_as_float(t.y & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float one(const float* w) { return *w; }
  static __device__ __forceinline__ float one(const uint16_t* w) { return __uint_as_float((uint32_t)*w << 16); }

  // The same of a vector that all rows share: single values where the pieces are shifted.
  template <bool CHECK, class T>
  __device__ __forceinline__ void load_shared_as(const T* w, float (&v)[N][W]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (W == 4 && !SHIFT) {
        if (!CHECK || whole(i)) {
          const float4 t = four(w + i * 128);
          v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (!CHECK || real(i, k)) v[i][k] = one(w + i * 32 * W + k);
      }
    }
  }
  template <class T>
  __device__ __forceinline__ void load_shared(const T* w, float (&v)[N][W]) const {
    if (full)
      load_shared_as<false>(w + at, v);
    else
      load_shared_as<true>(w + at, v);
  }
  __device__ __forceinline__ void load_weight(const spax_norm& n, const void* w, float (&v)[N][W]) const {
    if (n.w_dtype == SPAX_W_FP32)
      load_shared(static_cast<const float*>(w), v);
    else
      load_shared(static_cast<const uint16_t*>(w), v);
  }
};

// Sums over a row's CTA, or over its cluster of CTAs, in a fixed order: the warps' sums meet in
// shared memory, and the CTAs' are written to every CTA of the cluster (a CTA reads its own copies
// only, so none is gone while another still reads). Each sum has buffers of its own.
struct RowSums {
  float warp[4][32], cta[4][8];
};
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool CLUSTER>
__device__ __forceinline__ float row_sum(float v, RowSums& S, int which) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int warps = blockDim.x / 32, lane = threadIdx.x % 32;
  if (warps > 1) {
    if (lane == 0) S.warp[which][threadIdx.x / 32] = v;
    __syncthreads();
    v = lane < warps ? S.warp[which][lane] : 0.0f;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  }
  if constexpr (CLUSTER) {
    const uint32_t n = cluster_size();
    if (threadIdx.x < n) {
      uint32_t there;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(there)
                   : "r"(smem_u32(&S.cta[which][cluster_rank()])), "r"(threadIdx.x));
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(there), "f"(v) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    v = 0.0f;
    for (uint32_t k = 0; k < n; ++k) v += S.cta[which][k];
  }
  return v;
}

// AHEAD: the weights and the gate are loaded with the row (few rows wait for less; many rows have
// other rows to wait beside).
template <int W, int N, bool SHIFT, bool AHEAD, bool CLUSTER>
__global__ void __launch_bounds__(W * N > 8 ? 512 : 1024, W * N > 8 ? 2 : 1)
    residual_norm_kernel(const NormLaunch a) {
  __shared__ RowSums sums;
  constexpr bool kAhead = AHEAD && W * N <= 8;
  constexpr int A = kAhead ? N : 1;
  if constexpr (CLUSTER) cluster_arrive();  // every CTA has begun before another writes to it
  pdl_wait();
  pdl_launch_dependents();
  const int token = CLUSTER ? blockIdx.x / cluster_size() : blockIdx.x;
  const int thread = threadIdx.x + (CLUSTER ? cluster_rank() * blockDim.x : 0);
  const long long row = (long long)token * a.d;
  Row<W, N, SHIFT> R;
  R.d = a.d;
  R.at = thread / 32 * (32 * N * W) + thread % 32 * W - (SHIFT ? (int)(row & 3) : 0);
  R.full = R.at >= 0 && R.at + (N - 1) * 32 * W + W <= a.d;
  const float inv_d = 1.0f / (float)a.d;
  const bool add = a.y != nullptr, post = add && a.has_post, pre = a.x && a.has_pre;
  auto load_gate = [&](float(&v)[N][W]) {
    if (a.gate_stride == 0)
      R.load_shared(a.gate, v);
    else
      R.load(a.gate + token * a.gate_stride, v);
  };

  float z[N][W], h[N][W];
  float g[A][W], w1[A][W], b1[A][W], w2[A][W], b2[A][W];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < W; ++k) z[i][k] = h[i][k] = 0.0f;
  if (add) R.load(a.y + row, z);
  R.load(a.h + row, h);
  if constexpr (kAhead) {
    if (a.gate) load_gate(g);
    if (post) {
      if (a.post.d_weight) R.load_weight(a.post, a.post.d_weight, w1);
      if (a.post.d_bias) R.load_weight(a.post, a.post.d_bias, b1);
    }
    if (pre) {
      if (a.pre.d_weight) R.load_weight(a.pre, a.pre.d_weight, w2);
      if (a.pre.d_bias) R.load_weight(a.pre, a.pre.d_bias, b2);
    }
  }

  auto times = [&](const float(&v)[N][W]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) z[i][k] *= v[i][k];
  };
  auto plus = [&](const float(&v)[N][W]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) z[i][k] += v[i][k];
  };
  // z normed: with its mean (LAYER) and 1 / sqrt(mean square + eps), values outside the row 0 before
  auto norm = [&](const spax_norm& n, int which, const float(&w)[A][W], const float(&b)[A][W]) {
    float s = 0.0f;
    if (n.kind == SPAX_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) s += z[i][k];
      const float mean = row_sum<CLUSTER>(s, sums, which) * inv_d;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) z[i][k] -= mean;
      if (!R.full) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int k = 0; k < W; ++k)
            if (!R.real(i, k)) z[i][k] = 0.0f;
      }
      s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) s = fmaf(z[i][k], z[i][k], s);
    const float inv = 1.0f / sqrtf(fmaf(row_sum<CLUSTER>(s, sums, which + 1), inv_d, n.eps));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) z[i][k] *= inv;
    float t[N][W];
    if (n.d_weight) {
      if constexpr (kAhead) {
        times(w);
      } else {
        R.load_weight(n, n.d_weight, t);
        times(t);
      }
    }
    if (n.d_bias) {
      if constexpr (kAhead) {
        plus(b);
      } else {
        R.load_weight(n, n.d_bias, t);
        plus(t);
      }
    }
  };
  if constexpr (CLUSTER) cluster_wait();
  if (post) norm(a.post, 0, w1, b1);
  if (a.gate) {
    if constexpr (kAhead) {
      times(g);
    } else {
      float t[N][W];
      load_gate(t);
      times(t);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float hv = a.res_scale * h[i][k];
      z[i][k] = add ? fmaf(a.out_scale, z[i][k], hv) : hv;
    }
  if (!R.full) {  // what lies outside the row may hold anything by now
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (!R.real(i, k)) z[i][k] = 0.0f;
  }
  if (a.r) R.store(a.r + row, z);
  if (!a.x) return;
  if (pre) norm(a.pre, 2, w2, b2);
  R.store(a.x + row, z);
}

template <int W, int N, bool SHIFT, bool AHEAD>
static cudaError_t launch_row(const NormLaunch& a, int ctas, int threads, cudaStream_t stream) {
  if (ctas == 1)
    return launch_pdl(residual_norm_kernel<W, N, SHIFT, AHEAD, false>, dim3(a.n_tok), dim3(threads), 0, stream, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n_tok * ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, residual_norm_kernel<W, N, SHIFT, AHEAD, true>, a);
}

// The shape for pieces of W values: few rows get as many threads as there are pieces of 4 values (or
// of four single values), many rows 4 pieces (8 single values) a thread; a row of more than a CTA
// takes a cluster of 2, 4 or 8 CTAs, which in every shape hold 32768 values.
template <int W, bool SHIFT, bool AHEAD>
static cudaError_t launch_width(const NormLaunch& a, cudaStream_t stream) {
  constexpr int MOST = AHEAD ? (W == 4 ? 1 : 4) : (W == 4 ? 4 : 8);  // pieces a thread
  const int pieces = (a.d + (SHIFT ? 3 : 0) + W - 1) / W;
  const int most = AHEAD ? 1024 : 512;  // threads in a CTA
  int n = MOST;
  while (n > 1 && pieces <= 32 * (n / 2)) n /= 2;
  int ctas = 1;
  while ((long long)ctas * most * n < pieces) ctas *= 2;
  if (ctas > 8) return cudaErrorInvalidValue;
  const int threads = ((pieces + ctas * n - 1) / (ctas * n) + 31) / 32 * 32;
  if constexpr (MOST >= 8)
    if (n == 8) return launch_row<W, 8, SHIFT, AHEAD>(a, ctas, threads, stream);
  if constexpr (MOST >= 4)
    if (n == 4) return launch_row<W, 4, SHIFT, AHEAD>(a, ctas, threads, stream);
  if constexpr (MOST >= 2)
    if (n == 2) return launch_row<W, 2, SHIFT, AHEAD>(a, ctas, threads, stream);
  return launch_row<W, 1, SHIFT, AHEAD>(a, ctas, threads, stream);
}

cudaError_t launch_residual_norm(const NormLaunch& a, int sm_count, cudaStream_t stream) {
  auto aligned = [](const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; };
  auto norm_ok = [&](const spax_norm& n) {
    const uintptr_t to = n.w_dtype == SPAX_W_FP32 ? 16 : 8;
    return aligned(n.d_weight, to) && aligned(n.d_bias, to);
  };
  const bool few = a.n_tok <= sm_count;
  const bool bases = aligned(a.h, 16) && aligned(a.y, 16) && aligned(a.gate, 16) && aligned(a.r, 16) &&
                     aligned(a.x, 16) && norm_ok(a.post) && norm_ok(a.pre);
  if (bases && a.d % 4 == 0 && a.gate_stride % 4 == 0)
    return few ? launch_width<4, false, true>(a, stream) : launch_width<4, false, false>(a, stream);
  // rows at an odd distance, all of them (a gate of every row's own as well) off by the same
  if (bases && !few && (a.gate_stride == 0 || a.gate_stride == a.d))
    return launch_width<4, true, false>(a, stream);
  return few ? launch_width<1, false, true>(a, stream) : launch_width<1, false, false>(a, stream);
}

}  // namespace spax
