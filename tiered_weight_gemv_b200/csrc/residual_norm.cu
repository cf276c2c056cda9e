// residual_norm.cu — r = res_scale * h + out_scale * gate * N_post(y), x = N_pre(r), by rows.
#include "layer.cuh"

namespace spax {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float norm_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kNormThreads / 32; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ float weight_at(const spax_norm& n, const void* w, int i, float none) {
  if (!w) return none;
  if (n.w_dtype == SPAX_W_FP32) return static_cast<const float*>(w)[i];
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(w)[i] << 16);
}

// The norm of the row z (in shared memory), in place.
__device__ void norm_row(const spax_norm& n, float* z, int d, float* red) {
  float mean = 0.0f;
  if (n.kind == SPAX_NORM_LAYER) {
    float s = 0.0f;
    for (int i = threadIdx.x; i < d; i += kNormThreads) s += z[i];
    mean = norm_sum(s, red) / d;
  }
  float s = 0.0f;
  for (int i = threadIdx.x; i < d; i += kNormThreads) s = fmaf(z[i] - mean, z[i] - mean, s);
  const float inv = 1.0f / sqrtf(norm_sum(s, red) / d + n.eps);
  for (int i = threadIdx.x; i < d; i += kNormThreads)
    z[i] = fmaf((z[i] - mean) * inv, weight_at(n, n.d_weight, i, 1.0f), weight_at(n, n.d_bias, i, 0.0f));
}

__global__ void __launch_bounds__(kNormThreads) residual_norm_kernel(const NormLaunch a) {
  extern __shared__ float z[];
  __shared__ float red[kNormThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const long long row = (long long)blockIdx.x * a.d;
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) z[i] = a.y ? a.y[row + i] : 0.0f;
  if (a.y && a.has_post) norm_row(a.post, z, a.d, red);
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
    const float g = a.y && a.gate ? a.gate[blockIdx.x * a.gate_stride + i] : 1.0f;
    const float r = a.res_scale * a.h[row + i] + (a.y ? a.out_scale * (z[i] * g) : 0.0f);
    z[i] = r;
    if (a.r) a.r[row + i] = r;
  }
  if (!a.x) return;
  if (a.has_pre) norm_row(a.pre, z, a.d, red);
  for (int i = threadIdx.x; i < a.d; i += kNormThreads) a.x[row + i] = z[i];
}

cudaError_t launch_residual_norm(const NormLaunch& a, cudaStream_t stream) {
  const int smem = a.d * 4;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(residual_norm_kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(residual_norm_kernel, dim3(a.n_tok), dim3(kNormThreads), (size_t)smem, stream, a);
}

}  // namespace spax
