// attention.cu — attention of one new token of each sequence over the paged key-value cache.
#include "layer.cuh"

namespace spax {

constexpr int kAttnThreads = 128;

__device__ __forceinline__ float cache_value(const spax_kv_cache& c, const void* pool, long long at) {
  if (c.dtype == SPAX_KV_BF16)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(pool)[at] << 16);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(pool)[at], __NV_E4M3)));
}

__device__ __forceinline__ float block_reduce(float v, bool max, float* red) {
  for (int o = 16; o; o >>= 1) {
    const float u = __shfl_xor_sync(~0u, v, o);
    v = max ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kAttnThreads / 32; ++w) v = max ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

// One CTA for each (sequence, query head): tiles of 128 positions, one score for each thread, a
// running maximum and sum, and two output entries for each thread.
__global__ void __launch_bounds__(kAttnThreads) attention_kernel(const AttnLaunch a) {
  __shared__ float q[256], p[kAttnThreads], red[kAttnThreads / 32];
  __shared__ long long off[kAttnThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int seq = blockIdx.y, head = blockIdx.x, D = a.cache.head_dim;
  const int kvh = head / (a.n_heads / a.cache.n_kv_heads);
  int len = a.lens[seq];
  if (len < 0 || len > a.max_pages * a.cache.page_size) {
    if (threadIdx.x == 0) record_status(a.status, SPAX_ERR_INDEX);
    len = 0;
  }
  const int lo = a.prm.window > 0 ? max(0, len - a.prm.window) : 0;
  for (int i = threadIdx.x; i < D; i += kAttnThreads) q[i] = a.q[seq * a.q_stride + head * D + i];
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
  for (int j0 = lo; j0 < len; j0 += kAttnThreads) {
    const int j = j0 + threadIdx.x;
    long long at = -1;
    float s = -INFINITY;
    if (j < len) {
      at = cache_row(a.cache, a.table + (long long)seq * a.max_pages, j);
      if (at < 0) record_status(a.status, SPAX_ERR_INDEX);
    }
    if (at >= 0) {
      at += kvh * a.cache.head_stride;
      float acc = 0.0f;
      for (int i = 0; i < D; ++i) acc = fmaf(q[i], cache_value(a.cache, a.cache.d_k, at + i), acc);
      s = acc * a.prm.scale * a.cache.k_scale;
      if (a.prm.softcap > 0.0f) s = a.prm.softcap * tanhf(s / a.prm.softcap);
    }
    const float m_new = fmaxf(m, block_reduce(s, true, red));
    const float base = m_new == -INFINITY ? 0.0f : m_new;
    p[threadIdx.x] = expf(s - base);
    off[threadIdx.x] = at;
    const float fade = expf(m - base);
    l = l * fade + block_reduce(p[threadIdx.x], false, red);
    m = m_new;
    for (int k = 0; k < 2; ++k) {
      const int i = threadIdx.x + k * kAttnThreads;
      if (i >= D) break;
      float acc = 0.0f;
      for (int u = 0; u < min(kAttnThreads, len - j0); ++u)
        if (off[u] >= 0) acc = fmaf(p[u], cache_value(a.cache, a.cache.d_v, off[u] + i), acc);
      o[k] = o[k] * fade + acc;
    }
    __syncthreads();
  }
  const float inv = l > 0.0f ? a.cache.v_scale / l : l == 0.0f ? 0.0f : l;
  for (int k = 0; k < 2; ++k) {
    const int i = threadIdx.x + k * kAttnThreads;
    if (i < D) a.out[((long long)seq * a.n_heads + head) * D + i] = o[k] * inv;
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(long long)seq * a.n_heads + head] = l == 0.0f ? -INFINITY : m + logf(l);
}

size_t attention_ws_bytes(int, int, int, int) { return 256; }

cudaError_t launch_paged_attention(const AttnLaunch& a, int, cudaStream_t stream) {
  return launch_pdl(attention_kernel, dim3(a.n_heads, a.n_seq), dim3(kAttnThreads), 0, stream, a);
}

}  // namespace spax
