// kv_append.cu — rotate q and k by position and write k and v into the paged cache.
#include "layer.cuh"

namespace spax {

// The turn of pair i at position pos: cos and sin of pos * f_i. The angle is reduced to a fraction
// of a turn in fp64 (|error| below 2^-50 turns up to positions of 2^31 at f = 1), split into two
// floats, and the small one applied to first order: cos(a + b) = cos a - b sin a + O(b^2), with
// b < 2^-24, so the result has the accuracy of sincospif itself at any position.
__device__ __forceinline__ float2 turn_of(int pos, double f) {
  const double turns = (double)pos * f * 0.15915494309189533577;  // 1 / 2 pi
  const double half = 2.0 * (turns - rint(turns));                // half turns, in [-1, 1]
  const float hi = (float)half;
  const float b = (float)(half - (double)hi) * 3.14159265358979f;
  float s, c;
  sincospif(hi, &s, &c);
  return make_float2(fmaf(-b, s, c), fmaf(b, c, s));
}

constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendLaunch a) {
  __shared__ float2 turn[128];
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int pos = a.pos[t];
  if (pos < 0) return;  // padding
  const int seq = a.seq ? a.seq[t] : t;
  long long off = -1;
  if (seq >= 0 && seq < a.n_seq && pos < a.max_pages * a.cache.page_size)
    off = cache_row(a.cache, a.table + (long long)seq * a.max_pages, pos);
  if (off < 0) {
    if (threadIdx.x == 0) record_status(a.status, SPAX_ERR_INDEX);
    return;
  }
  const int rot = a.rope.rot_dim, half = rot / 2, D = a.cache.head_dim, K = a.cache.n_kv_heads;
  for (int i = threadIdx.x; i < half; i += kAppendThreads) turn[i] = turn_of(pos, a.rope.d_inv_freq[i]);
  __syncthreads();
  const int heads = a.n_heads + 2 * K;
  // one item: one pair of entries of one head (a pair past the rotated ones has angle 0)
  for (int e = threadIdx.x; e < heads * (D / 2); e += kAppendThreads) {
    const int head = e / (D / 2), i = e - head * (D / 2);
    const bool rotated = i < half && head < a.n_heads + K;
    const int i0 = i < half && !a.rope.interleaved ? i : 2 * i;
    const int i1 = i < half && !a.rope.interleaved ? i + half : 2 * i + 1;
    const bool is_q = head < a.n_heads, is_k = !is_q && head < a.n_heads + K;
    const int h = is_q ? head : is_k ? head - a.n_heads : head - a.n_heads - K;
    const float* src = is_q ? a.q + t * a.q_stride : is_k ? a.k + t * a.k_stride : a.v + t * a.v_stride;
    float x = src[h * D + i0], y = src[h * D + i1];
    if (rotated) {
      const float2 cs = turn[i];
      const float xr = x * cs.x - y * cs.y, yr = y * cs.x + x * cs.y;
      x = xr;
      y = yr;
    }
    if (is_q) {
      float* dst = a.q_out + t * a.q_out_stride + h * D;
      dst[i0] = x;
      dst[i1] = y;
    } else {
      void* pool = is_k ? a.cache.d_k : a.cache.d_v;
      const long long at = off + h * a.cache.head_stride;
      if (a.cache.dtype == SPAX_KV_BF16) {
        uint16_t* dst = static_cast<uint16_t*>(pool) + at;
        dst[i0] = to_bf16(x);
        dst[i1] = to_bf16(y);
      } else {
        const float scale = is_k ? a.cache.k_scale : a.cache.v_scale;
        uint8_t* dst = static_cast<uint8_t*>(pool) + at;
        dst[i0] = to_e4m3(__fdiv_rn(x, scale));
        dst[i1] = to_e4m3(__fdiv_rn(y, scale));
      }
    }
  }
}

cudaError_t launch_kv_append(const AppendLaunch& a, cudaStream_t stream) {
  return launch_pdl(kv_append_kernel, dim3(a.n_tok), dim3(kAppendThreads), 0, stream, a);
}

}  // namespace spax
