// kv_append.cu — rotate q and k by position and write k and v into the paged cache.
//
// A token's heads are cut into items of 8 entries: 4 pairs of a rotated head, 8 neighbours of what
// is not turned. An item is two 16-byte loads and the stores of the same entries, so the kernel
// moves each byte once; a prompt is bound by HBM, one token by the chain position -> page -> store.
// The loads of a thread's items therefore go out before the position is known, and the turns of the
// token's pairs are computed once for each CTA, by a thread a pair, while they are in flight.
#include "layer.cuh"

namespace spax {

// The turn of a pair at position pos: cos and sin of pos * f. The angle is formed in fp64 (its error
// is below pos * f * 2^-51 radians), reduced to a fraction of a half turn there and split into two
// floats; the small one enters to first order, cos(a + b) = cos a - b sin a + O(b^2) with b < 2^-23,
// so the result has the accuracy of sincospif.
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

// The turns of a token's pairs, read two at a time in 16 bytes.
struct alignas(16) Turns {
  float2 of[128];
};
static_assert(alignof(Turns) >= sizeof(float4), "the shared array is placed by its type's alignment");

__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  return (uint32_t)to_bf16(x) | ((uint32_t)to_bf16(y) << 16);
}
// Saturates: past 448 (infinities too) it is 448.
__device__ __forceinline__ uint32_t e4m3_quad(float4 v) {
  const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(v.x, v.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(v.z, v.w), __NV_SATFINITE, __NV_E4M3);
  return a | (b << 16);
}

// N items a thread: 1 spreads a few tokens over the GPU; 3 keeps a token in few CTAs, so that its
// turns are computed once, and four CTAs on an SM. Measured on B200, 8000 tokens of 48 heads of 128
// (361 MB): 57 us (6.28 TB/s) with 3, 61 with 4 (a quarter of the threads' items missing there), 70
// with 2; one token of 96 heads 1.9 us, a chain of three dependent loads.
template <int N>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const AppendLaunch a) {
  __shared__ Turns turns;
  float2* const turn = turns.of;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x, tid = threadIdx.x;
  const int D = a.cache.head_dim, K = a.cache.n_kv_heads, H = a.n_heads;
  const int rot = a.rope.rot_dim, half = rot / 2;
  const int pos = a.pos[t];
  const int seq = a.seq ? a.seq[t] : t;
  const double f = tid < half ? a.rope.d_inv_freq[tid] : 0.0;

  const uint32_t per_head = D / 8, items = (uint32_t)(H + 2 * K) * per_head;
  const uint32_t first = (blockIdx.y * N) * kAppendThreads + tid;
  int head[N], da[N], db[N], pair[N];  // pair: of the item's first two entries, -1: not turned
  float4 x[N], y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t e = first + i * kAppendThreads;
    head[i] = e < items ? (int)(e / per_head) : -1;
    if (head[i] < 0) continue;
    const int p = (int)(e - head[i] * per_head);
    const bool turned = 8 * p < rot && head[i] < H + K;
    pair[i] = turned ? 4 * p : -1;
    da[i] = turned && !a.rope.interleaved ? 4 * p : 8 * p;
    db[i] = turned && !a.rope.interleaved ? half + 4 * p : 8 * p + 4;
    const float* src = head[i] < H       ? a.q + t * a.q_stride + (long long)head[i] * D
                       : head[i] < H + K ? a.k + t * a.k_stride + (long long)(head[i] - H) * D
                                         : a.v + t * a.v_stride + (long long)(head[i] - H - K) * D;
    x[i] = *reinterpret_cast<const float4*>(src + da[i]);
    y[i] = *reinterpret_cast<const float4*>(src + db[i]);
  }

  if (pos < 0) return;  // padding (the whole CTA)
  long long off = -1;
  if (seq >= 0 && seq < a.n_seq && pos < a.max_pages * a.cache.page_size)
    off = cache_row(a.cache, a.table + (long long)seq * a.max_pages, pos);
  if (off < 0) {
    if (tid == 0 && blockIdx.y == 0) record_status(a.status, SPAX_ERR_INDEX);
    return;
  }
  if (tid < half) turn[tid] = turn_of(pos, f);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (head[i] < 0) continue;
    if (pair[i] >= 0) {
      const float4 cs01 = *reinterpret_cast<const float4*>(turn + pair[i]);
      const float4 cs23 = *reinterpret_cast<const float4*>(turn + pair[i] + 2);
      auto turn_pair = [](float& u, float& v, float c, float s) {
        const float w = u * c - v * s;
        v = v * c + u * s;
        u = w;
      };
      if (a.rope.interleaved) {
        turn_pair(x[i].x, x[i].y, cs01.x, cs01.y);
        turn_pair(x[i].z, x[i].w, cs01.z, cs01.w);
        turn_pair(y[i].x, y[i].y, cs23.x, cs23.y);
        turn_pair(y[i].z, y[i].w, cs23.z, cs23.w);
      } else {
        turn_pair(x[i].x, y[i].x, cs01.x, cs01.y);
        turn_pair(x[i].y, y[i].y, cs01.z, cs01.w);
        turn_pair(x[i].z, y[i].z, cs23.x, cs23.y);
        turn_pair(x[i].w, y[i].w, cs23.z, cs23.w);
      }
    }
    if (head[i] < H) {
      float* dst = a.q_out + t * a.q_out_stride + (long long)head[i] * D;
      *reinterpret_cast<float4*>(dst + da[i]) = x[i];
      *reinterpret_cast<float4*>(dst + db[i]) = y[i];
      continue;
    }
    const bool keys = head[i] < H + K;
    void* pool = keys ? a.cache.d_k : a.cache.d_v;
    const long long at = off + (head[i] - H - (keys ? 0 : K)) * a.cache.head_stride;
    if (a.cache.dtype == SPAX_KV_BF16) {
      uint16_t* dst = static_cast<uint16_t*>(pool) + at;
      *reinterpret_cast<uint2*>(dst + da[i]) = make_uint2(bf16_pair(x[i].x, x[i].y), bf16_pair(x[i].z, x[i].w));
      *reinterpret_cast<uint2*>(dst + db[i]) = make_uint2(bf16_pair(y[i].x, y[i].y), bf16_pair(y[i].z, y[i].w));
    } else {
      const float s = keys ? a.cache.k_scale : a.cache.v_scale;
      auto scaled = [s](float4 v) {
        return make_float4(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s), __fdiv_rn(v.z, s), __fdiv_rn(v.w, s));
      };
      uint8_t* dst = static_cast<uint8_t*>(pool) + at;
      *reinterpret_cast<uint32_t*>(dst + da[i]) = e4m3_quad(scaled(x[i]));
      *reinterpret_cast<uint32_t*>(dst + db[i]) = e4m3_quad(scaled(y[i]));
    }
  }
}

cudaError_t launch_kv_append(const AppendLaunch& a, int sm_count, cudaStream_t stream) {
  const long long items = (long long)(a.n_heads + 2 * a.cache.n_kv_heads) * (a.cache.head_dim / 8);
  const long long ctas = (items + kAppendThreads - 1) / kAppendThreads;
  // one item a thread while that is at most four CTAs an SM
  if (a.n_tok * ctas <= 4 * sm_count)
    return launch_pdl(kv_append_kernel<1>, dim3(a.n_tok, (unsigned)ctas), dim3(kAppendThreads), 0, stream, a);
  return launch_pdl(kv_append_kernel<3>, dim3(a.n_tok, (unsigned)((ctas + 2) / 3)), dim3(kAppendThreads), 0,
                    stream, a);
}

}  // namespace spax
