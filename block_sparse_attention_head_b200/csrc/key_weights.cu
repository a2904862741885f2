// The attention mass of packed prompts' keys (instagen_key_weights).  Simple
// form: one warp per key, with the d elements of a row spread over the lanes.
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kRowThreads = 128;

// The sequence that row t belongs to (-1: none), found by the whole warp.
__device__ __forceinline__ int find_seq(const int32_t* cu, int nseq, int T, int t, int& lo, int& hi) {
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < nseq; s0 += 32) {
    const int s = s0 + lane;
    int l = 0, h = 0;
    if (s < nseq) seq_rows(cu, s, T, l, h);
    const unsigned hit = __ballot_sync(0xffffffffu, t >= l && t < h);
    if (hit) {
      const int src = __ffs(hit) - 1;
      lo = __shfl_sync(0xffffffffu, l, src);
      hi = __shfl_sync(0xffffffffu, h, src);
      return s0 + src;
    }
  }
  return -1;
}

template <typename T, int D>
__device__ __forceinline__ float row_dot(const float (&q)[D / 32], const T* k) {
  const int lane = threadIdx.x & 31;
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) s = fmaf(q[e], to_f32(k[lane + 32 * e]), s);
  return warp_sum(s);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) key_weights_rows_kernel(PromptArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)a.Tk * a.Hkv) return;
  const int j = (int)(row / a.Hkv), hk = (int)(row % a.Hkv);
  int q0, q1, k0, k1;
  const int s = find_seq(a.cu_k, a.nseq, a.Tk, j, k0, k1);
  if (s < 0) return;
  seq_rows(a.cu_q, s, a.Tq, q0, q1);
  const int first = a.causal ? max(0, (j - k0) - ((k1 - k0) - (q1 - q0))) : 0;
  const T* k = static_cast<const T*>(a.K) + j * a.k_tok + hk * a.k_head;
  float kf[D / 32], w = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) kf[e] = to_f32(k[lane + 32 * e]);
  for (int g = 0; g < a.G; ++g) {
    const int h = hk * a.G + g;
    for (int t = q0 + first; t < q1; ++t) {
      const float lse = a.lse[(size_t)h * a.Tq + t];
      const float x = row_dot<T, D>(kf, static_cast<const T*>(a.Q) + t * a.q_tok + h * a.q_head) * a.scale_log2;
      w += lse == -INFINITY ? 0.f : exp2f(x - lse * kLog2E);
    }
  }
  if (lane == 0) a.weights[(size_t)hk * a.Tk + j] += w;
}
}  // namespace

size_t key_weights_ws(const PromptArgs&) { return 256; }

template <typename F>
static cudaError_t by_type(int dtype, int d, F f) {
  if (dtype == IG_BF16) return d == 128 ? f((__nv_bfloat16)0.f, std::integral_constant<int, 128>())
                                        : f((__nv_bfloat16)0.f, std::integral_constant<int, 64>());
  return d == 128 ? f((__half)0.f, std::integral_constant<int, 128>())
                  : f((__half)0.f, std::integral_constant<int, 64>());
}

cudaError_t launch_key_weights(const PromptArgs& a, cudaStream_t s) {
  const long long rows = (long long)a.Tk * a.Hkv;
  if (rows == 0 || a.Tq == 0) return cudaSuccess;
  return by_type(a.dtype, a.d, [&](auto t, auto d) {
    key_weights_rows_kernel<decltype(t), decltype(d)::value>
        <<<(unsigned)((rows + 3) / 4), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace ig
