// Attention of one new token per sequence over a shared prefix and its own
// cache (instagen_prefix_attention).  Simple form: one warp per query row.
#include "serve.cuh"

namespace ig {

namespace {
template <typename T, int D>
__global__ void __launch_bounds__(128) step_rows_kernel(StepArgs a, float* lse_out) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.Hq) return;
  const int b = (int)(row / a.Hq), h = (int)(row % a.Hq), hk = h / a.G;
  const int n = live_slots(a.lens, b, a.cap);
  const T* q = static_cast<const T*>(a.Q) + b * a.q_seq + h * D;
  float qf[D / 32], o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    qf[e] = to_f32(q[lane + 32 * e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int part = 0; part < 2; ++part) {
    const size_t off = part ? ((size_t)b * a.Hkv + hk) * a.cap * D : (size_t)hk * a.prefix_head;
    const T* k = static_cast<const T*>(part ? a.Kc : a.Kp) + off;
    const T* v = static_cast<const T*>(part ? a.Vc : a.Vp) + off;
    const int keys = part ? n : a.P;
    for (int j = 0; j < keys; ++j) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) x = fmaf(qf[e], to_f32(k[(size_t)j * D + lane + 32 * e]), x);
      x = warp_sum(x) * a.scale_log2;
      const float mn = fmaxf(m, x);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float alpha = exp2f(m - base), p = exp2f(x - base);
      l = l * alpha + p;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) o[e] = o[e] * alpha + p * to_f32(v[(size_t)j * D + lane + 32 * e]);
      m = mn;
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  T* dst = static_cast<T*>(a.O) + (size_t)row * D;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) dst[lane + 32 * e] = from_f32<T>(o[e] * inv);
  if (lane == 0) {
    const float lse = (m + log2f(l)) * kLn2;
    if (a.lse) a.lse[row] = lse;
    if (lse_out) lse_out[row] = lse;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(128) step_weights_kernel(StepArgs a, const float* lse) {
  const int bh = blockIdx.y, b = bh / a.Hkv, hk = bh % a.Hkv;
  const int n = live_slots(a.lens, b, a.cap);
  const int j = blockIdx.x * 128 + threadIdx.x;
  if (j >= n) return;
  const T* k = static_cast<const T*>(a.Kc) + ((size_t)bh * a.cap + j) * D;
  float w = 0.f;
  for (int g = 0; g < a.G; ++g) {
    const int h = hk * a.G + g;
    const T* q = static_cast<const T*>(a.Q) + b * a.q_seq + h * D;
    float x = 0.f;
    for (int e = 0; e < D; ++e) x = fmaf(to_f32(q[e]), to_f32(k[e]), x);
    w += exp2f(x * a.scale_log2 - lse[b * a.Hq + h] * kLog2E);
  }
  a.weights[(size_t)bh * a.cap + j] += w;
}

template <typename T, int D>
cudaError_t run(const StepArgs& a, cudaStream_t s) {
  float* lse = a.weights ? static_cast<float*>(a.ws) : nullptr;
  step_rows_kernel<T, D><<<(unsigned)(((long long)a.B * a.Hq + 3) / 4), 128, 0, s>>>(a, lse);
  if (a.weights && a.cap)
    step_weights_kernel<T, D><<<dim3((a.cap + 127) / 128, a.B * a.Hkv), 128, 0, s>>>(a, lse);
  return cudaGetLastError();
}
}  // namespace

size_t step_ws(const StepArgs& a, bool with_weights) {
  return with_weights ? ((size_t)a.B * a.Hq * 4 + 255) / 256 * 256 : 256;
}

cudaError_t launch_step(const StepArgs& a, cudaStream_t s) {
  if (a.dtype == IG_BF16) return a.d == 128 ? run<__nv_bfloat16, 128>(a, s) : run<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? run<__half, 128>(a, s) : run<__half, 64>(a, s);
}

}  // namespace ig
