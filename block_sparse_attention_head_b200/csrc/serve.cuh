// Internal launch interface of the language-model entry points
// (instagen_prompt_attention, instagen_key_weights, instagen_prefix_attention,
// instagen_evict): arguments and shared device helpers.
#pragma once
#include "instagen.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace ig {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2E = 1.4426950408889634f;

struct PromptArgs {
  const void* Q;
  const void* K;
  const void* V;
  const int32_t* cu_q;  // [nseq + 1]
  const int32_t* cu_k;
  int nseq, Hq, Hkv, G, d, Tq, Tk, dtype, causal;
  float scale_log2;  // softmax_scale * log2(e)
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;
  void* O;
  float* lse;      // [Hq, Tq]: out of the attention, in of the key weights; may be null for the former
  float* weights;  // [Hkv, Tk] (key weights)
  void* ws;
};
size_t prompt_attention_ws(const PromptArgs& a);
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t s);
size_t key_weights_ws(const PromptArgs& a);
cudaError_t launch_key_weights(const PromptArgs& a, cudaStream_t s);

struct StepArgs {
  const void* Q;
  const void* Kp;
  const void* Vp;
  const void* Kc;
  const void* Vc;
  const int32_t* lens;
  int B, Hq, Hkv, G, d, P, cap, dtype;
  float scale_log2;
  int64_t q_seq, prefix_head;
  void* O;
  float* lse;      // [B, Hq] or null
  float* weights;  // [B, Hkv, cap] or null
  void* ws;
};
size_t step_ws(const StepArgs& a, bool with_weights);
cudaError_t launch_step(const StepArgs& a, cudaStream_t s);

struct EvictArgs {
  const void* K;
  const void* V;
  const float* weights;
  const int32_t* pos;
  const int32_t* lens;
  int B, Hkv, d, cap, budget, recent, cap_out;
  bool in_place;
  void* K_out;
  void* V_out;
  float* weights_out;
  int32_t* pos_out;
  int32_t* lens_out;
  void* ws;
};
size_t evict_ws(int B, int Hkv, int budget);
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

// Launches kernel(args...); overlap: it may start before the kernel in front of
// it in the stream has ended (see launch_dependents).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool overlap, cudaStream_t s,
                         const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------ device helpers
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}

// Rows [lo, hi) of a packed sequence, clamped into [0, T].
__device__ __forceinline__ void clamp_rows(int& lo, int& hi, int T) {
  if (lo < 0 || hi < lo || hi > T) {
    raise_error(kErrIndex);
    lo = min(max(lo, 0), T);
    hi = min(max(hi, lo), T);
  }
}

// Live slots of a cache, clamped into [0, cap].
__device__ __forceinline__ int live_slots(const int32_t* lens, int b, int cap) {
  int n = lens[b];
  if (n < 0 || n > cap) {
    raise_error(kErrIndex);
    n = min(max(n, 0), cap);
  }
  return n;
}

// Overlapped launches (programmatic dependent launch).  A kernel launched with
// launch_after may start once every CTA of the kernel before it has called
// launch_dependents or ended; wait_prior_grids returns when that kernel is
// complete and its writes are visible (at once after an ordinary launch).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_prior_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace ig
