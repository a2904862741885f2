// C ABI of the language-model entry points (declared in include/instagen.h):
// argument checks and argument blocks; the launches are in prompt.cu, step.cu
// and evict.cu.
#include "serve.cuh"

#include <cmath>

namespace {

int check_heads(int Hq, int Hkv, int d, int dtype) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv) return IG_ERR_INVALID_ARG;
  if (dtype != IG_BF16 && dtype != IG_F16) return IG_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return IG_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hq / Hkv > 1024) return IG_ERR_UNSUPPORTED;
  return IG_OK;
}

bool good_scale(float c) { return std::isfinite(c) && c > 0.f && std::isfinite(c * ig::kLog2E); }

// A 3-D tensor's strides in elements: positive, whole 16-byte steps, at least
// a row apart (dimensions of one entry may have any), within TMA's 2^40 bytes.
bool good_strides(int64_t tok, int64_t head, int T, int H, int d) {
  const int64_t most = int64_t(1) << 38;
  if (T > 1 && (tok < d || tok % 8 || tok > most)) return false;
  if (H > 1 && (head < d || head % 8 || head > most)) return false;
  return true;
}

int prompt_args(const instagen_prompt_params* p, ig::PromptArgs* a) {
  if (!p) return IG_ERR_INVALID_ARG;
  if (p->nseq < 1 || p->Tq < 0 || p->Tk < 0 || (p->causal != 0 && p->causal != 1)) return IG_ERR_INVALID_ARG;
  int rc = check_heads(p->Hq, p->Hkv, p->d, p->dtype);
  if (rc) return rc;
  if (!good_scale(p->softmax_scale)) return IG_ERR_INVALID_ARG;
  const long long most = 2147483647LL - 1024;
  if (p->nseq > (1 << 20) || (long long)p->nseq * p->Hkv > (1 << 26) || (long long)p->Tq * p->Hq > most || (long long)p->Tk * p->Hkv > most)
    return IG_ERR_UNSUPPORTED;
  if (!good_strides(p->q_tok, p->q_head, p->Tq, p->Hq, p->d) || !good_strides(p->k_tok, p->k_head, p->Tk, p->Hkv, p->d))
    return IG_ERR_INVALID_ARG;
  *a = ig::PromptArgs{};
  a->nseq = p->nseq;
  a->Hq = p->Hq;
  a->Hkv = p->Hkv;
  a->G = p->Hq / p->Hkv;
  a->d = p->d;
  a->Tq = p->Tq;
  a->Tk = p->Tk;
  a->dtype = p->dtype;
  a->causal = p->causal;
  a->scale_log2 = p->softmax_scale * ig::kLog2E;
  // a stride that is not used gets the value of a dense tensor
  auto put = [&](int64_t& tok, int64_t& head, int64_t t, int64_t h, int T, int H) {
    tok = T > 1 ? t : (int64_t)p->d * H;
    head = H > 1 ? h : p->d;
  };
  put(a->q_tok, a->q_head, p->q_tok, p->q_head, p->Tq, p->Hq);
  put(a->k_tok, a->k_head, p->k_tok, p->k_head, p->Tk, p->Hkv);
  put(a->v_tok, a->v_head, p->v_tok, p->v_head, p->Tk, p->Hkv);
  put(a->o_tok, a->o_head, p->o_tok, p->o_head, p->Tq, p->Hq);
  return IG_OK;
}

// fp32 buffers are read and written element by element
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// (need = 256: the call uses none)
bool good_ws(const void* ws, size_t have, size_t need) {
  if (need == 256 && !ws) return true;
  return ws && have >= need && !(reinterpret_cast<uintptr_t>(ws) & 255u);
}

int step_args(const instagen_cache_params* p, ig::StepArgs* a) {
  if (!p) return IG_ERR_INVALID_ARG;
  if (p->B < 1 || p->P < 0 || p->cap < 0) return IG_ERR_INVALID_ARG;
  int rc = check_heads(p->Hq, p->Hkv, p->d, p->dtype);
  if (rc) return rc;
  const long long most = 2147483647LL - 1024;
  if ((long long)p->B * p->Hkv > 65535 || (long long)p->B * p->Hq > most || (long long)p->B * p->Hkv * p->cap > most ||
      (long long)p->P * p->Hkv > most)
    return IG_ERR_UNSUPPORTED;
  *a = ig::StepArgs{};
  a->B = p->B;
  a->Hq = p->Hq;
  a->Hkv = p->Hkv;
  a->G = p->Hq / p->Hkv;
  a->d = p->d;
  a->P = p->P;
  a->cap = p->cap;
  a->dtype = p->dtype;
  a->q_seq = p->B > 1 ? p->q_seq : (int64_t)p->Hq * p->d;
  a->prefix_head = p->Hkv > 1 ? p->prefix_head : (int64_t)p->P * p->d;
  return IG_OK;
}

int step_attention_args(const instagen_cache_params* p, ig::StepArgs* a) {
  const int rc = step_args(p, a);
  if (rc) return rc;
  if (!good_scale(p->softmax_scale)) return IG_ERR_INVALID_ARG;
  if (a->q_seq < (int64_t)p->Hq * p->d || a->q_seq % 8 || a->q_seq > (int64_t(1) << 38)) return IG_ERR_INVALID_ARG;
  if (p->P > 0 && (a->prefix_head < (int64_t)p->P * p->d || a->prefix_head % 8 || a->prefix_head > (int64_t(1) << 38)))
    return IG_ERR_INVALID_ARG;
  a->scale_log2 = p->softmax_scale * ig::kLog2E;
  return IG_OK;
}

}  // namespace

extern "C" {

size_t instagen_prompt_attention_workspace_size(const instagen_prompt_params* p) {
  ig::PromptArgs a;
  return prompt_args(p, &a) ? 0 : ig::prompt_attention_ws(a);
}

int instagen_prompt_attention(const void* Q, const void* K, const void* V, const int32_t* cu_q, const int32_t* cu_k,
                              const instagen_prompt_params* p, void* O, float* lse, void* ws, size_t ws_bytes,
                              void* stream) {
  ig::PromptArgs a;
  const int rc = prompt_args(p, &a);
  if (rc) return rc;
  if (!good_strides(p->v_tok, p->v_head, p->Tk, p->Hkv, p->d) || !good_strides(p->o_tok, p->o_head, p->Tq, p->Hq, p->d))
    return IG_ERR_INVALID_ARG;
  if (p->Tq == 0) return IG_OK;
  if (!Q || !O || !cu_q || !cu_k || (p->Tk > 0 && (!K || !V))) return IG_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned4(lse)) return IG_ERR_INVALID_ARG;
  if (!good_ws(ws, ws_bytes, ig::prompt_attention_ws(a))) return IG_ERR_WORKSPACE;
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.O = O;
  a.lse = lse;
  a.ws = ws;
  return cuda_status(ig::launch_prompt_attention(a, static_cast<cudaStream_t>(stream)));
}

size_t instagen_key_weights_workspace_size(const instagen_prompt_params* p) {
  ig::PromptArgs a;
  return prompt_args(p, &a) ? 0 : ig::key_weights_ws(a);
}

int instagen_key_weights(const void* Q, const void* K, const float* lse, const int32_t* cu_q, const int32_t* cu_k,
                         const instagen_prompt_params* p, float* weights, void* ws, size_t ws_bytes, void* stream) {
  ig::PromptArgs a;
  const int rc = prompt_args(p, &a);
  if (rc) return rc;
  if (p->Tq == 0 || p->Tk == 0) return IG_OK;
  if (!Q || !K || !lse || !cu_q || !cu_k || !weights) return IG_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned4(lse) || !aligned4(weights)) return IG_ERR_INVALID_ARG;
  if (!good_ws(ws, ws_bytes, ig::key_weights_ws(a))) return IG_ERR_WORKSPACE;
  a.Q = Q;
  a.K = K;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.lse = const_cast<float*>(lse);
  a.weights = weights;
  a.ws = ws;
  return cuda_status(ig::launch_key_weights(a, static_cast<cudaStream_t>(stream)));
}

size_t instagen_prefix_attention_workspace_size(const instagen_cache_params* p, int32_t with_weights) {
  ig::StepArgs a;
  return step_attention_args(p, &a) ? 0 : ig::step_ws(a, with_weights != 0);
}

int instagen_prefix_attention(const void* Q, const void* Kp, const void* Vp, const void* Kc, const void* Vc,
                              const int32_t* lens, const instagen_cache_params* p, void* O, float* lse,
                              float* weights, void* ws, size_t ws_bytes, void* stream) {
  ig::StepArgs a;
  const int rc = step_attention_args(p, &a);
  if (rc) return rc;
  if (!Q || !O || !lens || (p->P > 0 && (!Kp || !Vp)) || (p->cap > 0 && (!Kc || !Vc))) return IG_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(Kp) || !aligned16(Vp) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O) ||
      !aligned4(lse) || !aligned4(weights))
    return IG_ERR_INVALID_ARG;
  if (!good_ws(ws, ws_bytes, ig::step_ws(a, weights != nullptr))) return IG_ERR_WORKSPACE;
  a.Q = Q;
  a.Kp = Kp;
  a.Vp = Vp;
  a.Kc = Kc;
  a.Vc = Vc;
  a.lens = lens;
  a.O = O;
  a.lse = lse;
  a.weights = weights;
  a.ws = ws;
  return cuda_status(ig::launch_step(a, static_cast<cudaStream_t>(stream)));
}

size_t instagen_evict_workspace_size(const instagen_cache_params* p, int32_t budget) {
  ig::StepArgs a;
  if (step_args(p, &a) || budget < 1) return 0;
  const size_t n = ig::evict_ws(a.B, a.Hkv, budget);
  return n <= 256 ? 512 : n;  // (never the 256 of a call without scratch)
}

int instagen_evict(const void* K, const void* V, const float* weights, const int32_t* pos, const int32_t* lens,
                   const instagen_cache_params* p, int32_t budget, int32_t recent, void* K_out, void* V_out,
                   float* weights_out, int32_t* pos_out, int32_t* lens_out, int32_t cap_out, void* ws,
                   size_t ws_bytes, void* stream) {
  ig::StepArgs c;
  const int rc = step_args(p, &c);
  if (rc) return rc;
  if (budget < 1 || recent < 0 || budget > cap_out) return IG_ERR_INVALID_ARG;
  if ((long long)c.B * c.Hkv * cap_out > 2147483647LL - 1024) return IG_ERR_UNSUPPORTED;
  if ((c.cap > 0 && (!K || !V || !weights || !pos)) || !lens || !K_out || !V_out || !weights_out || !pos_out ||
      !lens_out)
    return IG_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned16(K_out) || !aligned16(V_out)) return IG_ERR_INVALID_ARG;
  const int same = (K == K_out) + (V == V_out) + (weights == weights_out) + (pos == pos_out) + (lens == lens_out);
  if ((same != 0 && same != 5) || (same == 5 && cap_out != c.cap)) return IG_ERR_INVALID_ARG;
  if (!ws || !good_ws(ws, ws_bytes, instagen_evict_workspace_size(p, budget))) return IG_ERR_WORKSPACE;
  ig::EvictArgs a;
  a.K = K;
  a.V = V;
  a.weights = weights;
  a.pos = pos;
  a.lens = lens;
  a.B = c.B;
  a.Hkv = c.Hkv;
  a.d = c.d;
  a.cap = c.cap;
  a.budget = budget;
  a.recent = recent;
  a.cap_out = cap_out;
  a.in_place = same == 5;
  a.K_out = K_out;
  a.V_out = V_out;
  a.weights_out = weights_out;
  a.pos_out = pos_out;
  a.lens_out = lens_out;
  a.ws = ws;
  return cuda_status(ig::launch_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
