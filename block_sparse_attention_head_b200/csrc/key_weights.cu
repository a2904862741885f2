// The attention mass of packed prompts' keys (instagen_key_weights):
//   weights[hk, j] += sum over the heads h of hk's group and the queries i that
//   see j of 2^(c q_i.k_j - lse_i log2(e)),  c = softmax_scale log2(e).
//
// The product is taken the other way round than for attention: S^T = K Q^T
// puts the keys on the TMEM lanes, so a key's mass is summed by the one thread
// that owns its lane, without atomics or shuffles, and nothing is written back
// to TMEM.  A CTA owns 256 keys (two chains of M = 128 rows of K, on chip once)
// and walks the tiles of 256 queries of one head that see them, head after
// head; each Q tile is the B operand (N = 256) of both chains, which keeps the
// shared-memory reads of an MMA below its tensor time (at N = 128 they are
// equal).  lse comes through shared memory, converted once per tile to its
// negative in log2 units (-inf for rows that see nothing or do not exist).
//
// Bound: the exponentials, 2 * 2048 MUFU cycles per tile and CTA against 2 *
// 1024 tensor cycles (d = 128); three eighths of those of unmasked tiles run
// on the FMA pipe instead (degree 5: the sums keep fp32's digits).  Sixteen
// warps share them, four per scheduler, two to a TMEM lane.
//
// Few keys, many queries: nsplit CTAs share a key pair, each over its part of
// the tiles, and add_parts_kernel adds their sums in order.
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kKwThreads = 640;  // 16 warps of sums, 2 MMA, loader, lse
constexpr int kKwTile = 256;   // keys per CTA, queries per tile
constexpr int kKwLseRing = 4;

template <int D>
struct KwSmem {
  static constexpr int kKeyBytes = D * 256;   // 128 keys
  static constexpr int kQBytes = D * 512;     // 256 queries
  static constexpr int kK = 0;
  static constexpr int kQ = kK + 2 * kKeyBytes;
  static constexpr int kLse = kQ + 2 * kQBytes;
  static constexpr int kXch = kLse + kKwLseRing * kKwTile * 4;  // the second half rows' sums
  static constexpr int kBars = kXch + 256 * 4;
  static constexpr int kMisc = kBars + 24 * 8;
  static constexpr int kBytes = kMisc + 64;
  static constexpr size_t bytes() { return 1024 + kBytes; }
};
static_assert(KwSmem<128>::bytes() <= 232448, "shared memory budget");
}  // namespace

struct KwArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  const float* lse;
  float* weights;
  float* parts;  // [nsplit, Hkv, Tk] when nsplit > 1
  int nseq, Hkv, G, Tq, Tk, causal, nsplit, npair;
  float scale_log2;
};

template <typename T, int D>
__global__ void __launch_bounds__(kKwThreads, 1)
    key_weights_kernel(KwArgs a, const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k) {
  using L = KwSmem<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* nlse = reinterpret_cast<float*>(smem + L::kLse);
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_full = bars + 0;
  uint64_t* q_full = bars + 1;   // [2] stages
  uint64_t* q_empty = bars + 3;  // [2]
  uint64_t* s_full = bars + 5;   // [2] chains
  uint64_t* s_empty = bars + 7;  // [2]
  uint64_t* l_full = bars + 9;   // [kKwLseRing]
  uint64_t* l_empty = bars + 13; // [kKwLseRing]
  uint64_t* fin = bars + 17;     // [2] chains
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 0);
  volatile int* abort_flag = misc + 1;
  int* work = misc + 2;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % a.Hkv;
  const int z = blockIdx.x / a.Hkv % a.nsplit;
  const int t_glob = blockIdx.x / a.Hkv / a.nsplit;

  if (warp == 0) {
    const SeqPair p = find_pair(a.cu_k, a.cu_q, a.nseq, 1, t_glob);
    if (lane == 0) *reinterpret_cast<SeqPair*>(work) = p;
  }
  __syncthreads();
  const SeqPair sp = *reinterpret_cast<const SeqPair*>(work);
  const int local = sp.local;
  if (sp.seq < 0 || local < 0) return;
  int q0s = sp.other_lo, q1s = sp.other_hi, k0s = sp.lo, k1s = sp.hi;
  clamp_rows(q0s, q1s, a.Tq);
  clamp_rows(k0s, k1s, a.Tk);
  const int nq = q1s - q0s, nk = k1s - k0s;
  const int kb = local * kKwTile;  // first key of the pair
  if (kb >= nk) return;
  const int off = nk - nq;         // causal: query i sees key j iff i >= j - off
  const int i0 = a.causal ? max(0, kb - off) / kKwTile : 0;
  const int ntile = max(0, (nq + kKwTile - 1) / kKwTile - i0);
  const int visits = ntile * a.G;
  const int v0 = (int)((long long)visits * z / a.nsplit), v1 = (int)((long long)visits * (z + 1) / a.nsplit);
  const int nv = v1 - v0;

  if (tid == 0) {
    mbar_init(k_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 256);
      mbar_init(&fin[i], 1);
    }
    for (int i = 0; i < kKwLseRing; ++i) {
      mbar_init(&l_full[i], 32);
      mbar_init(&l_empty[i], 512);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t k_s = smem_u32(smem + L::kK), q_s = smem_u32(smem + L::kQ);

  float acc = 0.f;
  if (warp == 18) {
    // ================================================================ loader
    if (lane == 0 && nv > 0) {
      mbar_arrive_expect_tx(k_full, 2 * L::kKeyBytes);
      for (int t = 0; t < 2; ++t)
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(k_s + t * L::kKeyBytes + c * 16384, &tmap_k, 64 * c, k0s + kb + 128 * t, hk, k_full);
    }
    int issued = 0;
    for (int i = 0; i < nv; ++i) {
      const int st = i & 1, v = v0 + i;
      if (i >= 2 && !mbar_wait_warp(&q_empty[st], ((i >> 1) - 1) & 1, abort_flag)) break;
      if (lane == 0) {
        const int row = q0s + (i0 + v % ntile) * kKwTile, head = hk * a.G + v / ntile;
        mbar_arrive_expect_tx(&q_full[st], L::kQBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(q_s + st * L::kQBytes + c * 32768, &tmap_q, 64 * c, row, head, &q_full[st]);
      }
      issued = i + 1;
    }
    if (nv > 0) mbar_wait_drain(k_full, 0);  // no copy in flight is left behind
    for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait_drain(&q_full[i & 1], (i >> 1) & 1);
  } else if (warp == 19) {
    // =================================================================== lse
    for (int i = 0; i < nv; ++i) {
      const int st = i % kKwLseRing, v = v0 + i;
      const int tok = (i0 + v % ntile) * kKwTile, head = hk * a.G + v / ntile;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = tok + lane + 32 * e;
        const float y = row < nq ? __ldg(a.lse + (size_t)head * a.Tq + q0s + row) : -INFINITY;
        x[e] = y == -INFINITY ? -INFINITY : -y * kLog2E;
      }
      if (i >= kKwLseRing && !mbar_wait_warp(&l_empty[st], (i / kKwLseRing - 1) & 1, abort_flag)) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) nlse[st * kKwTile + lane + 32 * e] = x[e];
      mbar_arrive(&l_full[st]);
    }
  } else if (warp >= 16) {
    // =================================================================== MMA
    const int t = warp - 16;
    const uint32_t idesc = umma_idesc_f16kind(128, 256, false, false, kHalf);
    const uint64_t kd = umma_desc_sw128(k_s + t * L::kKeyBytes, 16, 1024);
    const uint64_t qd0 = umma_desc_sw128(q_s, 16, 1024);
    const uint32_t s_t = tmem + 256 * t;
    bool ok = nv == 0 || mbar_wait_warp(k_full, 0, abort_flag);
    for (int i = 0; i < nv && ok; ++i) {
      ok = mbar_wait_warp(&q_full[i & 1], (i >> 1) & 1, abort_flag) &&
           (i == 0 || mbar_wait_warp(&s_empty[t], (i - 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint64_t qd = qd0 + (uint64_t)(i & 1) * (uint64_t)(L::kQBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_bf16_ss(s_t, kd + (uint64_t)((k >> 2) * 1024 + (k & 3) * 2), qd + (uint64_t)((k >> 2) * 2048 + (k & 3) * 2),
                       idesc, k > 0 ? 1u : 0u);
        umma_commit(&s_full[t]);
        umma_commit(&q_empty[i & 1]);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(&fin[t]);
    __syncwarp();
    mbar_wait_drain(&fin[t], 0);
  } else {
    // ================================================================ sums
    // four warpgroups: chain t's lanes, columns [128 half, 128 half + 128)
    const int t = warp >> 3, half = (warp >> 2) & 1, qd = warp & 3;
    const int key = kb + 128 * t + 32 * qd + lane;
    const uint32_t s_col = tmem + (uint32_t)((32 * qd) << 16) + 256 * t + 128 * half;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    for (int i = 0; i < nv; ++i) {
      const int tok = (i0 + (v0 + i) % ntile) * kKwTile + 128 * half;
      // columns [lo, hi) of the half tile: queries that exist and see this key
      const int lo = a.causal ? key - off - tok : 0, hi = nq - tok;
      const bool whole = hi >= 128 && (!a.causal || kb + 128 * t + 127 - off <= tok);
      const float* nl = nlse + (i % kKwLseRing) * kKwTile + 128 * half;
      if (!mbar_wait_warp(&l_full[i % kKwLseRing], (i / kKwLseRing) & 1, abort_flag)) break;
      if (!mbar_wait_warp(&s_full[t], i & 1, abort_flag)) break;
      tc_fence_after();
      uint64_t sum[2] = {0ull, 0ull};
      auto chunk = [&](int c, float (&v)[32], auto masked) {
        constexpr bool kMask = decltype(masked)::value;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 n4 = *reinterpret_cast<const float4*>(nl + 32 * c + e);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint64_t y = fma2(pack2(v[e + 2 * h], v[e + 2 * h + 1]), scale2, h ? pack2(n4.z, n4.w) : pack2(n4.x, n4.y));
            if (!kMask && ((e >> 1) + h) % 8 < 3) {
              y = ex2_poly2<5>(y);
            } else {
              float p0, p1;
              unpack2(y, p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              if constexpr (kMask) {
                const int col = 32 * c + e + 2 * h;
                p0 = col >= lo && col < hi ? p0 : 0.f;
                p1 = col + 1 >= lo && col + 1 < hi ? p1 : 0.f;
              }
              y = pack2(p0, p1);
            }
            sum[h] = add2(sum[h], y);
          }
        }
      };
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float x[32];
        tmem_ld32(s_col + 32 * c, x);
        tmem_wait_ld();
        pin_regs32(x);
        if (c == 3) {
          tc_fence_before();
          mbar_arrive(&s_empty[t]);
        }
        if (whole)
          chunk(c, x, std::false_type());
        else
          chunk(c, x, std::true_type());
      }
      mbar_arrive(&l_empty[i % kKwLseRing]);
      float s0, s1;
      unpack2(add2(sum[0], sum[1]), s0, s1);
      acc += s0 + s1;
    }
    if (half == 1) xch[128 * t + 32 * qd + lane] = acc;
  }
  tc_fence_before();
  __syncthreads();
  if (warp < 16 && !((warp >> 2) & 1)) {
    const int lane_t = 128 * (warp >> 3) + 32 * (warp & 3) + lane;
    if (kb + lane_t < nk) {
      const size_t at = (size_t)hk * a.Tk + k0s + kb + lane_t;
      acc += xch[lane_t];
      if (a.nsplit > 1)
        a.parts[(size_t)z * a.Hkv * a.Tk + at] = acc;
      else
        a.weights[at] += acc;
    }
  }
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// weights += the parts' sums, for the keys of sequences (one thread each).
__global__ void __launch_bounds__(256) add_parts_kernel(KwArgs a) {
  const size_t n = (size_t)a.Hkv * a.Tk, at = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= n) return;
  const int j = (int)(at % a.Tk);
  int lo = 0, hi = a.nseq;  // the last sequence that starts at or before j
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_k[mid] <= j)
      lo = mid;
    else
      hi = mid;
  }
  if (j < a.cu_k[lo] || j >= a.cu_k[lo + 1]) return;
  float s = 0.f;
  for (int z = 0; z < a.nsplit; ++z) s += a.parts[z * n + at];
  a.weights[at] += s;
}

// CTAs per key pair: where the pairs leave SMs idle, the visits are split so
// that about every SM has a CTA, in parts of at least 2.
static int key_weight_splits(const PromptArgs& a) {
  const long long ctas = row_pairs(a.Tk, 1, a.nseq) * a.Hkv;
  const long long visits = (long long)a.G * ((a.Tq / a.nseq + kKwTile - 1) / kKwTile);
  long long n = ctas >= kSms ? 1 : kSms / ctas;
  if (n > visits / 2) n = visits / 2;
  return n < 1 ? 1 : (int)n;
}

size_t key_weights_ws(const PromptArgs& a) {
  const int n = key_weight_splits(a);
  return n == 1 ? 256 : (size_t)n * a.Hkv * a.Tk * 4 + 256;
}

template <typename T, int D>
static cudaError_t run_key_weights(const KwArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, cudaStream_t s) {
  const size_t sm = KwSmem<D>::bytes();
  cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  key_weights_kernel<T, D><<<(unsigned)((long long)a.npair * a.Hkv * a.nsplit), kKwThreads, sm, s>>>(a, tq, tk);
  return cudaGetLastError();
}

cudaError_t launch_key_weights(const PromptArgs& p, cudaStream_t s) {
  KwArgs a{};
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.lse = p.lse;
  a.weights = p.weights;
  a.nseq = p.nseq;
  a.Hkv = p.Hkv;
  a.G = p.G;
  a.Tq = p.Tq;
  a.Tk = p.Tk;
  a.causal = p.causal;
  a.scale_log2 = p.scale_log2;
  a.nsplit = key_weight_splits(p);
  a.npair = (int)row_pairs(p.Tk, 1, p.nseq);
  a.parts = static_cast<float*>(p.ws);
  CUtensorMap tq, tk;
  cudaError_t e = make_tmap_rows(&tq, p.Q, p.dtype, p.d, p.Tq, p.Hq, p.q_tok, p.q_head, 256);
  if (e == cudaSuccess) e = make_tmap_rows(&tk, p.K, p.dtype, p.d, p.Tk, p.Hkv, p.k_tok, p.k_head, 128);
  if (e != cudaSuccess) return e;
  if (p.dtype == IG_BF16)
    e = p.d == 128 ? run_key_weights<__nv_bfloat16, 128>(a, tq, tk, s) : run_key_weights<__nv_bfloat16, 64>(a, tq, tk, s);
  else
    e = p.d == 128 ? run_key_weights<__half, 128>(a, tq, tk, s) : run_key_weights<__half, 64>(a, tq, tk, s);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  add_parts_kernel<<<(unsigned)(((size_t)a.Hkv * a.Tk + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ig
