// The attention mass of packed prompts' keys (instagen_key_weights):
//   weights[hk, j] += sum over the heads h of hk's group and the queries i that
//   see j of 2^(c q_i.k_j - lse_i log2(e)),  c = softmax_scale log2(e).
//
// The product is taken the other way round than for attention: S^T = K Q^T
// puts the keys on the TMEM lanes, so a key's mass is summed by the threads
// that own its lane, without atomics or shuffles, and nothing is written back
// to TMEM.  A CTA owns 256 keys (two chains of M = 128) and walks the tiles of
// 128 queries of one head that see them, head after head.  The keys are the A
// operand and stay in TMEM (written once), so that a product only reads the
// query tile from shared memory, 64 bytes a cycle; with both operands there it
// reads 128, all there is.  Three score tiles of 128 columns rotate between
// the MMA warp and four warpgroups, each of which takes every fourth one:
// product, load and exponentials of three visits overlap.  (Two warpgroups with
// twice the registers and a whole row in them took 9% longer for 2048 queries on
// 16384 keys, 32/4 heads, d = 128, which take 370 us now.)  lse comes through
// shared memory, converted once per tile to its negative in log2 units (-inf
// for rows that see nothing or do not exist).
//
// Bound: the exponentials, 2 * 1024 MUFU cycles per query tile and CTA against
// 2 * 512 tensor cycles (d = 128); three eighths of those of unmasked tiles run
// on the FMA pipe instead (degree 5: the sums keep fp32's digits).
//
// Few keys, many queries: nsplit CTAs share a key pair, each over its part of
// the tiles, and add_parts_kernel adds their sums in order.
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kKwThreads = 640;  // 16 warps of sums, MMA, spare, loader, lse
constexpr int kKwKeys = 256;     // keys per CTA
constexpr int kKwTile = 128;     // queries per tile
constexpr int kKwStages = 6;     // query tiles on chip
constexpr int kKwLse = 8;        // lse tiles
// TMEM columns: the keys [0, 64) and [64, 128), three score tiles from 128 on
constexpr uint32_t kKwS = 128;

template <int D>
struct KwSmem {
  static constexpr int kQBytes = D * 256;  // 128 queries
  static constexpr int kQ = 0;
  static constexpr int kLse = kQ + kKwStages * kQBytes;
  static constexpr int kXch = kLse + kKwLse * kKwTile * 4;  // sums of the second warpgroup of a chain
  static constexpr int kBars = kXch + 256 * 4;
  static constexpr int kMisc = kBars + 48 * 8;
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
  const void* K;
  int64_t k_tok, k_head;
};

template <typename T, int D>
__global__ void __launch_bounds__(kKwThreads, 1)
    key_weights_kernel(KwArgs a, const __grid_constant__ CUtensorMap tmap_q) {
  using L = KwSmem<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* nlse = reinterpret_cast<float*>(smem + L::kLse);
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_ready = bars + 0;
  uint64_t* fin = bars + 1;
  uint64_t* s_full = bars + 2;                     // [4] warpgroups: the visit's scores are there
  uint64_t* s_empty = bars + 6;                    // [3] score tiles
  uint64_t* q_full = bars + 9;                     // [kKwStages]
  uint64_t* q_empty = q_full + kKwStages;          // [kKwStages]
  uint64_t* l_full = q_empty + kKwStages;          // [kKwLse]
  uint64_t* l_empty = l_full + kKwLse;             // [kKwLse]
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 0);
  volatile int* abort_flag = misc + 1;
  int* work = misc + 2;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.x % a.Hkv;
  const int z = blockIdx.x / a.Hkv % a.nsplit;
  const int t_glob = blockIdx.x / a.Hkv / a.nsplit;

  launch_dependents();
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
  const int kb = local * kKwKeys;  // first key of the pair
  if (kb >= nk) return;
  const int off = nk - nq;         // causal: query i sees key j iff i >= j - off
  const int i0 = a.causal ? max(0, kb - off) / kKwTile : 0;
  const int ntile = max(0, (nq + kKwTile - 1) / kKwTile - i0);
  const int visits = ntile * a.G;
  const int v0 = (int)((long long)visits * z / a.nsplit), v1 = (int)((long long)visits * (z + 1) / a.nsplit);
  const int nv = v1 - v0;

  if (tid == 0) {
    mbar_init(k_ready, 256);
    mbar_init(fin, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&s_empty[i], 128);
    for (int i = 0; i < kKwStages; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kKwLse; ++i) {
      mbar_init(&l_full[i], 32);
      mbar_init(&l_empty[i], 256);
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
  const uint32_t q_s = smem_u32(smem + L::kQ);

  float acc = 0.f;
  if (warp >= 16) setmaxnreg_dec<64>();  // 4 * 32 * 64 + 16 * 32 * 104 = 640 * 96
  if (warp == 18) {
    // ================================================================ loader
    int issued = 0;
    for (int i = 0; i < nv; ++i) {
      const int st = i % kKwStages, v = v0 + i;
      if (i >= kKwStages && !mbar_wait_warp(&q_empty[st], (i / kKwStages - 1) & 1, abort_flag)) break;
      if (lane == 0) {
        const int row = q0s + (i0 + v % ntile) * kKwTile, head = hk * a.G + v / ntile;
        mbar_arrive_expect_tx(&q_full[st], L::kQBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(q_s + st * L::kQBytes + c * 16384, &tmap_q, 64 * c, row, head, &q_full[st]);
      }
      issued = i + 1;
    }
    for (int i = max(0, issued - kKwStages); i < issued; ++i)  // no copy in flight is left behind
      mbar_wait_drain(&q_full[i % kKwStages], (i / kKwStages) & 1);
  } else if (warp == 19) {
    // =================================================================== lse
    for (int i = 0; i < nv; ++i) {
      const int st = i % kKwLse, v = v0 + i;
      const int tok = (i0 + v % ntile) * kKwTile, head = hk * a.G + v / ntile;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = tok + lane + 32 * e;
        const float y = row < nq ? __ldg(a.lse + (size_t)head * a.Tq + q0s + row) : -INFINITY;
        x[e] = y == -INFINITY ? -INFINITY : -y * kLog2E;
      }
      if (i >= kKwLse && !mbar_wait_warp(&l_empty[st], (i / kKwLse - 1) & 1, abort_flag)) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) nlse[st * kKwTile + lane + 32 * e] = x[e];
      mbar_arrive(&l_full[st]);
    }
  } else if (warp >= 16) {
    // =================================================================== MMA
    // visit v: tile v / 2 of the list, chain v % 2, score tile v % 3
    if (warp == 16) {
      const uint32_t idesc = umma_idesc_f16kind(128, 128, false, false, kHalf);
      const uint64_t qd0 = umma_desc_sw128(q_s, 16, 1024);
      bool ok = nv == 0 || mbar_wait_warp(k_ready, 0, abort_flag);
      for (int v = 0; v < 2 * nv && ok; ++v) {
        const int i = v >> 1, st = i % kKwStages, b = v % 3;
        if (!(v & 1)) ok = mbar_wait_warp(&q_full[st], (i / kKwStages) & 1, abort_flag);
        if (ok && v >= 3) ok = mbar_wait_warp(&s_empty[b], (v / 3 - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t qd = qd0 + (uint64_t)st * (uint64_t)(L::kQBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_f16_ts(tmem + kKwS + 128 * b, tmem + 64 * (v & 1) + 8 * k, qd + (uint64_t)((k >> 2) * 1024 + (k & 3) * 2),
                        idesc, k > 0 ? 1u : 0u);
          umma_commit(&s_full[v & 3]);
          if (v & 1) umma_commit(&q_empty[st]);
        }
        __syncwarp();
      }
      if (elect_one()) umma_commit(fin);
      __syncwarp();
      mbar_wait_drain(fin, 0);
    }
  } else {
    // ================================================================ sums
    // warpgroup w: visits v = w mod 4, so chain w % 2 and every other tile
    setmaxnreg_inc<104>();
    const int t = (warp >> 2) & 1, half = warp >> 3, qd = warp & 3;
    const int key = kb + 128 * t + 32 * qd + lane;
    const uint32_t lane_off = (uint32_t)((32 * qd) << 16);
    if (half == 0) {  // the chain's keys into TMEM: two elements to a column
      const int row = min(k0s + key, a.Tk - 1);  // (rows past the end are garbage that is not summed)
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.K) + row * a.k_tok + hk * a.k_head);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __ldg(src + 8 * c + e);
        tmem_st32(tmem + lane_off + 64 * t + 32 * c, reinterpret_cast<const float*>(v));
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(k_ready);
    }
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    for (int i = half; i < nv; i += 2) {
      const int v = 2 * i + t, b = v % 3;
      const int tok = (i0 + (v0 + i) % ntile) * kKwTile;
      // columns [lo, hi) of the tile: queries that exist and see this key
      const int lo = a.causal ? key - off - tok : 0, hi = nq - tok;
      const bool whole = hi >= 128 && (!a.causal || kb + 128 * t + 127 - off <= tok);
      const float* nl = nlse + (i % kKwLse) * kKwTile;
      const uint32_t s_col = tmem + lane_off + kKwS + 128 * b;
      if (!mbar_wait_warp(&l_full[i % kKwLse], (i / kKwLse) & 1, abort_flag)) break;
      if (!mbar_wait_warp(&s_full[v & 3], (i >> 1) & 1, abort_flag)) break;
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
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x0[32], x1[32];
        tmem_ld32(s_col + 64 * c, x0);
        tmem_ld32(s_col + 64 * c + 32, x1);
        tmem_wait_ld();
        pin_regs32(x0);
        pin_regs32(x1);
        if (c == 1) {
          tc_fence_before();
          mbar_arrive(&s_empty[b]);
        }
        if (whole) {
          chunk(2 * c, x0, std::false_type());
          chunk(2 * c + 1, x1, std::false_type());
        } else {
          chunk(2 * c, x0, std::true_type());
          chunk(2 * c + 1, x1, std::true_type());
        }
      }
      mbar_arrive(&l_empty[i % kKwLse]);
      float s0, s1;
      unpack2(add2(sum[0], sum[1]), s0, s1);
      acc += s0 + s1;
    }
    if (half == 1) xch[128 * t + 32 * qd + lane] = acc;
  }
  tc_fence_before();
  __syncthreads();
  if (warp < 8) {
    const int lane_t = 128 * (warp >> 2) + 32 * (warp & 3) + lane;
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
  // this grid's end is that of key_weights_kernel's, even where no key is joined
  if (blockIdx.x == 0) wait_prior_grids();
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
  wait_prior_grids();  // key_weights_kernel's parts
  float s = 0.f;
  for (int z = 0; z < a.nsplit; ++z) s += a.parts[z * n + at];
  a.weights[at] += s;
}

// CTAs per key pair: the visits of a pair are split where that shortens the
// whole: waves of CTAs times a CTA's visits and the 6 that its start and end
// cost, in parts of at least 4 visits.  Measured (bf16, d = 128, causal) with 0, 3,
// 6, 12 for them: 2048 queries on 16384 keys, 32/4 heads 664, 373, 369, 370 us; 6 x
// up to 1000, 32/8 76, 57, 49, 56; 4 x up to 512, 32/8 26.5, 26.5, 32.8, 32.8; 8192,
// 8/8 277, 102, 102, 102; 256 on 8192, 64 on 30000, 16 x 300 and 3 x 100: the same.
static int key_weight_splits(const PromptArgs& a) {
  const long long ctas = row_pairs(a.Tk, 1, a.nseq) * a.Hkv;
  const long long visits = (long long)a.G * ((a.Tq / a.nseq + kKwTile - 1) / kKwTile);
  long long best = 1, cost = -1;
  for (long long n = 1; n <= 64 && (n == 1 || visits / n >= 4); ++n) {
    const long long c = (ctas * n + kSms - 1) / kSms * ((visits + n - 1) / n + 6);
    if (cost < 0 || c < cost) {
      best = n;
      cost = c;
    }
  }
  return (int)best;
}

size_t key_weights_ws(const PromptArgs& a) {
  const int n = key_weight_splits(a);
  return n == 1 ? 256 : (size_t)n * a.Hkv * a.Tk * 4 + 256;
}

template <typename T, int D>
static cudaError_t run_key_weights(const KwArgs& a, const CUtensorMap& tq, cudaStream_t s) {
  const size_t sm = KwSmem<D>::bytes();
  cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  key_weights_kernel<T, D><<<(unsigned)((long long)a.npair * a.Hkv * a.nsplit), kKwThreads, sm, s>>>(a, tq);
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
  a.K = p.K;
  a.k_tok = p.k_tok;
  a.k_head = p.k_head;
  CUtensorMap tq;
  cudaError_t e = make_tmap_rows(&tq, p.Q, p.dtype, p.d, p.Tq, p.Hq, p.q_tok, p.q_head);
  if (e != cudaSuccess) return e;
  if (p.dtype == IG_BF16)
    e = p.d == 128 ? run_key_weights<__nv_bfloat16, 128>(a, tq, s) : run_key_weights<__nv_bfloat16, 64>(a, tq, s);
  else
    e = p.d == 128 ? run_key_weights<__half, 128>(a, tq, s) : run_key_weights<__half, 64>(a, tq, s);
  if (e != cudaSuccess || a.nsplit == 1) return e;
  return launch_after(add_parts_kernel, dim3((unsigned)(((size_t)a.Hkv * a.Tk + 255) / 256)), 256, 0, true, s, a);
}

}  // namespace ig
