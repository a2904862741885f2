// Dense attention on the tensor cores, for packed prompts and for a prefix
// that a batch shares (instagen_prompt_attention, instagen_prefix_attention).
//
// A key/value head serves the G query heads of its group, so the query rows
// of a sequence are numbered r = token * G + head of the group, and a CTA
// takes 256 consecutive rows of one (sequence, key/value head) in two tiles of
// 128 over the same key tiles: every K and V tile brought on chip serves all
// the heads of the group.  Per key tile j and row tile t:
//   S_t = Q_t K_j^T     tcgen05 (M=128, N=128), fp32 in TMEM
//   P_t = 2^(c S_t - m_t), rounded to the tensors' type, into S_t's columns
//   O_t += P_t V_j      tcgen05 with A (P_t) read from TMEM
// with c = softmax_scale log2(e) and m_t the running maximum, raised only when
// it grows by more than 8 (P <= 256), which keeps rescaling O rare.  For fp16,
// whose steps are 2^-24 from 2^-14 down, m_t is held 7 lower (P <= 2^15): a weight
// of 2^-21 of the row's largest still has all its digits, a smaller one is off by
// at most 2^-32 of it (without: 2^-14 and 2^-25, which l would not share).  Each chain
// has a softmax warpgroup (one thread per row) and an MMA warp; K and V have a
// loader warp each.  The chains take turns on the tensor pipe, so that one's
// exponentials run under the other's products: left to themselves they fall
// into step, and a key tile takes 4180 cycles instead of 3120.  A CTA with one
// row tile gives chain 0 the even and chain 1 the odd key tiles and merges the
// two partial softmaxes at the end.
//
// Bound: 4 * 512 tensor cycles per key tile and CTA (d = 128) against 2 * 1024
// of exponentials on the MUFU, a quarter of which (in unmasked tiles) run on
// the FMA pipe instead.  16384 tokens, 16/4 heads, d = 128: 0.90 ms in a single
// run (1.23 PFLOP/s, tensor pipe 63%), 0.97-1.0 back to back, where the card
// is at its power limit.  Short sequences: one
// wave of 148 CTAs of 256 rows takes 14.9 us on one key tile (launch, ends,
// query rows, first product; output, exit), 28.9 on 8 and 44.4 on 16, that is
// 1.8 to 1.9 us per key tile.
//
// Few rows, many keys: nsplit CTAs share a row tile pair, each over its part
// of the key tiles, and write normalised partial outputs with their log-sum-
// exp, which combine_kernel joins.
//
// Masks: a row sees a prefix of its sequence's keys (causal or not), so a tile
// is full, cut, or skipped.  Keys behind the sequence's end are never seen; V
// rows there may hold anything, so the last tile's are zeroed on chip (0 * NaN
// would reach every row).
#include "serve.cuh"

#include <type_traits>

namespace ig {

namespace {
constexpr int kTcThreads = 384;
constexpr int kTcRows = 256;        // query rows per CTA
constexpr float kTcThreshold = 8.f;
constexpr float kTcHalfShift = 7.f;  // fp16: m below the row's maximum
// TMEM columns: S_0 [0,128), S_1 [128,256), O_0 [256,..), O_1 [384,..)
constexpr uint32_t kTcO = 256;

template <int D>
struct TcSmem {
  static constexpr int kTileBytes = D * 256;  // 128 rows of D 16-bit values
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + 2 * kTileBytes;
  static constexpr int kXch = kV + 2 * kTileBytes;  // chain 1's row maxima and sums
  static constexpr int kBars = kXch + 2 * 128 * 4;
  static constexpr int kMisc = kBars + 24 * 8;
  static constexpr int kBytes = kMisc + 64;
  static constexpr size_t bytes() { return 1024 + kBytes; }
};
static_assert(TcSmem<128>::bytes() <= 232448, "shared memory budget");

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Two floats in one 64-bit register: packed fp32 arithmetic of sm_100.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x of two values on the FMA pipe, x < 128: x = n + f with n the nearest
// integer (adding 1.5 * 2^23 leaves n in the low mantissa bits) and 2^f, |f| <=
// 1/2, by a polynomial with the smallest relative error (Remez exchange,
// coefficients rounded to fp32).
//   Degree 5 (1.6e-7): times 2^n, which has the bits 0 for n = -127, so below
//   2^-126.5 gives 0, and NaN stays NaN.
//   Degree 4 (2.9e-6, 2.6e-6 without the constant held at 1): n is added to the
//   exponent's bits.  x is at least -127, where f >= 0 and the constant's bits
//   end at 0 or above: below 2^-126 gives less, -inf gives 0.  A NaN does not
//   stay one (as a product it would: the 16384-token prompt takes 2% longer);
//   the caller's row maximum keeps it.
template <int kDegree>
__device__ __forceinline__ uint64_t ex2_poly2(uint64_t x2) {
  constexpr float c0 = kDegree == 5 ? 1.0000001192092896f : 1.f;
  constexpr float c1 = kDegree == 5 ? 0.6931469440460205f : 0.6931241750717163f;
  constexpr float c2 = kDegree == 5 ? 0.24022120237350464f : 0.24024099111557007f;
  constexpr float c3 = kDegree == 5 ? 0.05550713092088699f : 0.055906426161527634f;
  constexpr float c4 = kDegree == 5 ? 0.009675540961325169f : 0.009582852944731712f;
  constexpr float c5 = 0.0013276472454890609f;
  static_assert(kDegree == 4 || kDegree == 5, "degree");
  float a, b;
  unpack2(x2, a, b);
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(a));  // -127
  asm("max.NaN.f32 %0, %0, 0fC2FE0000;" : "+f"(b));
  const uint64_t x = pack2(a, b);
  const uint64_t n = add2(x, pack2(12582912.f, 12582912.f));
  const uint64_t f = fma2(add2(n, pack2(-12582912.f, -12582912.f)), pack2(-1.f, -1.f), x);
  uint64_t p = pack2(c4, c4);
  if constexpr (kDegree == 5) p = fma2(pack2(c5, c5), f, p);
  p = fma2(p, f, pack2(c3, c3));
  p = fma2(p, f, pack2(c2, c2));
  p = fma2(p, f, pack2(c1, c1));
  p = fma2(p, f, pack2(c0, c0));
  float n0, n1;
  unpack2(n, n0, n1);
  const uint32_t e0 = __float_as_uint(n0) << 23, e1 = __float_as_uint(n1) << 23;
  if constexpr (kDegree == 5) return mul2(p, pack2(__uint_as_float(e0 + 0x3f800000u), __uint_as_float(e1 + 0x3f800000u)));
  float p0, p1;
  unpack2(p, p0, p1);
  return pack2(__uint_as_float(__float_as_uint(p0) + e0), __uint_as_float(__float_as_uint(p1) + e1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) return pack_f16x2(lo, hi);
  return pack_bf16x2(lo, hi);
}
}  // namespace

struct TcArgs {
  const void* Q;
  void* O;
  float* lse;       // [Hq, Tq] natural log, or null
  float* o_part;    // [nsplit, Tq, Hq, D] (nsplit > 1 or partial)
  float* lse_part;  // [nsplit, Tq, Hq] log2
  const int32_t* cu_q;  // null: one sequence of Tq and Tk rows
  const int32_t* cu_k;
  int nseq, Hq, Hkv, G, Tq, Tk, causal, nsplit, ntile;
  bool partial;    // write o_part / lse_part
  int short_last;  // > 0: pair numbers from here on are the sequences' last pairs of one row tile
  float scale_log2;
  int64_t q_tok, q_head, o_tok, o_head;
};

// Row tile pair -> sequence.  Sequence s owns the pair numbers [f(s), f(s+1)),
// f(s) = floor(cu_q[s] G / 256) + s: at least ceil(n_q G / 256) of them (the
// others are idle), and f needs no sum over the sequences before, so a warp
// finds s by a 32-way search.
// The sequence of pair number t (-1: none), t's place in it and its rows; the
// ends are loaded along with the keys of the search, in one round for up to 32
// sequences.
struct SeqPair {
  int seq, local, lo, hi, other_lo, other_hi;
};
__device__ __forceinline__ SeqPair find_pair(const int32_t* cu, const int32_t* cu_other, int nseq, int G, int t) {
  const int lane = threadIdx.x & 31;
  SeqPair p{-1, 0, 0, 0, 0, 0};
  int lo = 0, hi = nseq;
  bool found = false;
  while (hi - lo > 1 || !found) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    int c0 = 0, c1 = 0, o0 = 0, o1 = 0;
    if (at < hi) {
      c0 = cu[at];
      c1 = cu[at + 1];
      o0 = cu_other[at];
      o1 = cu_other[at + 1];
    }
    const int first = (int)(((long long)c0 * G) >> 8) + at;
    const unsigned hit = __ballot_sync(0xffffffffu, at < hi && first <= t);
    if (!hit) return p;
    const int src = 31 - __clz(hit);
    p.local = t - __shfl_sync(0xffffffffu, first, src);
    p.lo = __shfl_sync(0xffffffffu, c0, src);
    p.hi = __shfl_sync(0xffffffffu, c1, src);
    p.other_lo = __shfl_sync(0xffffffffu, o0, src);
    p.other_hi = __shfl_sync(0xffffffffu, o1, src);
    lo += src * step;
    hi = min(hi, lo + step);
    found = true;
  }
  p.seq = lo;
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_kernel(TcArgs a, const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
  using L = TcSmem<D>;
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr float kShift = kHalf ? kTcHalfShift : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* xch = reinterpret_cast<float*>(smem + L::kXch);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* q_full = bars + 0;   // [2] row tiles
  uint64_t* k_full = bars + 2;   // [2] stages
  uint64_t* k_empty = bars + 4;  // [2]
  uint64_t* v_full = bars + 6;   // [2]
  uint64_t* v_empty = bars + 8;  // [2]
  uint64_t* s_full = bars + 10;  // [2] chains
  uint64_t* p_head = bars + 12;  // [2] chains: the tile's first 96 keys of P
  uint64_t* p_tail = bars + 14;  // [2] chains: the last 32
  uint64_t* o_done = bars + 16;  // [2] chains
  uint64_t* fin = bars + 18;     // [2] chains
  uint64_t* v_fixed = bars + 20;
  uint64_t* turn = bars + 21;    // [2] chains: may issue its next block of MMAs
  int* misc = reinterpret_cast<int*>(smem + L::kMisc);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 0);
  volatile int* abort_flag = misc + 1;
  int* work = misc + 2;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  if (tid == 320) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  const int hk = blockIdx.x % a.Hkv;
  const int t_glob = (blockIdx.x / a.Hkv) % a.ntile;
  const int z = blockIdx.x / a.Hkv / a.ntile;

  // ---- which rows
  int q0s = 0, q1s = a.Tq, k0s = 0, k1s = a.Tk, local = t_glob;
  if (a.cu_q) {
    if (a.short_last > 0 && t_glob >= a.short_last) {
      if (tid == 0) {
        const int s = t_glob - a.short_last;
        *reinterpret_cast<SeqPair*>(work) = {s, 0, a.cu_q[s], a.cu_q[s + 1], a.cu_k[s], a.cu_k[s + 1]};
      }
    } else if (warp == 0) {
      const SeqPair p = find_pair(a.cu_q, a.cu_k, a.nseq, a.G, t_glob);
      if (lane == 0) *reinterpret_cast<SeqPair*>(work) = p;
    }
    __syncthreads();
    const SeqPair p = *reinterpret_cast<const SeqPair*>(work);
    if (p.seq < 0) return;
    local = p.local;
    q0s = p.lo;
    q1s = p.hi;
    k0s = p.other_lo;
    k1s = p.other_hi;
    clamp_rows(q0s, q1s, a.Tq);
    clamp_rows(k0s, k1s, a.Tk);
  }
  const int nq = q1s - q0s, nk = k1s - k0s, G = a.G;
  const int R = nq * G;
  // the last rows of a sequence see the most keys: they go first
  const int pair = (R + kTcRows - 1) / kTcRows - 1 - local;
  if (pair < 0 || local < 0) return;
  // a sequence's last pair of one row tile goes behind all others, if asked for
  if (a.short_last > 0 && (t_glob >= a.short_last) != (local == 0 && R - pair * kTcRows <= 128)) return;
  const int r0 = pair * kTcRows;
  const int rows0 = min(128, R - r0), rows1 = max(0, min(128, R - r0 - 128));
  const bool one = rows1 == 0;  // one row tile: chains take the even / odd key tiles
  auto seen = [&](int r) { return a.causal ? min(nk, max(0, r / G + 1 + nk - nq)) : nk; };  // keys that row r sees
  // key tiles [j0, j1) of this CTA; chain t's end
  const int ntk = (seen(r0 + rows0 + rows1 - 1) + 127) / 128;
  const int j0 = (int)((long long)ntk * z / a.nsplit), j1 = (int)((long long)ntk * (z + 1) / a.nsplit);
  const int end0 = one ? j1 : max(j0, min(j1, (seen(r0 + rows0 - 1) + 127) / 128));
  const int nj = j1 - j0;
  const int cut = nk & 127 ? nk >> 7 : -1;  // the key tile that the sequence ends in

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&k_empty[i], one ? 1 : 2);
      mbar_init(&v_empty[i], one ? 1 : 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_head[i], 128);
      mbar_init(&p_tail[i], 128);
      mbar_init(&o_done[i], 1);
      mbar_init(&fin[i], 1);
      mbar_init(&turn[i], 1);
    }
    mbar_init(v_fixed, 32);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t q_s = smem_u32(smem + L::kQ);
  const uint32_t k_s = smem_u32(smem + L::kK);
  const uint32_t v_s = smem_u32(smem + L::kV);
  constexpr int kChunks = D / 8;             // 16-byte chunks of a row
  constexpr int kRowsPerStep = 32 / kChunks; // rows a warp moves at once

  if (warp >= 8) {
    setmaxnreg_dec<72>();
    if (warp >= 10) {
      // ============================================================ loaders
      // warp 10 brings K, warp 11 V: a stage of K is free long before the V of
      // the same tile, and with one row tile the next K is needed soon after
      const bool is_v = warp == 11;
      const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const uint32_t base = is_v ? v_s : k_s;
      int issued = 0;
      for (int i = 0; i < nj; ++i) {
        const int s = i & 1, row = k0s + (j0 + i) * 128;
        if (i >= 2 && !mbar_wait_warp(&empty[s], ((i >> 1) - 1) & 1, abort_flag)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], L::kTileBytes);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(base + s * L::kTileBytes + c * 16384, map, 64 * c, row, hk, &full[s]);
        }
        issued = i + 1;
        if (is_v && j0 + i == cut) {  // zero the V rows behind the sequence's end
          mbar_wait_drain(&full[s], (i >> 1) & 1);
          for (int c = 0; c < D / 64; ++c)
            for (int b = (nk & 127) * 8 + lane; b < 1024; b += 32)
              st_shared_v4(base + s * L::kTileBytes + c * 16384 + b * 16, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          mbar_arrive(v_fixed);
        }
      }
      for (int i = max(0, issued - 2); i < issued; ++i)  // no copy in flight is left behind
        mbar_wait_drain(&full[i & 1], (i >> 1) & 1);
    } else {
      // ================================================================ MMA
      // warp 8 + t issues chain t: S_t(first), then PV_t(previous), S_t(next),
      // ... PV_t(last); the warp waits in step, one elected lane issues
      const int t = warp - 8;
      const uint32_t idesc_qk = umma_idesc_f16kind(128, 128, false, false, kHalf);
      const uint32_t idesc_pv = umma_idesc_f16kind(128, D, false, true, kHalf);
      constexpr uint64_t kTileStep = (uint64_t)(L::kTileBytes >> 4);
      const uint64_t qd = umma_desc_sw128(q_s, 16, 1024) + (uint64_t)(one ? 0 : t) * kTileStep;
      const uint64_t kd0 = umma_desc_sw128(k_s, 16, 1024);
      const uint64_t vd0 = umma_desc_sw128(v_s, 16384, 1024);
      const uint32_t s_t = tmem + 128 * t, o_t = tmem + kTcO + 128 * t;
      const int step = one ? 2 : 1, i0 = one ? t : 0;
      const int iend = (!one && t == 0 ? end0 : j1) - j0;
      bool ok = true;
      // PV_t of tile i (the chain's ph-th), in two parts as P arrives
      auto issue_pv = [&](int i, int ph) -> bool {
        const uint64_t vd = vd0 + (uint64_t)(i & 1) * kTileStep;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 6; ++k)
            umma_f16_ts(o_t, s_t + 8 * k, vd + (uint64_t)(k * 128), idesc_pv, (ph > 0 || k > 0) ? 1u : 0u);
        }
        __syncwarp();
        if (!mbar_wait_warp(&p_tail[t], ph & 1, abort_flag)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 6; k < 8; ++k) umma_f16_ts(o_t, s_t + 8 * k, vd + (uint64_t)(k * 128), idesc_pv, 1u);
          umma_commit(&v_empty[i & 1]);
        }
        __syncwarp();
        return true;
      };
      auto issue_s = [&](int i) {
        const uint64_t kd = kd0 + (uint64_t)(i & 1) * kTileStep;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)((k >> 2) * 1024 + (k & 3) * 2);
            umma_bf16_ss(s_t, qd + off, kd + off, idesc_qk, k > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[t]);
          umma_commit(&k_empty[i & 1]);
        }
        __syncwarp();
      };
      // block b: PV of the chain's tile b - 1, S of its tile b.  The chains
      // take turns block by block: left to themselves they fall into step,
      // both in their softmax and then both on the tensor pipe.
      const int n = max(0, (iend - i0 + step - 1) / step);
      const int n_other = t == 1 ? max(0, ((one ? nj : end0 - j0) + step - 1) / step) : max(0, one ? nj / 2 : nj);
      if (n > 0) {
        ok = mbar_wait_warp(&q_full[one ? 0 : t], 0, abort_flag);
        fence_proxy_async_smem();
      }
      for (int b = 0; b <= n && ok && n > 0; ++b) {
        const int i = i0 + b * step, prev = i - step;
        if (b < n) ok = mbar_wait_warp(&k_full[i & 1], (i >> 1) & 1, abort_flag);
        if (ok && b > 0)
          ok = mbar_wait_warp(&v_full[prev & 1], (prev >> 1) & 1, abort_flag) &&
               (j0 + prev != cut || mbar_wait_warp(v_fixed, 0, abort_flag));
        if (ok && b < n) {
          const int pass = t == 0 ? b - 1 : b;  // the other chain's block that comes first
          if (pass >= 0 && pass < n_other) ok = mbar_wait_warp(&turn[t], pass & 1, abort_flag);
        }
        // last, so that the waits above are over by the time P is there
        if (ok && b > 0) ok = mbar_wait_warp(&p_head[t], (b - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (b > 0) ok = issue_pv(prev, b - 1);
        if (ok && b < n) {
          issue_s(i);
          if (lane == 0) mbar_arrive(&turn[t ^ 1]);
        }
      }
      if (elect_one()) {
        if (ok) umma_commit(&o_done[t]);
        umma_commit(&fin[t]);
      }
      __syncwarp();
      // key tiles that only chain 1 reads: hand the stages on for it
      if (!one && t == 0) {
        for (int i = max(0, iend); i < nj && ok; ++i) {
          ok = mbar_wait_warp(&k_full[i & 1], (i >> 1) & 1, abort_flag) &&
               mbar_wait_warp(&v_full[i & 1], (i >> 1) & 1, abort_flag);
          if (ok && lane == 0) {
            mbar_arrive(&k_empty[i & 1]);
            mbar_arrive(&v_empty[i & 1]);
          }
        }
      }
      mbar_wait_drain(&fin[t], 0);
    }
  } else {
    // ============================================================== softmax
    setmaxnreg_inc<216>();
    const int t = warp >> 2, qd = warp & 3;
    const int r = 32 * qd + lane;  // row of the tile == TMEM lane
    const int nrows = t == 0 ? rows0 : rows1;
    const int rt = r0 + 128 * t;   // first row of the tile
    const uint32_t lane_off = (uint32_t)((32 * qd) << 16);
    const uint32_t s_col = tmem + lane_off + 128 * t, o_col = tmem + lane_off + kTcO + 128 * t;
    // this warp's 32 query rows, whole rows at a time: lane -> row lane /
    // kChunks of a step, 16-byte chunk lane % kChunks
    const int ch = lane % kChunks;
    if (nrows > 0) {
      int row = 32 * qd + lane / kChunks;
      const int tok0 = rt / G, tok1 = (rt + row) / G;
      int head = rt + row - tok1 * G;
      const T* Q = static_cast<const T*>(a.Q) + (int64_t)q0s * a.q_tok + (int64_t)(hk * G) * a.q_head + 8 * ch;
      const T* first = Q + (int64_t)tok0 * a.q_tok + (int64_t)(rt - tok0 * G) * a.q_head;  // a row that exists
      const T* at = Q + (int64_t)tok1 * a.q_tok + (int64_t)head * a.q_head;
      const int64_t wrap = a.q_tok - (int64_t)G * a.q_head;
      uint4 v[32 / kRowsPerStep];  // every load on its way before the first is stored
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerStep; ++i) {
        v[i] = __ldg(reinterpret_cast<const uint4*>(row < nrows ? at : first));
        row += kRowsPerStep;
        head += kRowsPerStep;
        at += kRowsPerStep * a.q_head;
#pragma unroll
        for (int e = 0; e < kRowsPerStep; ++e) {  // at most one token further per row
          const bool over = head >= G;
          head -= over ? G : 0;
          at += over ? wrap : 0;
        }
      }
      row = 32 * qd + lane / kChunks;
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerStep; ++i, row += kRowsPerStep) {
        const bool there = row < nrows;
        st_shared_v4(q_s + t * L::kTileBytes + (ch >> 3) * 16384 + sw128_offset(row, ch & 7), there ? v[i].x : 0u,
                     there ? v[i].y : 0u, there ? v[i].z : 0u, there ? v[i].w : 0u);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&q_full[t]);
    const int see = one || t == 0 ? (r < rows0 ? seen(r0 + r) : 0) : (r < rows1 ? seen(rt + r) : 0);
    // tiles below `whole` need no mask in any row of the tile
    const int whole = (one ? seen(r0) : seen(min(rt, R - 1))) >> 7;
    float m = -INFINITY, l = 0.f;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    bool ok = true;
    const int step = one ? 2 : 1;
    const int jend = !one && t == 0 ? end0 : j1;
    int ph = 0;

    auto visit = [&](int j, auto masked) {
      constexpr bool kMask = decltype(masked)::value;
      float x4[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, x4[c]);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 4; ++c) pin_regs32(x4[c]);
      if constexpr (kMask) {
        const int lim = see - j * 128;
#pragma unroll
        for (int c = 0; c < 128; ++c) x4[c >> 5][c & 31] = c < lim ? x4[c >> 5][c & 31] : -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 2)
        mx[(c >> 1) & 3] = fmax3_nan(mx[(c >> 1) & 3], x4[c >> 5][c & 31], x4[c >> 5][(c & 31) + 1]);
      const float top = fmax3_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * a.scale_log2 - kShift;
      // the first key of a row always raises; NaN does, and l is NaN from there on
      const bool raise = !(top <= m + kTcThreshold);
      float alpha = 1.f;
      if (raise) {
        alpha = ex2_approx(m - top);
        m = top;
      }
      // O_t holds the chain's earlier products (the tensor pipe finished them
      // before S_t(j)); the next one waits for p_head
      if (ph > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(o_col + 32 * c, o);
          tmem_wait_ld();
          pin_regs32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tmem_st32(o_col + 32 * c, o);
        }
      }
      const float base = m == -INFINITY ? 0.f : -m;  // no key so far: 2^(-inf) = 0
      const uint64_t base2 = pack2(base, base);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          uint64_t y = fma2(pack2(x4[c4][e], x4[c4][e + 1]), scale2, base2);
          float p0, p1;
          if (!kMask && (e & 6) == 6) {
            y = ex2_poly2<4>(y);
            unpack2(y, p0, p1);
          } else {
            unpack2(y, p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            y = pack2(p0, p1);
          }
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
          p[e >> 1] = pack16<T>(p0, p1);
        }
        tmem_st16(s_col + 16 * c4, p);
        if (c4 == 2) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_head[t]);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_tail[t]);
      float s0, s1;
      unpack2(add2(sum[0], sum[1]), s0, s1);
      l = l * alpha + (s0 + s1);
    };

    for (int j = j0 + (one ? t : 0); j < jend; j += step, ++ph) {
      if (!mbar_wait_warp(&s_full[t], ph & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (j < whole)
        visit(j, std::false_type());
      else
        visit(j, std::true_type());
    }
    if (ok) ok = mbar_wait_warp(&o_done[t], 0, abort_flag);
    tc_fence_after();
    bool have = ph > 0;  // O_t was written
    float w0 = 1.f, w1 = 0.f;
    bool have1 = false;
    if (one) {
      // merge the two chains' partial softmaxes of the same rows
      if (t == 1) {
        xch[r] = m;
        xch[128 + r] = l;
      }
      named_bar_sync(1, 256);
      if (t == 0) {
        have1 = nj > 1;
        if (ok) ok = mbar_wait_warp(&o_done[1], 0, abort_flag);
        tc_fence_after();
        const float m1 = xch[r], l1 = xch[128 + r];
        const float mm = fmaxf(m, m1);
        w0 = m == -INFINITY ? 0.f : ex2_approx(m - mm);
        w1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
        l = l * w0 + l1 * w1;
        m = mm;
      }
    }
    if (ok && nrows > 0) {
      const int rr = rt + r;
      const int tok = q0s + rr / G, head = hk * G + rr % G;
      const bool valid = r < nrows;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (valid) {
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        if (a.partial)
          a.lse_part[((size_t)z * a.Tq + tok) * a.Hq + head] = lse2;
        else if (a.lse)
          a.lse[(size_t)head * a.Tq + tok] = lse2 * kLn2;
      }
      if (!a.partial || have) {  // an empty part's rows are not read
        // 128 bytes of every row at a time through this warp's rows of the
        // query tile (no MMA reads it any more), so that a store writes whole
        // lines: 32 fp32 columns of a part, 64 of O
        uint8_t* stage = smem + L::kQ + t * L::kTileBytes + 32 * qd * 128;
        const uint32_t stage_s = smem_u32(stage);
        const int64_t off = !valid      ? -1
                            : a.partial ? (int64_t)((((size_t)z * a.Tq + tok) * a.Hq + head) * D * 4)
                                        : (tok * a.o_tok + head * a.o_head) * 2;
        uint8_t* out = a.partial ? reinterpret_cast<uint8_t*>(a.o_part) : static_cast<uint8_t*>(a.O);
        const bool zero = !have || __any_sync(0xffffffffu, l == 0.f);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float o[2][32];
          if (have) {
            tmem_ld32(o_col + 64 * c, o[0]);
            tmem_ld32(o_col + 64 * c + 32, o[1]);
            tmem_wait_ld();
            pin_regs32(o[0]);
            pin_regs32(o[1]);
            if (have1) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float o1[32];
                tmem_ld32(o_col + 128 + 64 * c + 32 * h, o1);
                tmem_wait_ld();
                pin_regs32(o1);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[h][e] = o[h][e] * w0 + o1[e] * w1;
              }
            }
          }
          if (zero) {
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] = have && l != 0.f ? o[e >> 5][e & 31] : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] *= inv;
          auto copy_out = [&](int col) {  // col: bytes from the row's start
            __syncwarp();
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = *reinterpret_cast<const uint4*>(stage + sw128_offset(4 * i + lane / 8, lane & 7));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t to = __shfl_sync(0xffffffffu, off, 4 * i + lane / 8);
              if (to >= 0) *reinterpret_cast<uint4*>(out + to + col + 16 * (lane & 7)) = v[i];
            }
            __syncwarp();
          };
          if (a.partial) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                st_shared_v4(stage_s + sw128_offset(lane, e), __float_as_uint(o[h][4 * e]),
                             __float_as_uint(o[h][4 * e + 1]), __float_as_uint(o[h][4 * e + 2]),
                             __float_as_uint(o[h][4 * e + 3]));
              copy_out(256 * c + 128 * h);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              st_shared_v4(stage_s + sw128_offset(lane, e), pack16<T>(o[e >> 2][8 * (e & 3)], o[e >> 2][8 * (e & 3) + 1]),
                           pack16<T>(o[e >> 2][8 * (e & 3) + 2], o[e >> 2][8 * (e & 3) + 3]),
                           pack16<T>(o[e >> 2][8 * (e & 3) + 4], o[e >> 2][8 * (e & 3) + 5]),
                           pack16<T>(o[e >> 2][8 * (e & 3) + 6], o[e >> 2][8 * (e & 3) + 7]));
            copy_out(128 * c);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) wait_prior_grids();  // this grid's end is that of the one it overlaps, too
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial outputs of rows (token, head) over the splits: weights
// 2^(lse_z - max) / sum.  One warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(128) combine_kernel(TcArgs a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const size_t rows = (size_t)a.Tq * a.Hq;
  // this grid's end is that of attend_kernel's, even where no row is joined
  if (blockIdx.x == 0) wait_prior_grids();
  if (row >= (long long)rows) return;
  const int tok = (int)(row / a.Hq), head = (int)(row % a.Hq);
  if (a.cu_q) {  // rows of no sequence stay as they were
    int lo = 0, hi = a.nseq;
    bool found = false;
    while (hi - lo > 1 || !found) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const unsigned hit = __ballot_sync(0xffffffffu, at < hi && a.cu_q[at] <= tok);
      if (!hit) return;
      lo += (31 - __clz(hit)) * step;
      hi = min(hi, lo + step);
      found = true;
    }
    if (tok >= a.cu_q[lo + 1]) return;
  }
  wait_prior_grids();  // attend_kernel's parts
  float top = -INFINITY;
  for (int z = 0; z < a.nsplit; ++z) top = fmaxf(top, a.lse_part[z * rows + row]);
  float o[D / 32], sum = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
  for (int z = 0; z < a.nsplit; ++z) {
    const float x = a.lse_part[z * rows + row];
    if (x == -INFINITY) continue;
    const float w = exp2f(x - top);
    sum += w;
    const float* src = a.o_part + (z * rows + row) * D;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = fmaf(w, src[lane + 32 * e], o[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* dst = static_cast<T*>(a.O) + tok * a.o_tok + head * a.o_head;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) dst[lane + 32 * e] = from_f32<T>(o[e] * inv);
  if (a.lse && lane == 0) a.lse[(size_t)head * a.Tq + tok] = (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------- host
// [heads, rows, d] 16-bit tensor with strides (elements), boxes of box_rows
// rows x 64 columns in the UMMA 128-byte swizzle.
static cudaError_t make_tmap_rows(CUtensorMap* m, const void* base, int dtype, int d, int rows, int heads, int64_t tok,
                                  int64_t head, unsigned box_rows = 128) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorUnknown;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
  cuuint64_t strides[2] = {(cuuint64_t)tok * 2, (cuuint64_t)head * 2};
  cuuint32_t box[3] = {64, box_rows, 1}, estr[3] = {1, 1, 1};
  const CUresult r = fn(m, dtype == IG_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kSms = 148;

// Row tile pairs of packed sequences (an upper bound, see find_pair).
static long long row_pairs(int Tq, int G, int nseq) { return ((long long)Tq * G >> 8) + nseq; }
// and of one sequence of known length.
static long long row_pairs_one(int n, int G) { return ((long long)n * G + 255) >> 8; }

// CTAs per row tile pair: where the pairs leave SMs idle, the keys are split
// so that about every SM has a CTA, in parts of at least 4 key tiles.
// Measured (graph replays, bf16, d = 128), parts of at least 2, 4, 8, 16, 32
// tiles: 64 rows of 8/2 heads on 8192 keys 22.8, 21.3, 25.9, 38.1, 64.3 us; on
// 32768 keys 32.8, 32.9, 32.3, 41.4, 65.5; a step of 32 sequences, 32/8 heads,
// behind 4000 keys 26.2, 22.9, 28.7, 48.0, 48.0.
static int key_splits(long long ctas, long long keys) {
  if (ctas >= kSms) return 1;
  const long long by_keys = keys / 512;
  long long n = kSms / ctas;
  if (n > by_keys) n = by_keys;
  if (n > 64) n = 64;
  return n < 1 ? 1 : (int)n;
}

template <typename T, int D>
static cudaError_t run_attend(const TcArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s,
                              bool overlap = false) {
  const size_t sm = TcSmem<D>::bytes();
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_after(attend_kernel<T, D>, dim3((unsigned)((long long)a.ntile * a.Hkv * a.nsplit)), kTcThreads, sm,
                      overlap, s, a, tk, tv);
}

static cudaError_t dispatch_attend(const TcArgs& a, int dtype, int d, const CUtensorMap& tk, const CUtensorMap& tv,
                                   cudaStream_t s) {
  if (dtype == IG_BF16)
    return d == 128 ? run_attend<__nv_bfloat16, 128>(a, tk, tv, s) : run_attend<__nv_bfloat16, 64>(a, tk, tv, s);
  return d == 128 ? run_attend<__half, 128>(a, tk, tv, s) : run_attend<__half, 64>(a, tk, tv, s);
}

static int prompt_splits(const PromptArgs& a) {
  if (a.Tq == 0) return 1;  // nothing to join
  return key_splits(row_pairs(a.Tq, a.G, a.nseq) * a.Hkv, a.Tk / a.nseq);
}

size_t prompt_attention_ws(const PromptArgs& a) {
  const int n = prompt_splits(a);
  return n == 1 ? 256 : (size_t)n * a.Tq * a.Hq * (a.d + 1) * 4;
}

cudaError_t launch_prompt_attention(const PromptArgs& p, cudaStream_t s) {
  TcArgs a{};
  a.Q = p.Q;
  a.O = p.O;
  a.lse = p.lse;
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.nseq = p.nseq;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.G;
  a.Tq = p.Tq;
  a.Tk = p.Tk;
  a.causal = p.causal;
  a.scale_log2 = p.scale_log2;
  a.q_tok = p.q_tok;
  a.q_head = p.q_head;
  a.o_tok = p.o_tok;
  a.o_head = p.o_head;
  a.ntile = (int)row_pairs(p.Tq, p.G, p.nseq);
  a.nsplit = prompt_splits(p);
  // Long keys and few units: the sequences' last pairs, where they hold one row
  // tile (half the time), start last and fill the end.  4 chunks of 257 rows
  // on up to 8191 keys, 40 heads, bf16: 268 us against 274 to 281; 2 of 1100 on
  // up to 6000, 16 heads: 110.6 against 113.8; 4 of 300 on 4096, 4 of 385 on 8191
  // and 8 of 100 on 3000: the same.  Each costs an idle CTA of a microsecond, so
  // not with many short sequences.
  if (a.nsplit == 1 && p.nseq * p.Hkv <= 2 * kSms && p.Tk / p.nseq >= 2048) {
    a.short_last = a.ntile;
    a.ntile += p.nseq;
  }
  a.partial = a.nsplit > 1;
  a.o_part = static_cast<float*>(p.ws);
  a.lse_part = a.o_part + (size_t)a.nsplit * p.Tq * p.Hq * p.d;
  CUtensorMap tk, tv;
  // without any key rows no load is issued; the maps then only need an address
  cudaError_t e = make_tmap_rows(&tk, p.Tk ? p.K : p.Q, p.dtype, p.d, p.Tk ? p.Tk : 1, p.Hkv, p.k_tok, p.k_head);
  if (e == cudaSuccess)
    e = make_tmap_rows(&tv, p.Tk ? p.V : p.Q, p.dtype, p.d, p.Tk ? p.Tk : 1, p.Hkv, p.v_tok, p.v_head);
  if (e == cudaSuccess) e = dispatch_attend(a, p.dtype, p.d, tk, tv, s);
  if (e != cudaSuccess || !a.partial) return e;
  const dim3 grid((unsigned)(((long long)p.Tq * p.Hq + 3) / 4));
  if (p.dtype == IG_BF16)
    return p.d == 128 ? launch_after(combine_kernel<__nv_bfloat16, 128>, grid, 128, 0, true, s, a)
                      : launch_after(combine_kernel<__nv_bfloat16, 64>, grid, 128, 0, true, s, a);
  return p.d == 128 ? launch_after(combine_kernel<__half, 128>, grid, 128, 0, true, s, a)
                    : launch_after(combine_kernel<__half, 64>, grid, 128, 0, true, s, a);
}

}  // namespace ig
