// Attention of one new token per sequence over a prefix that the batch shares
// and the sequence's own cache (instagen_prefix_attention).
//
// Three kernels write and join partial softmaxes: every part leaves its
// normalised output rows and their log-sum-exp (log2), finish_kernel weighs
// them by 2^(lse - max) and normalises once.
//   prefix  The B * G query rows that read one key/value head form one matrix,
//           so the prefix is read once for the batch: attend_kernel (tensor
//           cores, see prompt.cu), its keys split over the SMs.
//   own     rows_kernel: the G rows of a sequence against its own keys.  Bound
//           by the cache's bytes (G / 2 multiply-adds per byte): a warp takes
//           16 keys of every 64-key tile with m16n8k16 products, whose score
//           registers are the next product's operand registers, so scores
//           never leave the registers; tiles stream through a TMA ring.  A
//           prefix with at most 16 rows, or a short one that is read again for
//           every 16 rows (kRowsPasses), goes the same way in the same launch.
//   finish  join, and add the own keys' weights 2^(score - lse) from the scores
//           that rows_kernel left (4 G bytes per key beside the 4 d it read).
// The launches overlap (neither of the two reads what the other writes), and
// finish_kernel's CTAs wait where they need the parts.  The prefix goes first
// where it leaves SMs for all of the caches' CTAs (32 sequences behind 4000
// keys, with weights: 29.7 us against 35.8); else the caches do, and the prefix's
// CTAs take the SMs as they come free (8 sequences with 3000 keys of their own
// behind 30000: 60 us against 73; 128 with 200 behind 32768: 108.6 against 111.6).
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kRowsThreads = 160;  // 4 warps of 16 keys, 1 loader
constexpr int kRowsKeys = 64;      // keys per tile
// Tiles of 64 keys x 16 rows, over all heads, up to which a prefix goes through
// rows_kernel.  Measured against attend_kernel, whole calls with caches of 50
// keys: 12.3 us against 15.4 (8 sequences, 32/8 heads, 64 keys: 16 tiles), 16.4
// against 17.5 (32 sequences, 256 keys: 256), 10.3 against 16.4 (16, 16/2 heads,
// d = 64, 1024 keys: 256), 20.6 against 20.5 (32, 32/8 heads, 1024 keys: 1024),
// 37 against 26.7 (4096 keys: 4096).
constexpr int kRowsPasses = 1024;
constexpr int kFinishKeys = 2048;  // keys that a CTA of the weights' part takes at a time

// kLong: 96 KB in flight and two CTAs per SM, the faster stream; else 64 KB and
// three CTAs, whose starts and ends hide one another, for short shares.
// Measured, d = 128: 8 caches of 65000 keys 228 us against 248, 128 caches of
// 200 keys 33 us against 28.
template <int D, bool kLong>
struct RowsSmem {
  static constexpr int kTileBytes = kRowsKeys * D * 2;
  static constexpr int kStages = (D == 128 ? 1 : 2) * (kLong ? 3 : 2);
  static constexpr int kRing = 0;                   // [stage][K, V]
  static constexpr int kMl = kRing + kStages * 2 * kTileBytes;  // [4 warps][16 rows] maxima, then sums
  static constexpr int kBars = kMl + 2 * 4 * 16 * 4;
  static constexpr int kMisc = kBars + 2 * kStages * 8;
  static constexpr size_t bytes() { return 1024 + kMisc + 16; }
  static_assert(4 * 16 * D * 4 <= kStages * 2 * kTileBytes, "the warps' outputs are joined in the ring");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
}  // namespace

struct RowsArgs {
  const void* Q;
  const int32_t* lens;
  int B, Hq, Hkv, G, P, cap;
  int nown;     // splits of a cache
  int npre;     // splits of the prefix in this kernel (0: attend_kernel has it)
  int nslot;    // partial results per row: the prefix's, then the cache's
  int own_slot; // slot of the cache's first split
  int own_rows; // ceil(G / 16)
  int pre_rows; // ceil(B G / 16)
  bool direct;  // the only part: write O and lse
  float scale_log2;
  int64_t q_seq;
  float* o_part;    // [nslot, B * Hq, D]
  float* lse_part;  // [nslot, B * Hq] log2
  float* score;     // [B, Hkv, G, cap] log2 units, or null
  void* O;
  float* lse;
  float* weights;
};

template <typename T, int D, bool kLong>
__global__ void __launch_bounds__(kRowsThreads, kLong ? 2 : 3)
    rows_kernel(RowsArgs a, const __grid_constant__ CUtensorMap tmap_kp, const __grid_constant__ CUtensorMap tmap_vp,
                const __grid_constant__ CUtensorMap tmap_kc, const __grid_constant__ CUtensorMap tmap_vc) {
  using L = RowsSmem<D, kLong>;
  // fp16: the largest weight is 2^15, so that small ones keep their digits (see prompt.cu)
  constexpr float kShift = std::is_same<T, __half>::value ? 15.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* ml = reinterpret_cast<float*>(smem + L::kMl);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* empty = full + L::kStages;
  volatile int* abort_flag = reinterpret_cast<int*>(smem + L::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  launch_dependents();
  // ---- which rows, which keys
  int idx = blockIdx.x, hk, b0, rows, row0, n, split, nsplit, slot, z;
  const bool pre = idx < a.npre * a.Hkv * a.pre_rows;
  if (pre) {
    hk = idx % a.Hkv;
    idx /= a.Hkv;
    row0 = idx % a.pre_rows * 16;
    split = idx / a.pre_rows;
    nsplit = a.npre;
    b0 = 0;
    rows = a.B * a.G;
    n = a.P;
    slot = split;
    z = hk;
  } else {
    idx -= a.npre * a.Hkv * a.pre_rows;
    hk = idx % a.Hkv;
    idx /= a.Hkv;
    b0 = idx % a.B;
    idx /= a.B;
    row0 = idx % a.own_rows * 16;
    split = idx / a.own_rows;
    nsplit = a.nown;
    rows = a.G;
    n = live_slots(a.lens, b0, a.cap);
    slot = a.own_slot + split;
    z = b0 * a.Hkv + hk;
  }
  const int ntile = (n + kRowsKeys - 1) / kRowsKeys;
  const int t0 = (int)((long long)ntile * split / nsplit), t1 = (int)((long long)ntile * (split + 1) / nsplit);
  const int nt = t1 - t0;

  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const uint32_t ring = smem_u32(smem + L::kRing);

  if (warp == 4) {
    // ================================================================ loader
    int issued = 0;
    for (int i = 0; i < nt; ++i) {
      const int st = i % L::kStages;
      if (i >= L::kStages && !mbar_wait_warp(&empty[st], (i / L::kStages - 1) & 1, abort_flag)) break;
      issued = i + 1;
      if (lane == 0) {
        const uint32_t dst = ring + st * 2 * L::kTileBytes;
        mbar_arrive_expect_tx(&full[st], 2 * L::kTileBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(dst + c * kRowsKeys * 128, pre ? &tmap_kp : &tmap_kc, 64 * c, (t0 + i) * kRowsKeys, z, &full[st]);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(dst + L::kTileBytes + c * kRowsKeys * 128, pre ? &tmap_vp : &tmap_vc, 64 * c,
                      (t0 + i) * kRowsKeys, z, &full[st]);
      }
    }
    for (int i = max(0, issued - L::kStages); i < issued; ++i)  // no copy in flight is left behind
      mbar_wait_drain(&full[i % L::kStages], (i / L::kStages) & 1);
    return;
  }

  // ------------------------------------------------- 16 rows x 16 keys a tile
  const int ra = row0 + (lane >> 2), rb = ra + 8;  // this lane's rows
  auto q_row = [&](int r) -> const T* {
    return static_cast<const T*>(a.Q) + (int64_t)(b0 + r / a.G) * a.q_seq + (int64_t)(hk * a.G + r % a.G) * D;
  };
  uint32_t q[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const int c = 16 * k + (lane & 3) * 2;
    q[k][0] = ra < rows ? *reinterpret_cast<const uint32_t*>(q_row(ra) + c) : 0u;
    q[k][1] = rb < rows ? *reinterpret_cast<const uint32_t*>(q_row(rb) + c) : 0u;
    q[k][2] = ra < rows ? *reinterpret_cast<const uint32_t*>(q_row(ra) + c + 8) : 0u;
    q[k][3] = rb < rows ? *reinterpret_cast<const uint32_t*>(q_row(rb) + c + 8) : 0u;
  }
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int key_k = 16 * warp + (lane >> 4) * 8 + (lane & 7), chunk_k = (lane >> 3) & 1;  // ldmatrix rows of K
  const int key_v = 16 * warp + ((lane >> 3) & 1) * 8 + (lane & 7), chunk_v = lane >> 4;  // and of V
  bool ok = true;
  for (int i = 0; i < nt; ++i) {
    const int st = i % L::kStages;
    if (!mbar_wait_warp(&full[st], (i / L::kStages) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const uint32_t ks = ring + st * 2 * L::kTileBytes, vs = ks + L::kTileBytes;
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b[4];
      const int ch = 2 * k + chunk_k;
      ldmatrix_x4(ks + (ch >> 3) * (kRowsKeys * 128) + sw128_offset(key_k, ch & 7), b);
      mma_16816<T>(s[0], q[k], b[0], b[1]);
      mma_16816<T>(s[1], q[k], b[2], b[3]);
    }
    const int key0 = (t0 + i) * kRowsKeys + 16 * warp;  // the warp's first key
    const int lim = n - key0;                           // keys that exist
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[h][e] = 8 * h + (lane & 3) * 2 + (e & 1) < lim ? s[h][e] * a.scale_log2 : -INFINITY;
    if (!pre && a.score) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e < 2 ? ra : rb;
        float* dst = a.score + ((size_t)z * a.G + r) * a.cap + key0 + (lane & 3) * 2 + (e & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (r < rows && 8 * h + (lane & 3) * 2 + (e & 1) < lim) dst[8 * h] = s[h][e];
      }
    }
    if (lim < 16) {  // V rows behind the end may hold anything: 0 * NaN would reach every row
      for (int x = lane; x < 16 * (D / 8); x += 32) {
        const int row = x / (D / 8), ch = x % (D / 8);
        if (row >= lim) st_shared_v4(vs + (ch >> 3) * (kRowsKeys * 128) + (16 * warp + row) * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    float alpha[2];
    bool moved = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // rows ra, rb
      float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[h], top - kShift);
      const float base = mn == -INFINITY ? 0.f : mn;  // no key so far
      alpha[h] = ex2_approx(m[h] - base);
      moved |= mn > m[h];
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[t][2 * h + e] = ex2_approx(s[t][2 * h + e] - base);
          sum += s[t][2 * h + e];
        }
      l[h] = l[h] * alpha[h] + sum;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] *= alpha[e >> 1];
    }
    const uint32_t p[4] = {pack16<T>(s[0][0], s[0][1]), pack16<T>(s[0][2], s[0][3]), pack16<T>(s[1][0], s[1][1]),
                           pack16<T>(s[1][2], s[1][3])};
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t b[4];
      const int ch = 2 * d + chunk_v;
      ldmatrix_x4_trans(vs + (ch >> 3) * (kRowsKeys * 128) + sw128_offset(key_v, ch & 7), b);
      mma_16816<T>(o[2 * d], p, b[0], b[1]);
      mma_16816<T>(o[2 * d + 1], p, b[2], b[3]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  // ---- join the four warps
  if (!ok && lane == 0) *abort_flag = 1;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      ml[warp * 16 + (lane >> 2) + 8 * h] = m[h];
      ml[64 + warp * 16 + (lane >> 2) + 8 * h] = l[h];
    }
  }
  named_bar_sync(1, 128);  // every warp is done with the ring
  float* ow = reinterpret_cast<float*>(smem + L::kRing);  // [4][16][D]
  {
    float w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      const float top = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r]));
      w[h] = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - top);
    }
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(ow + (warp * 16 + (lane >> 2) + 8 * h) * D + 8 * d + (lane & 3) * 2) =
            make_float2(o[d][2 * h] * w[h], o[d][2 * h + 1] * w[h]);
  }
  wait_prior_grids();  // this grid's end is that of the one it overlaps, too
  named_bar_sync(1, 128);
  if (*abort_flag) return;
  for (int x = tid; x < 16 * (D / 4); x += 128) {
    const int r = x / (D / 4), c = x % (D / 4) * 4;
    if (row0 + r >= rows) break;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[16 * w + r]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float mw = ml[16 * w + r], lw = ml[64 + 16 * w + r];
      sum += mw == -INFINITY ? lw : lw * ex2_approx(mw - top);  // (no maximum: 0, or NaN)
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(ow + (16 * w + r) * D + c);
      v.x += y.x;
      v.y += y.y;
      v.z += y.z;
      v.w += y.w;
    }
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
    const size_t row = (size_t)(b0 + (row0 + r) / a.G) * a.Hq + hk * a.G + (row0 + r) % a.G;
    if (a.direct) {
      *reinterpret_cast<uint2*>(static_cast<T*>(a.O) + row * D + c) =
          make_uint2(pack16<T>(v.x, v.y), pack16<T>(v.z, v.w));
      if (c == 0 && a.lse) a.lse[row] = lse2 * kLn2;
    } else {
      *reinterpret_cast<float4*>(a.o_part + ((size_t)slot * a.B * a.Hq + row) * D + c) = v;
      if (c == 0) a.lse_part[(size_t)slot * a.B * a.Hq + row] = lse2;
    }
  }
}

// blockIdx.y = 0 joins the parts of the G rows of one (sequence, key/value
// head); the others share the weights of its own keys, kFinishKeys at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256) finish_kernel(RowsArgs a) {
  extern __shared__ float lse2[];  // [G]
  const int bh = blockIdx.x, b = bh / a.Hkv, hk = bh % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t rows = (size_t)a.B * a.Hq, row0 = (size_t)b * a.Hq + hk * a.G;
  const bool join = blockIdx.y == 0;
  const int n = join ? 0 : live_slots(a.lens, b, a.cap);
  const int j0 = ((int)blockIdx.y - 1) * kFinishKeys, jstep = ((int)gridDim.y - 1) * kFinishKeys;
  if (!join && j0 >= n) return;
  wait_prior_grids();
  for (int g = warp; g < a.G; g += 8) {
    const float* lp = a.lse_part + row0 + g;
    const float x0 = lane < a.nslot ? lp[lane * rows] : -INFINITY;
    float top = x0, sum = 0.f;
    for (int i = lane + 32; i < a.nslot; i += 32) top = fmaxf(top, lp[i * rows]);
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    // (top does not keep a NaN, the sum does)
    auto part = [&](float x) { return x == -INFINITY ? 0.f : exp2f(x - top); };
    sum = part(x0);
    for (int i = lane + 32; i < a.nslot; i += 32) sum += part(lp[i * rows]);
    sum = warp_sum(sum);
    const float y = sum == 0.f ? -INFINITY : top + log2f(sum);
    if (lane == 0) lse2[g] = y == -INFINITY ? INFINITY : y;  // scores of -inf alone: no weight
    if (!join) continue;
    if (lane == 0 && a.lse) a.lse[row0 + g] = y * kLn2;
    float o[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
    for (int i0 = 0; i0 < a.nslot; i0 += 32) {
      // lane i: the weight of part i0 + i (an empty part's rows were not written)
      const float x = i0 == 0 ? x0 : i0 + lane < a.nslot ? lp[(i0 + lane) * rows] : -INFINITY;
      const float w = x == -INFINITY ? 0.f : exp2f(x - y);
      const unsigned some = __ballot_sync(0xffffffffu, x != -INFINITY);
      const int end = min(32, a.nslot - i0);
#pragma unroll 8
      for (int i = 0; i < end; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* src = a.o_part + ((i0 + i) * rows + row0 + g) * D + lane * (D / 32);
        float v[D / 32];
        if constexpr (D == 128)
          *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
        else
          *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = (some >> i) & 1 ? fmaf(wi, v[e], o[e]) : o[e];
      }
    }
    T* dst = static_cast<T*>(a.O) + (row0 + g) * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack16<T>(o[e], o[e + 1]);
  }
  if (join) return;
  __syncthreads();
  const float* score = a.score + (size_t)bh * a.G * a.cap;
  float* weights = a.weights + (size_t)bh * a.cap;
  // 8 keys a thread: their weights and two heads' scores in flight at once
  constexpr int kKeys = kFinishKeys / 256;
  const int j1 = n;
  for (int j = j0 + threadIdx.x; j < n; j += jstep) {
    float sum[kKeys], old[kKeys];
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
      old[e] = j + 256 * e < j1 ? weights[j + 256 * e] : 0.f;
      sum[e] = 0.f;
    }
#pragma unroll 2
    for (int g = 0; g < a.G; ++g) {
      const float y = lse2[g];
      const float* sg = score + (size_t)g * a.cap;
      float x[kKeys];
#pragma unroll
      for (int e = 0; e < kKeys; ++e) x[e] = j + 256 * e < j1 ? sg[j + 256 * e] : -INFINITY;
#pragma unroll
      for (int e = 0; e < kKeys; ++e) sum[e] += ex2_approx(x[e] - y);
    }
#pragma unroll
    for (int e = 0; e < kKeys; ++e)
      if (j + 256 * e < j1) weights[j + 256 * e] = old[e] + sum[e];
  }
}

namespace {
struct StepPlan {
  int nown, npre_rows, npre_tc;
  bool direct;
  size_t o_part, lse_part, score, total;
};

StepPlan step_plan(const StepArgs& a, bool with_weights) {
  StepPlan p{};
  const int own_rows = (a.G + 15) / 16;
  // own: enough CTAs for a few waves of three per SM, at least 16 tiles of a
  // full cache each
  const long long ctas = (long long)a.B * a.Hkv * own_rows;
  long long n = (8 * kSms + ctas - 1) / ctas;
  if (n > a.cap / 1024) n = a.cap / 1024;
  if (n > 64) n = 64;
  p.nown = a.cap == 0 ? 0 : n < 1 ? 1 : (int)n;
  if (a.P > 0) {
    const long long pre_rows = ((long long)a.B * a.G + 15) / 16;
    if (pre_rows == 1 || (a.P + kRowsKeys - 1) / kRowsKeys * pre_rows * a.Hkv <= kRowsPasses) {
      n = (4 * kSms + a.Hkv * pre_rows - 1) / (a.Hkv * pre_rows);
      if (n > a.P / 256) n = a.P / 256;
      if (n > 64) n = 64;
      p.npre_rows = n < 1 ? 1 : (int)n;
    } else {
      p.npre_tc = key_splits(row_pairs_one(a.B, a.G) * a.Hkv, a.P);
    }
  }
  const int nslot = p.nown + p.npre_rows + p.npre_tc;
  p.direct = nslot <= 1 && p.npre_tc == 0 && !with_weights;
  const size_t rows = (size_t)a.B * a.Hq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.lse_part = p.direct ? 0 : up(rows * nslot * a.d * 4);
  p.score = p.lse_part + (p.direct ? 0 : up(rows * nslot * 4));
  p.total = p.score + (with_weights ? up(rows * a.cap * 4) : 0);
  p.total = p.direct && !with_weights ? 256 : p.total < 512 ? 512 : p.total;  // 256: none needed
  return p;
}

template <typename T, int D, bool kLong>
cudaError_t run_rows(const RowsArgs& a, unsigned ctas, bool overlap, const CUtensorMap& kp, const CUtensorMap& vp,
                     const CUtensorMap& kc, const CUtensorMap& vc, cudaStream_t st) {
  const size_t sm = RowsSmem<D, kLong>::bytes();
  const cudaError_t e =
      cudaFuncSetAttribute(rows_kernel<T, D, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_after(rows_kernel<T, D, kLong>, dim3(ctas), kRowsThreads, sm, overlap, st, a, kp, vp, kc, vc);
}

template <typename T, int D>
cudaError_t run_step(const StepArgs& s, const StepPlan& p, cudaStream_t st) {
  RowsArgs a{};
  a.Q = s.Q;
  a.lens = s.lens;
  a.B = s.B;
  a.Hq = s.Hq;
  a.Hkv = s.Hkv;
  a.G = s.G;
  a.P = s.P;
  a.cap = s.cap;
  a.nown = p.nown;
  a.npre = p.npre_rows;
  a.nslot = p.nown + p.npre_rows + p.npre_tc;
  a.own_slot = p.npre_rows + p.npre_tc;
  a.own_rows = (s.G + 15) / 16;
  a.pre_rows = (int)(((long long)s.B * s.G + 15) / 16);
  a.direct = p.direct;
  a.scale_log2 = s.scale_log2;
  a.q_seq = s.q_seq;
  char* ws = static_cast<char*>(s.ws);
  a.o_part = reinterpret_cast<float*>(ws);
  a.lse_part = reinterpret_cast<float*>(ws + p.lse_part);
  a.score = s.weights ? reinterpret_cast<float*>(ws + p.score) : nullptr;
  a.O = s.O;
  a.lse = s.lse;
  a.weights = s.weights;
  cudaError_t e = cudaSuccess;
  // the prefix on the tensor cores
  auto prefix = [&](bool overlap) -> cudaError_t {
    TcArgs t{};
    t.Q = s.Q;
    t.o_part = a.o_part;
    t.lse_part = a.lse_part;
    t.nseq = 1;
    t.Hq = s.Hq;
    t.Hkv = s.Hkv;
    t.G = s.G;
    t.Tq = s.B;
    t.Tk = s.P;
    t.nsplit = p.npre_tc;
    t.ntile = (int)row_pairs_one(s.B, s.G);
    t.partial = true;
    t.scale_log2 = s.scale_log2;
    t.q_tok = s.q_seq;
    t.q_head = D;
    CUtensorMap tk, tv;
    cudaError_t e = make_tmap_rows(&tk, s.Kp, s.dtype, D, s.P, s.Hkv, D, s.prefix_head);
    if (e == cudaSuccess) e = make_tmap_rows(&tv, s.Vp, s.dtype, D, s.P, s.Hkv, D, s.prefix_head);
    return e != cudaSuccess ? e : run_attend<T, D>(t, tk, tv, st, overlap);
  };
  const long long ctas =
      (long long)a.npre * a.Hkv * a.pre_rows + (long long)a.nown * a.Hkv * a.B * a.own_rows;
  if (ctas > 0) {
    CUtensorMap kp, vp, kc, vc;
    // (a map that no CTA uses is a copy of the other)
    const bool pre = a.npre > 0, own = a.nown > 0;
    if (pre) {
      e = make_tmap_rows(&kp, s.Kp, s.dtype, D, s.P, s.Hkv, D, s.prefix_head, kRowsKeys);
      if (e == cudaSuccess) e = make_tmap_rows(&vp, s.Vp, s.dtype, D, s.P, s.Hkv, D, s.prefix_head, kRowsKeys);
    }
    if (own && e == cudaSuccess) {
      e = make_tmap_rows(&kc, s.Kc, s.dtype, D, s.cap, s.B * s.Hkv, D, (int64_t)s.cap * D, kRowsKeys);
      if (e == cudaSuccess) e = make_tmap_rows(&vc, s.Vc, s.dtype, D, s.cap, s.B * s.Hkv, D, (int64_t)s.cap * D, kRowsKeys);
    }
    if (e != cudaSuccess) return e;
    if (!pre) kp = kc, vp = vc;
    if (!own) kc = kp, vc = vp;
    // by the longest share: more than 32 tiles stream
    const int share = max(a.nown ? s.cap / a.nown : 0, a.npre ? s.P / a.npre : 0);
    const bool stream = share > 32 * kRowsKeys;
    // the prefix's CTAs take an SM each: they go first where the others leave
    // room for all of the caches' CTAs beside them
    const long long room = (kSms - (long long)p.npre_tc * row_pairs_one(s.B, s.G) * s.Hkv) * (stream ? 2 : 3);
    const bool prefix_first = p.npre_tc > 0 && ctas <= room;
    if (prefix_first) e = prefix(false);
    if (e == cudaSuccess)
      e = stream ? run_rows<T, D, true>(a, (unsigned)ctas, prefix_first, kp, vp, kc, vc, st)
                 : run_rows<T, D, false>(a, (unsigned)ctas, prefix_first, kp, vp, kc, vc, st);
    if (e == cudaSuccess && p.npre_tc > 0 && !prefix_first) e = prefix(true);
    if (e != cudaSuccess) return e;
  } else if (p.npre_tc > 0) {
    e = prefix(false);
    if (e != cudaSuccess) return e;
  }
  if (p.direct && ctas > 0) return cudaSuccess;
  // the weights' CTAs: about what the SMs hold at once
  const int caches = s.B * s.Hkv, chunks = (s.cap + kFinishKeys - 1) / kFinishKeys;
  const int share = min(chunks, (4 * kSms + caches - 1) / caches);
  const dim3 grid(caches, 1u + (s.weights ? (unsigned)share : 0u));
  return launch_after(finish_kernel<T, D>, grid, 256, s.G * 4, ctas > 0 || p.npre_tc > 0, st, a);
}
}  // namespace

size_t step_ws(const StepArgs& a, bool with_weights) { return step_plan(a, with_weights).total; }

cudaError_t launch_step(const StepArgs& a, cudaStream_t s) {
  const StepPlan p = step_plan(a, a.weights != nullptr);
  if (a.dtype == IG_BF16)
    return a.d == 128 ? run_step<__nv_bfloat16, 128>(a, p, s) : run_step<__nv_bfloat16, 64>(a, p, s);
  return a.d == 128 ? run_step<__half, 128>(a, p, s) : run_step<__half, 64>(a, p, s);
}

}  // namespace ig
