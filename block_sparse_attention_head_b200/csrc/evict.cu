// Eviction from the caches by accumulated attention weight (instagen_evict).
//
// Two launches.  evict_select_kernel, one CTA per (sequence, head): every slot
// gets a 32-bit key whose order is the order of eviction (recent, weight), and
// a radix select finds the key at the budget and how many of the slots equal
// to it stay (the lowest).  Weights and positions are read once into shared
// memory (twice the positions: the recent ones are known once the newest is);
// a pass counts one byte of the keys, lanes with equal bytes adding together,
// because weights share their exponents.  Then each warp walks a contiguous
// range of slots and, from the counts of the ranges before, lists the freed
// slots below the budget and the kept slots from the budget on.
// evict_move_kernel copies rows: the n-th of those into the n-th of these (in
// place), or every kept row (into another cache); it is bound by the rows'
// bytes.  Sources are at or above the budget and destinations below it, so
// moving in place has no order.
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kEvictKeys = 49152;  // keys held in shared memory; longer caches are read again in every pass
constexpr int kEvictMoveThreads = 256;
constexpr int kEvictMoveRows = 4;  // rows a thread copies, all loads in flight at once

// Ordered bits: a < b as numbers iff bits(a) < bits(b); -0 counts as +0, NaN
// is 1, below everything.  0 and 2^32 - 1 are no number's.
__device__ __forceinline__ uint32_t ordered_bits(float w) {
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block's warps of a value that each warp's
// lanes share.
__device__ __forceinline__ int warps_before(int v, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  __syncthreads();  // sums may still be read by the last call
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, lane < warp && lane < nw ? sums[lane] : 0);
}

struct EvictLists {
  int32_t* n;      // [B] live slots before
  int32_t* count;  // [B, Hkv] rows to move
  int32_t* dst;    // [B, Hkv, budget]
  int32_t* src;    // [B, Hkv, budget]
};

__host__ __device__ inline EvictLists carve(void* ws, int B, int Hkv, int budget) {
  EvictLists l;
  l.n = static_cast<int32_t*>(ws);
  l.count = l.n + B;
  l.dst = l.count + (size_t)B * Hkv;
  l.src = l.dst + (size_t)B * Hkv * budget;
  return l;
}

// kHeld: the keys fit shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(1024) evict_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t held[];
  __shared__ int hist[256];
  __shared__ int sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_equal, s_newest, s_safe;
  const int bh = blockIdx.x, b = bh / a.Hkv, nt = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  const int n = live_slots(a.lens, b, a.cap);
  if (tid == 0 && bh % a.Hkv == 0) l.n[b] = n;
  int32_t* dst = l.dst + (size_t)bh * a.budget;
  int32_t* src = l.src + (size_t)bh * a.budget;
  if (n <= a.budget) {  // everything stays
    if (!a.in_place)
      for (int i = tid; i < n; i += nt) src[i] = i;
    if (tid == 0) l.count[bh] = a.in_place ? 0 : n;
    return;
  }
  const float* w = a.weights + (size_t)bh * a.cap;
  const int32_t* pos = a.pos + (size_t)bh * a.cap;

  // the recent slots: pos > newest - recent
  int newest = INT32_MIN;
#pragma unroll 8
  for (int i = tid; i < n; i += nt) newest = max(newest, pos[i]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (tid == 0) {
    s_newest = INT32_MIN;
    s_safe = 0;
    s_need = a.budget;
    s_prefix = 0;
  }
  __syncthreads();
  if (lane == 0) atomicMax(&s_newest, newest);
  __syncthreads();
  const long long edge = (long long)s_newest - a.recent;
  int safe = 0;
#pragma unroll 8
  for (int i = tid; i < n; i += nt) safe += pos[i] > edge;
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0) atomicAdd(&s_safe, safe);
  __syncthreads();
  // either there are enough recent slots and the others are below all of
  // them, or the recent ones are above all others
  const bool among_safe = s_safe >= a.budget;
  auto read_key = [&](int i) -> uint32_t {
    const uint32_t key = ordered_bits(w[i]);
    return (pos[i] > edge) == among_safe ? key : among_safe ? 0u : 0xffffffffu;
  };
  if (kHeld) {
#pragma unroll 8
    for (int i = tid; i < n; i += nt) held[i] = read_key(i);
    __syncthreads();
  }
  auto key_at = [&](int i) -> uint32_t { return kHeld ? held[i] : read_key(i); };

  // radix select: after a pass, s_prefix holds the leading bytes of the key
  // at the budget, s_equal how many slots share them and s_need how many of
  // those stay; done when all of them do
  uint32_t mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += nt) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i0 = warp * 32; i0 < n; i0 += nt) {
      const int i = i0 + lane;
      const uint32_t key = i < n ? key_at(i) : 0u;
      const bool in = i < n && (key & mask) == prefix;
      const int digit = in ? (int)((key >> shift) & 255) : 256;
      const unsigned peers = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&hist[digit], __popc(peers));
    }
    __syncthreads();
    if (warp == 0) {  // the largest byte whose count from above reaches need
      int own = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) own += hist[255 - (8 * lane + e)];
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int need = s_need;
      int run = incl - own;
      __syncwarp();
      if (run < need && need <= incl) {
        for (int e = 0; e < 8; ++e) {
          const int byte = 255 - (8 * lane + e);
          if (run + hist[byte] >= need) {
            s_prefix = prefix | ((uint32_t)byte << shift);
            s_need = need - run;
            s_equal = hist[byte];
            break;
          }
          run += hist[byte];
        }
      }
    }
    mask |= 255u << shift;
    __syncthreads();
    if (s_need == s_equal) break;
  }
  const uint32_t level = s_prefix;
  const int equal_kept = s_need;
  const bool all_equal = s_need == s_equal;

  // ordered walk: every warp owns a contiguous range of slots
  const int nw = nt >> 5, seg = (n + 32 * nw - 1) / (32 * nw) * 32;
  const int i0 = min(n, warp * seg), i1 = min(n, i0 + seg);
  const unsigned below = (1u << lane) - 1;
  int equal_before = 0;
  if (!all_equal) {
    int equal = 0;
    for (int i = i0 + lane; i < i1; i += 32) equal += (key_at(i) & mask) == level;
    equal_before = warps_before(__reduce_add_sync(0xffffffffu, equal), sums);
  }
  // f(slot, below the budget and freed, from the budget on and kept) for the
  // range's slots, 32 at a time
  auto each = [&](auto f) {
    int eq = equal_before;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
      const uint32_t key = i < i1 ? key_at(i) & mask : 0u;
      bool kept = key > level;
      if (all_equal) {
        kept = key >= level;
      } else {
        const unsigned same = __ballot_sync(0xffffffffu, i < i1 && key == level);
        if (key == level) kept = eq + __popc(same & below) < equal_kept;
        eq += __popc(same);
      }
      f(i, i < i1 && !kept && i < a.budget, i < i1 && kept && i >= a.budget);
    }
  };
  int freed = 0, moving = 0;
  each([&](int, bool free, bool moves) {
    freed += __popc(__ballot_sync(0xffffffffu, free));
    moving += __popc(__ballot_sync(0xffffffffu, moves));
  });
  int f = warps_before(freed, sums), m = warps_before(moving, sums);
  if (warp == nw - 1 && lane == 0) l.count[bh] = a.in_place ? f + freed : a.budget;
  int32_t* from = a.in_place ? src : dst;  // out of place: dst is the list of the moving slots
  if (a.in_place) {
    each([&](int i, bool free, bool moves) {
      const unsigned fs = __ballot_sync(0xffffffffu, free), ms = __ballot_sync(0xffffffffu, moves);
      if (free) dst[f + __popc(fs & below)] = i;
      if (moves) src[m + __popc(ms & below)] = i;
      f += __popc(fs);
      m += __popc(ms);
    });
  } else {
    each([&](int i, bool, bool moves) {
      const unsigned ms = __ballot_sync(0xffffffffu, moves);
      if (moves) from[m + __popc(ms & below)] = i;
      m += __popc(ms);
    });
    __syncthreads();
    each([&](int i, bool free, bool) {
      const unsigned fs = __ballot_sync(0xffffffffu, free);
      if (i < i1 && i < a.budget) src[i] = free ? from[f + __popc(fs & below)] : i;
      f += __popc(fs);
    });
  }
}

template <int D>
__global__ void __launch_bounds__(kEvictMoveThreads) evict_move_kernel(EvictArgs a) {
  constexpr int kLanes = D / 8;                        // 16-byte chunks of a row
  constexpr int kGroup = kEvictMoveThreads / kLanes;   // rows at once
  const int bh = blockIdx.y, b = bh / a.Hkv;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  const int count = l.count[bh];
  if (blockIdx.x == 0 && bh % a.Hkv == 0 && threadIdx.x == 0) a.lens_out[b] = min(l.n[b], a.budget);
  const int32_t* dst = l.dst + (size_t)bh * a.budget;
  const int32_t* src = l.src + (size_t)bh * a.budget;
  const size_t in0 = (size_t)bh * a.cap, out0 = (size_t)bh * a.cap_out;
  const int c = threadIdx.x % kLanes, r0 = blockIdx.x * (kGroup * kEvictMoveRows) + threadIdx.x / kLanes;
  uint4 k[kEvictMoveRows], v[kEvictMoveRows];
  float w[kEvictMoveRows];
  int32_t p[kEvictMoveRows];
#pragma unroll
  for (int e = 0; e < kEvictMoveRows; ++e) {
    const int r = r0 + e * kGroup;
    if (r >= count) break;
    const size_t from = in0 + src[r];
    k[e] = static_cast<const uint4*>(a.K)[from * kLanes + c];
    v[e] = static_cast<const uint4*>(a.V)[from * kLanes + c];
    if (c == 0) {
      w[e] = a.weights[from];
      p[e] = a.pos[from];
    }
  }
#pragma unroll
  for (int e = 0; e < kEvictMoveRows; ++e) {
    const int r = r0 + e * kGroup;
    if (r >= count) break;
    const size_t to = out0 + (a.in_place ? dst[r] : r);
    static_cast<uint4*>(a.K_out)[to * kLanes + c] = k[e];
    static_cast<uint4*>(a.V_out)[to * kLanes + c] = v[e];
    if (c == 0) {
      a.weights_out[to] = w[e];
      a.pos_out[to] = p[e];
    }
  }
}
}  // namespace

size_t evict_ws(int B, int Hkv, int budget) {
  return ((size_t)B + (size_t)B * Hkv * (1 + 2 * (size_t)budget)) * 4;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  // short caches: several CTAs per SM; long ones: all of an SM's threads
  const int threads = a.cap <= 4096 ? 256 : 1024;
  cudaError_t e = cudaSuccess;
  if (a.cap <= kEvictKeys) {
    e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictKeys * 4);
    if (e != cudaSuccess) return e;
    evict_select_kernel<true><<<a.B * a.Hkv, threads, (size_t)a.cap * 4, s>>>(a);
  } else {
    evict_select_kernel<false><<<a.B * a.Hkv, threads, 0, s>>>(a);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = a.in_place ? min(a.budget, a.cap - a.budget) : a.budget;
  const int per_cta = kEvictMoveThreads / (a.d / 8) * kEvictMoveRows;
  const dim3 grid((unsigned)max(1, (rows + per_cta - 1) / per_cta), (unsigned)(a.B * a.Hkv));
  if (a.d == 128)
    evict_move_kernel<128><<<grid, kEvictMoveThreads, 0, s>>>(a);
  else
    evict_move_kernel<64><<<grid, kEvictMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ig
