// Eviction from the caches by accumulated attention weight (instagen_evict).
//
// Two launches.  evict_select_kernel, one CTA per (sequence, head): the slots
// compete by (recent, weight, lower slot).  A radix select over the weights'
// ordered bits, one byte per pass, finds the weight at the budget and how many
// of the keys equal to it stay (the lowest slots); one ordered pass then lists
// the freed slots below the budget and the kept slots from the budget on.
// evict_move_kernel copies rows: the n-th of those into the n-th of these (in
// place), or every kept row (into another cache).  Sources are at or above
// the budget and destinations below it, so moving in place has no order.
#include "serve.cuh"

namespace ig {

namespace {
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMoveThreads = 256;
constexpr int kEvictMoveRows = 32;  // rows per CTA of the move kernel

// Ordered bits: a < b as numbers iff bits(a) < bits(b); -0 counts as +0, NaN
// is below everything.
__device__ __forceinline__ uint32_t ordered_bits(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // warp_sums may still be read by the last scan
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[kEvictWarps - 1];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
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

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[kEvictWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_newest, s_safe;
  const int bh = blockIdx.x, b = bh / a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  const int n = live_slots(a.lens, b, a.cap);
  if (tid == 0 && bh % a.Hkv == 0) l.n[b] = n;
  int32_t* dst = l.dst + (size_t)bh * a.budget;
  int32_t* src = l.src + (size_t)bh * a.budget;
  if (n <= a.budget) {  // everything stays
    if (!a.in_place)
      for (int i = tid; i < n; i += kEvictThreads) src[i] = i;
    if (tid == 0) l.count[bh] = a.in_place ? 0 : n;
    return;
  }
  const float* w = a.weights + (size_t)bh * a.cap;
  const int32_t* pos = a.pos + (size_t)bh * a.cap;

  // the recent slots: pos > newest - recent
  int newest = INT32_MIN;
  for (int i = tid; i < n; i += kEvictThreads) newest = max(newest, pos[i]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (tid == 0) {
    s_newest = INT32_MIN;
    s_safe = 0;
  }
  __syncthreads();
  if (lane == 0) atomicMax(&s_newest, newest);
  __syncthreads();
  const long long edge = (long long)s_newest - a.recent;
  int safe = 0;
  for (int i = tid; i < n; i += kEvictThreads) safe += pos[i] > edge;
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0) atomicAdd(&s_safe, safe);
  __syncthreads();
  // either the recent slots alone compete (there are enough of them), or all
  // of them stay and the others compete for what is left of the budget
  const bool among_safe = s_safe >= a.budget;
  if (tid == 0) {
    s_need = among_safe ? a.budget : a.budget - s_safe;
    s_prefix = 0;
  }
  __syncthreads();
  auto competes = [&](int i) { return (pos[i] > edge) == among_safe; };

  // radix select: after a pass, s_prefix holds the leading bytes of the
  // weight at the budget and s_need how many of the slots sharing them stay
  uint32_t mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i = tid; i < n; i += kEvictThreads) {
      const uint32_t key = ordered_bits(w[i]);
      if (competes(i) && (key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < 32) {  // the largest byte whose suffix count reaches need
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
            break;
          }
          run += hist[byte];
        }
      }
    }
    mask |= 255u << shift;
    __syncthreads();
  }
  const uint32_t level = s_prefix;
  const int equal_kept = s_need;

  // ordered pass: every thread owns a contiguous run of slots
  const int run_len = (n + kEvictThreads - 1) / kEvictThreads;
  const int i0 = min(n, tid * run_len), i1 = min(n, i0 + run_len);
  int equal = 0, total;
  for (int i = i0; i < i1; ++i) equal += competes(i) && ordered_bits(w[i]) == level;
  const int equal_before = block_scan(equal, warp_sums, &total);
  auto each = [&](auto f) {
    int eq = equal_before;
    for (int i = i0; i < i1; ++i) {
      bool kept;
      if (competes(i)) {
        const uint32_t key = ordered_bits(w[i]);
        kept = key > level || (key == level && eq < equal_kept);
        eq += key == level;
      } else {
        kept = !among_safe;
      }
      f(i, kept);
    }
  };
  int freed = 0, moving = 0;
  each([&](int i, bool kept) {
    freed += i < a.budget && !kept;
    moving += i >= a.budget && kept;
  });
  int count, count2;
  int f = block_scan(freed, warp_sums, &count);
  int m = block_scan(moving, warp_sums, &count2);
  int32_t* from = a.in_place ? src : dst;  // out of place: dst is the list of the moving slots first
  each([&](int i, bool kept) {
    if (i >= a.budget && kept) from[m++] = i;
  });
  __syncthreads();
  each([&](int i, bool kept) {
    if (i < a.budget) {
      if (a.in_place) {
        if (!kept) dst[f++] = i;
      } else {
        src[i] = kept ? i : from[f++];
      }
    }
  });
  if (tid == 0) l.count[bh] = a.in_place ? count : a.budget;
}

template <int D>
__global__ void __launch_bounds__(kEvictMoveThreads) evict_move_kernel(EvictArgs a) {
  constexpr int kLanes = D / 8;  // 16-byte chunks of a row
  const int bh = blockIdx.y, b = bh / a.Hkv;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  const int count = l.count[bh];
  if (blockIdx.x == 0 && bh % a.Hkv == 0 && threadIdx.x == 0) a.lens_out[b] = min(l.n[b], a.budget);
  const int32_t* dst = l.dst + (size_t)bh * a.budget;
  const int32_t* src = l.src + (size_t)bh * a.budget;
  const size_t in0 = (size_t)bh * a.cap, out0 = (size_t)bh * a.cap_out;
  const int c = threadIdx.x % kLanes;
  const int end = min(count, (int)(blockIdx.x + 1) * kEvictMoveRows);
  for (int r = blockIdx.x * kEvictMoveRows + threadIdx.x / kLanes; r < end; r += kEvictMoveThreads / kLanes) {
    const size_t from = in0 + src[r], to = out0 + (a.in_place ? dst[r] : r);
    const uint4 k = static_cast<const uint4*>(a.K)[from * kLanes + c];
    const uint4 v = static_cast<const uint4*>(a.V)[from * kLanes + c];
    static_cast<uint4*>(a.K_out)[to * kLanes + c] = k;
    static_cast<uint4*>(a.V_out)[to * kLanes + c] = v;
    if (c == 0) {
      a.weights_out[to] = a.weights[from];
      a.pos_out[to] = a.pos[from];
    }
  }
}
}  // namespace

size_t evict_ws(int B, int Hkv, int budget) {
  return ((size_t)B + (size_t)B * Hkv * (1 + 2 * (size_t)budget)) * 4;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  evict_select_kernel<<<a.B * a.Hkv, kEvictThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int rows = a.in_place ? min(a.budget, a.cap - a.budget) : a.budget;
  const dim3 grid((unsigned)max(1, (rows + kEvictMoveRows - 1) / kEvictMoveRows), (unsigned)(a.B * a.Hkv));
  if (a.d == 128)
    evict_move_kernel<128><<<grid, kEvictMoveThreads, 0, s>>>(a);
  else
    evict_move_kernel<64><<<grid, kEvictMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace ig
