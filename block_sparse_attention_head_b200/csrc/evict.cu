// Eviction from the caches by accumulated attention weight (instagen_evict).
//
// Two launches.  evict_select_kernel, one cluster of S CTAs per (sequence,
// head), each owning the r-th part of the slots: every slot gets a 32-bit key
// whose order is the order of eviction (recent, weight), and a radix select
// finds the key at the budget and how many of the slots equal to it stay (the
// lowest).  Weights and positions are read once, into registers and from them
// into shared memory; a pass counts one byte of the keys (in the first
// one lanes with equal bytes add together, because weights share their
// exponents) and the CTAs of a cluster add their counts through distributed
// shared memory.  Then each
// warp walks a contiguous range of slots and, from the counts of the ranges
// before, lists the freed slots below the budget and the kept slots from the
// budget on.  The pass over the slots is a chain of latencies, so S grows (to
// 8) while there are SMs without a CTA: 64 caches of 16384 keys take 18 us in
// clusters of 4 and 37 alone.  evict_move_kernel copies rows: the n-th of those
// into the n-th of these (in place), or every kept row (into another cache); it
// is bound by the rows' bytes.  Sources are at or above the budget and
// destinations below it, so moving in place has no order.
#include "serve.cuh"

#include <cooperative_groups.h>

namespace ig {

namespace {
constexpr int kEvictKeys = 49152;  // keys held in a CTA's shared memory; longer parts are read again in every pass
constexpr int kEvictBatch = 8;     // slots a thread loads at once
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

// kHeld: the keys of a CTA's part fit shared memory.
template <bool kHeld>
__global__ void __launch_bounds__(1024) evict_select_kernel(EvictArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t held[];
  __shared__ int own[256];      // a pass's counts
  __shared__ int all[2][256];   // and the cluster's, alternating: zeroed a pass ahead
  __shared__ int sums[32];
  __shared__ int share[4];      // what the peers read: newest, recent slots, and the walk's counts
  __shared__ int part[8][2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_equal;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / S, b = bh / a.Hkv, nt = blockDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  const int n = live_slots(a.lens, b, a.cap);
  int32_t* dst = l.dst + (size_t)bh * a.budget;
  int32_t* src = l.src + (size_t)bh * a.budget;
  launch_dependents();
  if (tid == 0 && rank == 0 && bh % a.Hkv == 0) l.n[b] = n;
  if (n <= a.budget) {  // everything stays (all CTAs of the cluster leave here)
    if (!a.in_place)
      for (int i = rank * nt + tid; i < n; i += S * nt) src[i] = i;
    if (tid == 0 && rank == 0) l.count[bh] = a.in_place ? 0 : n;
    return;
  }
  // this CTA's slots [c0, c1), a whole number of warp steps but for the last
  const int per = (n + 32 * S - 1) / (32 * S) * 32;
  const int c0 = min(n, rank * per), c1 = min(n, c0 + per), cn = c1 - c0;
  const float* w = a.weights + (size_t)bh * a.cap + c0;
  const int32_t* pos = a.pos + (size_t)bh * a.cap + c0;
  // the sum (or maximum) over the cluster of one value per CTA
  auto cluster_all = [&](int v, int slot, bool maximum) -> int {
    if (tid == 0) share[slot] = v;
    if (S == 1) {
      __syncthreads();
      return share[slot];
    }
    cluster.sync();
    int all = maximum ? INT32_MIN : 0;
    for (int r = 0; r < S; ++r) {
      const int x = *cluster.map_shared_rank(&share[slot], r);
      all = maximum ? max(all, x) : all + x;
    }
    return all;
  };
  auto block_reduce = [&](int v, bool maximum) -> int {  // in thread 0
    v = maximum ? __reduce_max_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    v = lane < (nt >> 5) ? sums[lane] : maximum ? INT32_MIN : 0;
    return maximum ? __reduce_max_sync(0xffffffffu, v) : __reduce_add_sync(0xffffffffu, v);
  };

  // weights and positions on their way together; short parts stay in registers
  float w0[kEvictBatch];
  int32_t p0[kEvictBatch];
  int newest = INT32_MIN;
#pragma unroll
  for (int e = 0; e < kEvictBatch; ++e) {
    const int i = tid + e * nt;
    w0[e] = i < cn ? w[i] : 0.f;
    p0[e] = i < cn ? pos[i] : INT32_MIN;
  }
#pragma unroll
  for (int e = 0; e < kEvictBatch; ++e) newest = max(newest, p0[e]);
#pragma unroll 4
  for (int i = tid + kEvictBatch * nt; i < cn; i += nt) newest = max(newest, pos[i]);
  if (tid == 0) {
    s_need = a.budget;
    s_prefix = 0;
  }
  for (int i = tid; i < 256; i += nt) all[0][i] = 0;
  newest = cluster_all(block_reduce(newest, true), 0, true);
  // the recent slots: pos > newest - recent
  const long long edge = (long long)newest - a.recent;
  int safe = 0;
#pragma unroll
  for (int e = 0; e < kEvictBatch; ++e) safe += tid + e * nt < cn && p0[e] > edge;
#pragma unroll 4
  for (int i = tid + kEvictBatch * nt; i < cn; i += nt) safe += pos[i] > edge;
  safe = cluster_all(block_reduce(safe, false), 1, false);
  // either there are enough recent slots and the others are below all of
  // them, or the recent ones are above all others
  const bool among_safe = safe >= a.budget;
  auto make_key = [&](float x, int32_t at) -> uint32_t {
    return (at > edge) == among_safe ? ordered_bits(x) : among_safe ? 0u : 0xffffffffu;
  };
  if (kHeld) {
#pragma unroll
    for (int e = 0; e < kEvictBatch; ++e)
      if (tid + e * nt < cn) held[tid + e * nt] = make_key(w0[e], p0[e]);
#pragma unroll 4
    for (int i = tid + kEvictBatch * nt; i < cn; i += nt) held[i] = make_key(w[i], pos[i]);
  }
  auto key_at = [&](int i) -> uint32_t { return kHeld ? held[i] : make_key(w[i], pos[i]); };

  // radix select: after a pass, s_prefix holds the leading bytes of the key
  // at the budget, s_equal how many slots share them and s_need how many of
  // those stay; done when all of them do.  Every CTA of the cluster finds the
  // same.
  uint32_t mask = 0;
  for (int shift = 24, pass = 0; shift >= 0; shift -= 8, ++pass) {
    // (the next pass's total is zeroed before this pass's cluster.sync, which
    // every peer's additions to it come after; the first one before the syncs
    // above)
    for (int i = tid; i < 256; i += nt) {
      own[i] = 0;
      all[(pass & 1) ^ 1][i] = 0;
    }
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i0 = warp * 32; i0 < cn; i0 += nt) {
      const int i = i0 + lane;
      const uint32_t key = i < cn ? key_at(i) : 0u;
      const bool in = i < cn && (key & mask) == prefix;
      const int digit = (int)((key >> shift) & 255);
      if (pass > 0) {
        if (in) atomicAdd(&own[digit], 1);
        continue;
      }
      // sign and exponent: a warp holds few different ones, each added once
      const unsigned peers = __match_any_sync(0xffffffffu, in ? digit : 256);
      if (in && lane == __ffs(peers) - 1) atomicAdd(&own[digit], __popc(peers));
    }
    __syncthreads();
    const int* total = own;
    if (S > 1) {  // every CTA adds its counts to every CTA's total
      total = all[pass & 1];
      for (int i = tid; i < 256; i += nt)
        if (own[i])
          for (int r = 0; r < S; ++r) atomicAdd(cluster.map_shared_rank(&all[pass & 1][i], r), own[i]);
      cluster.sync();
    }
    if (warp == 0) {  // the largest byte whose count from above reaches need
      int c[8], mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = total[255 - (8 * lane + e)];
        mine += c[e];
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int need = s_need;
      int run = incl - mine;
      __syncwarp();
      if (run < need && need <= incl) {
        bool found = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!found && run + c[e] >= need) {
            s_prefix = prefix | ((uint32_t)(255 - (8 * lane + e)) << shift);
            s_need = need - run;
            s_equal = c[e];
            found = true;
          }
          run += c[e];
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

  // ordered walk: every warp owns a contiguous range of the CTA's slots
  const int nw = nt >> 5, seg = (cn + 32 * nw - 1) / (32 * nw) * 32;
  const int i0 = min(cn, warp * seg), i1 = min(cn, i0 + seg);
  const unsigned below = (1u << lane) - 1;
  // what the CTAs before this one count
  auto ranks_before = [&](int v, int slot) -> int {
    if (S == 1) return 0;
    if (tid == 0) share[slot] = v;
    cluster.sync();
    int before = 0;
    for (int r = 0; r < rank; ++r) before += *cluster.map_shared_rank(&share[slot], r);
    return before;
  };
  int equal_before = 0;
  if (!all_equal) {
    int equal = 0;
    for (int i = i0 + lane; i < i1; i += 32) equal += (key_at(i) & mask) == level;
    equal = __reduce_add_sync(0xffffffffu, equal);
    equal_before = warps_before(equal, sums);
    equal_before += ranks_before(block_reduce(lane == 0 ? equal : 0, false), 2);
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
      f(c0 + i, i < i1 && !kept && c0 + i < a.budget, i < i1 && kept && c0 + i >= a.budget);
    }
  };
  int freed = 0, moving = 0;
  each([&](int, bool free, bool moves) {
    freed += __popc(__ballot_sync(0xffffffffu, free));
    moving += __popc(__ballot_sync(0xffffffffu, moves));
  });
  int f = warps_before(freed, sums), m = warps_before(moving, sums);
  if (S > 1) {
    // the CTAs' totals, both in one exchange
    const int tf = block_reduce(lane == 0 ? freed : 0, false), tm = block_reduce(lane == 0 ? moving : 0, false);
    if (tid == 0) {
      share[0] = tf;
      share[3] = tm;
    }
    cluster.sync();
    if (tid < 2 * S) part[tid >> 1][tid & 1] = *cluster.map_shared_rank(&share[tid & 1 ? 3 : 0], tid >> 1);
    __syncthreads();
    for (int r = 0; r < rank; ++r) {
      f += part[r][0];
      m += part[r][1];
    }
  }
  if (rank == S - 1 && warp == nw - 1 && lane == 0) l.count[bh] = a.in_place ? f + freed : a.budget;
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
    // src of a slot that stays is itself, of the f-th freed one ~f: the move
    // looks the f-th moving slot up
    each([&](int i, bool free, bool moves) {
      const unsigned fs = __ballot_sync(0xffffffffu, free), ms = __ballot_sync(0xffffffffu, moves);
      if (moves) from[m + __popc(ms & below)] = i;
      if (i < c0 + i1 && i < a.budget) src[i] = free ? ~(f + __popc(fs & below)) : i;
      f += __popc(fs);
      m += __popc(ms);
    });
  }
  if (S > 1) cluster.sync();  // no CTA ends while a peer may still read its shared memory
}

template <int D>
__global__ void __launch_bounds__(kEvictMoveThreads) evict_move_kernel(EvictArgs a) {
  constexpr int kLanes = D / 8;                        // 16-byte chunks of a row
  constexpr int kGroup = kEvictMoveThreads / kLanes;   // rows at once
  const int bh = blockIdx.y, b = bh / a.Hkv;
  const EvictLists l = carve(a.ws, a.B, a.Hkv, a.budget);
  wait_prior_grids();
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
    int s = src[r];
    if (s < 0) s = dst[~s];  // a freed slot's number: the moving slot of that number
    const size_t from = in0 + s;
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

template <bool kHeld>
static cudaError_t run_select(const EvictArgs& a, int S, int threads, size_t smem, cudaStream_t s) {
  if (smem > 40 * 1024) {  // 48 KB with the static part need no leave
    // the most that any call asks for: the limit is the kernel's, and another
    // thread's call may be between setting it and its launch
    const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<kHeld>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kEvictKeys * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)S;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * S));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<kHeld>, a);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  // CTAs per cache: doubled while there are SMs without one and a CTA's part
  // is longer than 2048 slots
  int S = 1;
  while (S < 8 && 2 * S * a.B * a.Hkv <= 2 * kSms && a.cap / S > 2048) S *= 2;
  const int per = (a.cap + 32 * S - 1) / (32 * S) * 32;
  // short parts: several CTAs per SM; long ones: all of an SM's threads
  const int threads = per <= 2048 ? 256 : per <= 4096 ? 512 : 1024;
  cudaError_t e = per <= kEvictKeys ? run_select<true>(a, S, threads, (size_t)per * 4, s)
                                    : run_select<false>(a, S, threads, 0, s);
  if (e != cudaSuccess) return e;
  const int rows = a.in_place ? min(a.budget, a.cap - a.budget) : a.budget;
  const int per_cta = kEvictMoveThreads / (a.d / 8) * kEvictMoveRows;
  const dim3 grid((unsigned)max(1, (rows + per_cta - 1) / per_cta), (unsigned)(a.B * a.Hkv));
  return a.d == 128 ? launch_after(evict_move_kernel<128>, grid, kEvictMoveThreads, 0, true, s, a)
                    : launch_after(evict_move_kernel<64>, grid, kEvictMoveThreads, 0, true, s, a);
}

}  // namespace ig
