// gdn_plan.cu — the check of a packed batch and its division into segments, for the convolution and
// the selective scan: cu_seqlens must go from 0 to the token count without a step back, the slots must
// be distinct and inside the pool. A segment lies inside one sequence.
#include "gdn_ops.cuh"

namespace gdn {

namespace {

constexpr int kPlanThreads = 1024;  // and the largest batch that is checked and laid out in shared memory

// (a >= 0; a + b may not fit in 32 bits)
__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Sum over the warp's lanes, in every lane.
__device__ __forceinline__ int warp_sum_int(int x) { return __reduce_add_sync(0xffffffffu, x); }

// One block of a whole number of warps, at least B threads. Everything after the loads of idx and cu runs
// on shared memory; the two barriers before the table are what a short call waits for.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Plan plan, const int64_t* cu, const int64_t* idx, int B,
                                                            int64_t T, int64_t pool_size, SegmentRule rule) {
  __shared__ int64_t s_idx[kPlanThreads];
  __shared__ int s_start[kPlanThreads + 1], s_off[kPlanThreads + 1];
  launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t slot = tid < B ? idx[tid] : -1;
  const int64_t c0 = tid < B ? cu[tid] : T, c1 = tid < B ? cu[tid + 1] : T;
  const int64_t origin = cu[0], end = cu[B];
  s_idx[tid] = slot;
  if (tid < B) s_start[tid] = (int)c0;
  if (tid == 0) s_start[B] = (int)T;
  bool bad_seq = c1 < c0 || origin != 0 || end != T;
  bool bad_slot = tid < B && (slot < 0 || slot >= pool_size);
  if (B <= 32) {  // one warp holds all slots
    if (tid < 32) {
      const unsigned same = __match_any_sync(0xffffffffu, slot);  // every lane of the warp takes part
      bad_slot |= tid < B && __popc(same) > 1;
    }
    __syncthreads();
  } else {
    __syncthreads();
    const int until = min(B, tid);
#pragma unroll 8
    for (int j = 0; j < until; ++j) bad_slot |= s_idx[j] == slot;
  }
  bad_slot = bad_slot && tid < B;
  const int any_seq = __syncthreads_or(bad_seq), any_slot = __syncthreads_or(bad_slot);
  if (any_seq || any_slot) {
    if (tid == 0) {
      plan.status[1] = 0;
      plan.status[0] = any_seq ? GDN_ERR_BAD_SEQLENS : GDN_ERR_BAD_INDEX;
    }
    return;
  }

  // The segments' length: every warp by itself. Segments for one round of the card's blocks, where short
  // sequences (a quarter of a segment) fit in between; at most twice the even share of all tokens.
  int len = rule.least;
  if (rule.target > 0) {
    const int even = (int)min((T + rule.target - 1) / rule.target, (int64_t)INT32_MAX / 4);
    int lo = ceil_div(max(rule.least, even), rule.unit), hi = ceil_div(max(rule.least, 2 * even), rule.unit);  // units
    for (int mid = lo; lo < hi; mid = (lo + hi) >> 1) {  // the shortest first: one sequence, or equal ones, go by it
      const int l = mid * rule.unit;
      int count = 0;
      for (int s = lane; s < B; s += 32) {
        const int n = s_start[s + 1] - s_start[s];
        count += n > l / 4 ? ceil_div(n, l) : 0;
      }
      if (warp_sum_int(count) <= rule.target) hi = mid; else lo = mid + 1;
    }
    len = lo * rule.unit;
  }

  // First segment of each sequence, by the first warp: 32 sequences at a time.
  if (tid < 32) {
    int base = 0;
    for (int s0 = 0; s0 < B; s0 += 32) {
      const int s = s0 + lane;
      const int mine = s < B ? ceil_div(s_start[s + 1] - s_start[s], len) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (s < B) s_off[s] = base + incl - mine;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_off[B] = base;
  }
  __syncthreads();
  if (tid <= B) plan.seq_off[tid] = s_off[tid];
  if (tid == 0) plan.seq_off[B] = s_off[B];
  const int total = s_off[B];
  for (int j = tid; j < total; j += blockDim.x) {
    int lo = 0, hi = B - 1;  // the last sequence with s_off <= j (an empty one shares its offset with the next)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_off[mid] <= j) lo = mid; else hi = mid - 1;
    }
    const int c = j - s_off[lo], t0 = s_start[lo] + c * len;
    plan.seg_tab[j] = make_int4(lo, t0, min(len, s_start[lo + 1] - t0), c);
  }
  if (tid == 0) {
    plan.status[1] = total;
    plan.status[0] = GDN_OK;
  }
}

// The same for larger batches, whose slots the multi-block check has been over (the status word holds its
// outcome): segments of rule.least tokens, from global memory.
__global__ void __launch_bounds__(kPlanThreads) plan_large_kernel(Plan plan, const int64_t* cu, int B, int64_t T, int len) {
  __shared__ int s_warp[32];
  launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = cu[0] != 0 || cu[B] != T;
  for (int i = tid; i < B; i += kPlanThreads) bad |= cu[i + 1] < cu[i];
  const int any_seq = __syncthreads_or(bad), any_slot = plan.status[0] != GDN_OK;
  __syncthreads();
  if (any_seq || any_slot) {
    if (tid == 0) {
      plan.status[1] = 0;
      plan.status[0] = any_seq ? GDN_ERR_BAD_SEQLENS : GDN_ERR_BAD_INDEX;
    }
    return;
  }
  // Every thread owns a run of sequences; an exclusive sum over threads.
  const int per = ceil_div(B, kPlanThreads);
  const int s0 = min(B, tid * per), s1 = min(B, s0 + per);
  int mine = 0;
  for (int s = s0; s < s1; ++s) mine += ceil_div((int)(cu[s + 1] - cu[s]), len);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    before += w < warp ? s_warp[w] : 0;
    total += s_warp[w];
  }
  int at = before + incl - mine;
  for (int s = s0; s < s1; ++s) {
    plan.seq_off[s] = at;
    const int64_t n = cu[s + 1] - cu[s];
    for (int c = 0; (int64_t)c * len < n; ++c, ++at)
      plan.seg_tab[at] = make_int4(s, (int)(cu[s] + (int64_t)c * len), (int)min((int64_t)len, n - (int64_t)c * len), c);
  }
  if (tid == 0) {
    plan.seq_off[B] = total;
    plan.status[1] = total;
    plan.status[0] = GDN_OK;
  }
}

}  // namespace

SegmentRule segment_rule(int64_t T, int B, int unit, int least, int64_t target) {
  SegmentRule r{};
  r.unit = unit;
  r.least = least;
  if (B > kPlanThreads) {  // not cut at all: sequences enough to fill the card, unless most tokens are in a few of them
    r.least = (int)(T > least ? T : least);
  } else {
    r.target = (int)(target < (1 << 20) ? target : (1 << 20));
  }
  // A sequence of n tokens has at most n / len + 1 segments, and len is at least T / target.
  r.max_segs = T / r.least + B;
  if (r.target > 0 && r.max_segs > (int64_t)r.target + B) r.max_segs = (int64_t)r.target + B;
  return r;
}

cudaError_t launch_plan(const Plan& plan, const int64_t* cu_seqlens, const int64_t* cache_indices, int B, int64_t T,
                        int64_t pool_size, const SegmentRule& rule, cudaStream_t s, int* kernels) {
  if (B > kPlanThreads) {
    DecodeParams dp{};
    dp.cache_indices = cache_indices;
    dp.pool_size = pool_size;
    dp.B = B;
    dp.status = plan.status;
    if (cudaError_t e = cudaMemsetAsync(plan.status, 0, sizeof(int32_t), s)) return e;
    if (cudaError_t e = launch_decode_check(dp, s)) return e;
    plan_large_kernel<<<1, kPlanThreads, 0, s>>>(plan, cu_seqlens, B, T, rule.least);
    *kernels = 2;
    return cudaGetLastError();
  }
  const int64_t want = rule.max_segs < kPlanThreads ? (rule.max_segs > B ? rule.max_segs : B) : kPlanThreads;
  const int threads = (int)((want + 31) / 32 * 32 > 32 ? (want + 31) / 32 * 32 : 32);
  plan_kernel<<<1, threads, 0, s>>>(plan, cu_seqlens, cache_indices, B, T, pool_size, rule);
  *kernels = 1;
  return cudaGetLastError();
}

}  // namespace gdn
