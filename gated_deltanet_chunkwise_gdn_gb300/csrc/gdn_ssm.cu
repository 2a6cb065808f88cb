// gdn_ssm.cu — the selective state space scan over a packed batch and for single tokens, against a
// pool of fp32 states. For channel d (group g = d / (D / G)) and state n, token by token:
//
//   delta = softplus(dt + dt_bias)   (or dt + dt_bias)
//   h_n   = exp(delta A_{d,n}) h_n + delta x B_{g,n}
//   y     = sum_n C_{g,n} h_n + Dskip x,     out = y z sigmoid(z)   (or y)
//
// A thread owns one, two or four neighbouring channels (as many as load at once) and up to 16 of their
// states; more states are shared by 2 or 4 neighbouring lanes. The recurrence runs in registers, two
// states to a packed fp32 instruction; B and C of a tile of tokens are widened once per block into shared
// memory and read from there by every lane at once, so four channels a thread read them half as often
// as two: 16384 tokens x 4096 channels take 489 us with four, 507 with two, 729 with one.
//
// A prompt with few channels has too few threads for the card, so every sequence is cut into segments:
//   1. ssm_scan_kernel, MODE 1: each segment but the last of its sequence, from a zero state, gives its end
//      state and the sum of its deltas (exp(A sum delta) is the whole segment's decay).
//   2. ssm_carry_kernel: the segments' start states, in order, from the slot's state.
//   3. ssm_scan_kernel, MODE 0: each segment from its start state, with its outputs.
//
// What bounds it is not HBM (1.5 to 2 TB/s) but the arithmetic: two states and a token are two exponentials and
// three packed instructions, with the output four. A scheduler does a warp's ex2 in 4 cycles and a packed fp32
// instruction with three different operands in about 3, so 16 states of 32 channels take
// about 90 cycles without outputs and 106 with them (a loop of nothing else, measured); 65536 tokens x 2048
// channels take 297 and 355 us by that, and 369 and 538 us as measured, with the softplus, the gate's SiLU,
// the rows' conversions and B and C beside it. The first pass is two thirds of the third, so ssm_segments()
// cuts no finer than it takes to fill the card.
#include "gdn_ssm.cuh"

namespace gdn {

namespace {

// MODE 0: outputs from the start state, the end state to the pool. MODE 1: end state from zero only.
template <typename E, int V, int S, int P, int MODE>
__global__ void __launch_bounds__(kSsmThreads, 2) ssm_scan_kernel(SsmParams p, int blocks_per_group) {
  using M = SsmMap<V, S, P>;
  constexpr int kPer = MODE == 0 ? 2 : 1;       // B and C, or B
  constexpr int kTile = (M::kStates % 3 ? 512 : 384) / M::kStates;  // tokens of B and C in shared memory at a time
  constexpr int kStage = kTile * kPer * M::kStates / kSsmThreads;  // values a thread brings
  constexpr int U = V == 4 && MODE == 0 ? 2 : kSsmUnroll;   // tokens computed at a time, by the registers
  static_assert(kTile % U == 0, "whole groups of tokens in a tile");
  constexpr int kRows = MODE == 0 ? 3 : 2;      // x, dt and z, or x and dt
  constexpr int NG = V == 4 && MODE == 0 ? 6 : kSsmGroups;  // groups of rows in the ring
  __shared__ __align__(16) float s_bc[2][kTile][kPer][M::kStates];
  __shared__ RowRing<E, V, kRows, U * NG, kSsmThreads, true> ring;
  launch_dependents();
  const int nblk = blocks_per_group * p.G;
  const int seg = blockIdx.x / nblk, blk = blockIdx.x % nblk;
  const M m(p, blk / blocks_per_group, blk % blocks_per_group);
  float2 A2[V][S / 2];
  m.load_A(A2, p);
  float bias[V], skip[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = p.dt_bias && m.live ? p.dt_bias[m.d0 + v] : 0.f;
    skip[v] = MODE == 0 && p.Dskip && m.live ? p.Dskip[m.d0 + v] : 0.f;
  }
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK || seg >= p.plan.status[1]) return;
  const int4 sg = p.plan.seg_tab[seg];
  const bool last = seg + 1 == p.plan.seq_off[sg.x + 1];
  if (MODE == 1 && last) return;
  const int n = sg.z;
  const E* x = static_cast<const E*>(p.x) + (int64_t)sg.y * p.x_stride + m.d0;
  const E* dt = static_cast<const E*>(p.dt) + (int64_t)sg.y * p.dt_stride + m.d0;
  const E* z = p.z ? static_cast<const E*>(p.z) + (int64_t)sg.y * p.z_stride + m.d0 : nullptr;
  const E* Bm = static_cast<const E*>(p.Bm) + (int64_t)sg.y * p.b_stride + (int64_t)m.group * p.N;
  const E* Cm = static_cast<const E*>(p.Cm) + (int64_t)sg.y * p.c_stride + (int64_t)m.group * p.N;
  E* out = static_cast<E*>(p.out) + (int64_t)sg.y * p.D + m.d0;

  // A group of U tokens' rows into the ring.
  const E *sx = x, *sd = dt, *sz = z;
  int fetched = 0, put = 0, got = 0;
  auto fetch = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = m.live && fetched + u < n;
      ring.copy(put + u, 0, there ? sx : x, there);
      ring.copy(put + u, 1, there ? sd : dt, there);
      if (MODE == 0 && z) ring.copy(put + u, kRows - 1, there ? sz : z, there);
      sx += p.x_stride;
      sd += p.dt_stride;
      sz += p.z_stride;
    }
    fetched += U;
    put = put + U == U * NG ? 0 : put + U;
    ring_commit();
  };
  // B and C of the tile from token t0 on: fetched into registers a tile ahead, stored when the tile before
  // has been used.
  Raw<E, 1> staged[kStage];
  auto fetch_bc = [&](int t0) {
#pragma unroll
    for (int j = 0; j < kStage; ++j) {
      const int i = threadIdx.x + j * kSsmThreads;
      const int k = i % M::kStates, r = i / M::kStates, c = r % kPer;
      const int64_t t = t0 + r / kPer;
      staged[j].zero();
      if (k < p.N && t < n) staged[j].load(c == 0 ? Bm + t * p.b_stride + k : Cm + t * p.c_stride + k);
    }
  };
  auto store_bc = [&](int buf) {
#pragma unroll
    for (int j = 0; j < kStage; ++j) {
      float f[1];
      staged[j].widen(f);
      (&s_bc[buf][0][0][0])[threadIdx.x + j * kSsmThreads] = f[0];
    }
  };

#pragma unroll
  for (int g = 0; g + 1 < NG; ++g) fetch();
  fetch_bc(0);
  float2 h[V][S / 2];
  float* slot = p.pool + p.cache_indices[sg.x] * (int64_t)p.D * p.N;
  if (MODE == 0) {
    // A sequence of one segment starts from the slot itself, which only this thread reads and writes.
    m.load_state(h, sg.w == 0 && last ? slot : p.seg_state + (int64_t)seg * p.D * p.N, p);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < S / 2; ++i) h[v][i] = make_float2(0.f, 0.f);
  }
  float sum_delta[V];
#pragma unroll
  for (int v = 0; v < V; ++v) sum_delta[v] = 0.f;

  store_bc(0);
  __syncthreads();
  for (int t0 = 0, buf = 0; t0 < n; t0 += kTile, buf ^= 1) {
    const bool more = t0 + kTile < n;
    if (more) fetch_bc(t0 + kTile);
    const int tn = min(kTile, n - t0);
    for (int t1 = 0; t1 < tn; t1 += U) {
      // The group's tokens in three steps without a branch inside, so that independent tokens' work overlaps.
      // A token past the end is neutral: delta and u are zero.
      ring_wait<NG - 2>();
      Raw<E, V> rx[U], rz[U];
      float delta[U][V], u[U][V], y[U][V];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t t = t0 + t1 + i;
        rx[i] = ring.read(got + i, 0, x + t * p.x_stride);
        ring.read(got + i, 1, dt + t * p.dt_stride).widen(delta[i]);
        if (MODE == 0 && z) rz[i] = ring.read(got + i, kRows - 1, z + t * p.z_stride);
        add_v<V>(delta[i], bias);
      }
      got = got + U == U * NG ? 0 : got + U;
      fetch();  // into the places read one group ago
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < U; ++i) softplus_of<V>(delta[i]);
      }
      if (t1 + U > tn) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (t1 + i >= tn) delta[i][v] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        rx[i].widen(u[i]);
        mul_v<V>(u[i], delta[i]);
        if (MODE == 1) add_v<V>(sum_delta, delta[i]);
      }
      const float* bt = &s_bc[buf][t1][0][m.lane_p * S];
      constexpr int kRow = kPer * M::kStates;
      if (m.states == S) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          ssm_token<V, S, MODE == 0, false>(y[i], h, A2, bt + i * kRow, bt + i * kRow + M::kStates, delta[i], u[i], S);
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i)
          ssm_token<V, S, MODE == 0, true>(y[i], h, A2, bt + i * kRow, bt + i * kRow + M::kStates, delta[i], u[i], m.states);
      }
      if (MODE == 0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float fx[V];
          rx[i].widen(fx);
#pragma unroll
          for (int v = 0; v < V; ++v)
#pragma unroll
            for (int o = 1; o < P; o <<= 1) y[i][v] += __shfl_xor_sync(0xffffffffu, y[i][v], o);
          fma_v<V>(y[i], skip, fx);
        }
        if (z) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            float fz[V];
            rz[i].widen(fz);
            silu_v<V>(fz);
            mul_v<V>(y[i], fz);
          }
        }
        if (m.live && (P == 1 || m.lane_p == 0)) {
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (t1 + i < tn) store_vec<E, V>(out + (int64_t)(t0 + t1 + i) * p.D, y[i]);
        }
      }
    }
    if (more) store_bc(buf ^ 1);
    __syncthreads();
  }
  ring_wait<0>();
  if (MODE == 0) {
    if (last) m.store_state(slot, h, p);
  } else {
    m.store_state(p.seg_state + (int64_t)seg * p.D * p.N, h, p);
    if (m.live && m.lane_p == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) p.seg_delta[(int64_t)seg * p.D + m.d0 + v] = sum_delta[v];
  }
}

// Start states of the segments of every sequence with more than one: one thread per (sequence, channel,
// state) takes the segments in order. Slot j of seg_state holds segment j's end state from zero until
// its start state replaces it.
__global__ void __launch_bounds__(256) ssm_carry_kernel(SsmParams p) {
  launch_dependents();
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK) return;
  const int64_t per = (int64_t)p.D * p.N;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int j0 = p.plan.seq_off[b], j1 = p.plan.seq_off[b + 1];
    if (j1 - j0 < 2) continue;
    const float* slot = p.pool + p.cache_indices[b] * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < per; i += (int64_t)gridDim.x * 256) {
      const float a = p.A[i] * kLog2e;
      const int64_t d = i / p.N;
      float h = slot[i];
      for (int j = j0; j < j1; j += kCarryBatch) {  // (the last segment's own state is not used)
        float own[kCarryBatch], sum[kCarryBatch];
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          const bool there = j + k + 1 < j1;
          own[k] = there ? p.seg_state[(int64_t)(j + k) * per + i] : 0.f;
          sum[k] = there ? p.seg_delta[(int64_t)(j + k) * p.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          if (j + k < j1) p.seg_state[(int64_t)(j + k) * per + i] = h;
          h = fmaf(ex2(a * sum[k]), h, own[k]);
        }
      }
    }
  }
}

// One token per sequence, states a multiple of 4 with Q = N / 4 a power of two. A warp owns 32 channels
// of one sequence: lane l forms delta and u of channel l, and the 32 Q quads of states go over the lanes
// in the order of memory, so every load and store of states covers 512 consecutive bytes. A lane's quads
// are all of the same states, so it reads B and C once for all channels of a group. BCV: four of them at once.
// Bound by HBM and latency: 256 sequences x 4096 channels x 16 states in bf16 26 us (143 MB, 5.4 TB/s, part of
// it from L2). States are loaded before the batch's slots are checked, and written after.
template <typename E, int Q, bool BCV, int CHECK>
__global__ void __launch_bounds__(kSsmThreads) ssm_step_kernel(SsmParams p, int warps_per_seq) {
  const int lane = threadIdx.x & 31;
  int b, d0;
  split_item((uint64_t)blockIdx.x * (kSsmThreads / 32) + (threadIdx.x >> 5), warps_per_seq, b, d0);
  d0 *= 32;
  const int64_t slot = b < p.B ? p.cache_indices[b] : -1;
  const bool in = slot >= 0 && slot < p.pool_size;
  const int d = d0 + lane;
  const int quads = in ? min(32, p.D - d0) * Q : 0;  // quads of states of this warp's channels
  float4* st = reinterpret_cast<float4*>(p.pool + (slot * (int64_t)p.D + d0) * p.N);
  const float4* A = reinterpret_cast<const float4*>(p.A + (int64_t)d0 * p.N);
  float4 s[Q], a[Q <= 4 ? Q : 1];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    if (i * 32 + lane < quads) {
      s[i] = __ldcs(st + i * 32 + lane);
      if constexpr (Q <= 4) a[i] = __ldg(A + i * 32 + lane);
    }
  }
  float delta = 0.f, xv = 0.f, zv = 0.f, skip = 0.f;
  const bool has = in && d < p.D;
  if (has) {
    xv = elem_to_float(static_cast<const E*>(p.x)[b * p.x_stride + d]);
    delta = elem_to_float(static_cast<const E*>(p.dt)[b * p.dt_stride + d]);
    if (p.dt_bias) delta += p.dt_bias[d];
    if (p.z) zv = elem_to_float(static_cast<const E*>(p.z)[b * p.z_stride + d]);
    if (p.Dskip) skip = p.Dskip[d];
    if (p.softplus) delta = softplus2(make_float2(delta, delta)).x;
  }
  const float dx = delta * xv;
  const int per_group = p.G == 1 ? p.D : p.D / p.G, n = (lane % Q) * 4;
  auto group_of = [&](int ch) { return p.G == 1 ? 0 : ch / per_group; };
  float bq[4], cq[4];
  auto load_bc = [&](int g) {
    const E* Bg = static_cast<const E*>(p.Bm) + b * p.b_stride + (int64_t)g * p.N + n;
    const E* Cg = static_cast<const E*>(p.Cm) + b * p.c_stride + (int64_t)g * p.N + n;
    if constexpr (BCV) {
      load_vec<E, 4>(bq, Bg);
      load_vec<E, 4>(cq, Cg);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) bq[k] = elem_to_float(Bg[k]), cq[k] = elem_to_float(Cg[k]);
    }
  };
  int end = 0;  // the lane's channels before `end` are of the group whose B and C it has
  if (lane < quads) {
    const int g = group_of(d0 + lane / Q);
    end = (g + 1) * per_group;
    load_bc(g);
  }
  if (!step_slots_ok<CHECK>(p.cache_indices, p.B, p.pool_size, p.status) || !in) return;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int f = i * 32 + lane, c = f / Q;  // channel of the warp
    const float dl = __shfl_sync(0xffffffffu, delta, c) * kLog2e, dv = __shfl_sync(0xffffffffu, dx, c);
    float part = 0.f;
    if (f < quads) {
      if (d0 + c >= end) {
        const int g = group_of(d0 + c);
        end = (g + 1) * per_group;
        load_bc(g);
      }
      float4 av;
      if constexpr (Q <= 4) av = a[i]; else av = __ldg(A + f);
      float2 e0 = mul2(both(dl), make_float2(av.x, av.y)), e1 = mul2(both(dl), make_float2(av.z, av.w));
      e0 = make_float2(ex2(e0.x), ex2(e0.y)), e1 = make_float2(ex2(e1.x), ex2(e1.y));
      const float2 h0 = fma2(e0, make_float2(s[i].x, s[i].y), mul2(both(dv), make_float2(bq[0], bq[1])));
      const float2 h1 = fma2(e1, make_float2(s[i].z, s[i].w), mul2(both(dv), make_float2(bq[2], bq[3])));
      const float2 y2 = fma2(h1, make_float2(cq[2], cq[3]), mul2(h0, make_float2(cq[0], cq[1])));
      part = y2.x + y2.y;
      __stcs(st + f, make_float4(h0.x, h0.y, h1.x, h1.y));
    }
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    // Channel c's sum is in its Q lanes now: the lane of its output takes it.
    const float mine = __shfl_sync(0xffffffffu, part, (lane * Q) & 31);
    if (lane * Q / 32 == i) y = mine;
  }
  if (has) {
    y = fmaf(skip, xv, y);
    if (p.z) y *= zv * sigmoid_fast(zv);
    static_cast<E*>(p.out)[(int64_t)b * p.D + d] = float_to_elem<E>(y);
  }
}

// The same for any N and alignment, where quads do not fit: 256 sequences x 4096 channels x 16 states 44 us against the
// quads' 25, of 64 states 209 against 117. The states again go over the lanes in the order of memory, one by one; what
// each adds to its channel's output goes through shared memory, in rows of an odd length, so that a
// lane reads its channel's without conflicts.
template <typename E, int CHECK>
__global__ void __launch_bounds__(kSsmThreads) ssm_step_any_kernel(SsmParams p, int warps_per_seq) {
  constexpr int U = 8;  // states of a lane on their way
  extern __shared__ float s_parts[];
  const int lane = threadIdx.x & 31, N = p.N, pitch = N | 1;
  float* parts = s_parts + (threadIdx.x >> 5) * 32 * pitch;
  int b, d0;
  split_item((uint64_t)blockIdx.x * (kSsmThreads / 32) + (threadIdx.x >> 5), warps_per_seq, b, d0);
  d0 *= 32;
  const int64_t slot = b < p.B ? p.cache_indices[b] : -1;
  // A warp stays inside the pool whatever a verdict that came from a kernel before says.
  if (!step_slots_ok<CHECK>(p.cache_indices, p.B, p.pool_size, p.status) || slot < 0 || slot >= p.pool_size) return;
  const int d = d0 + lane, cells = min(32, p.D - d0) * N;
  const bool has = d < p.D;
  float* st = p.pool + (slot * (int64_t)p.D + d0) * N;
  const float* A = p.A + (int64_t)d0 * N;
  const E* Bm = static_cast<const E*>(p.Bm) + b * p.b_stride;
  const E* Cm = static_cast<const E*>(p.Cm) + b * p.c_stride;
  float xv = 0.f, delta = 0.f;
  if (has) {
    xv = elem_to_float(static_cast<const E*>(p.x)[b * p.x_stride + d]);
    delta = elem_to_float(static_cast<const E*>(p.dt)[b * p.dt_stride + d]) + (p.dt_bias ? p.dt_bias[d] : 0.f);
    if (p.softplus) delta = softplus2(make_float2(delta, delta)).x;
  }
  const float dx = delta * xv, dl = delta * kLog2e;
  const int per_group = p.D / p.G, whole = 32 / N, rest = 32 % N;
  int c = lane / N, n = lane % N;  // channel of the warp and state of the lane's next cell
  for (int f0 = 0; f0 < 32 * N; f0 += 32 * U) {
    float s[U], a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int f = f0 + u * 32 + lane;
      s[u] = f < cells ? __ldcs(st + f) : 0.f;
      a[u] = f < cells ? __ldg(A + f) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int f = f0 + u * 32 + lane;
      const float cl = __shfl_sync(0xffffffffu, dl, c & 31), cx = __shfl_sync(0xffffffffu, dx, c & 31);
      if (f < cells) {
        const int at = (p.G == 1 ? 0 : (d0 + c) / per_group * N) + n;
        const float h = fmaf(ex2(cl * a[u]), s[u], cx * elem_to_float(Bm[at]));
        __stcs(st + f, h);
        parts[c * pitch + n] = h * elem_to_float(Cm[at]);
      }
      c += whole, n += rest;
      if (n >= N) n -= N, ++c;
    }
  }
  __syncwarp();
  if (!has) return;
  float y = 0.f;
#pragma unroll 4
  for (int k = 0; k < N; ++k) y += parts[lane * pitch + k];
  if (p.Dskip) y = fmaf(p.Dskip[d], xv, y);
  if (p.z) {
    const float zv = elem_to_float(static_cast<const E*>(p.z)[b * p.z_stride + d]);
    y *= zv * sigmoid_fast(zv);
  }
  static_cast<E*>(p.out)[(int64_t)b * p.D + d] = float_to_elem<E>(y);
}

template <typename E, int V, int S, int P>
cudaError_t launch_scan_t(const SsmParams& p, bool split, cudaStream_t s, int* kernels) {
  using M = SsmMap<V, S, P>;
  const int per_group = p.D / p.G, bpg = (per_group + M::kChannels - 1) / M::kChannels;
  const dim3 grid((unsigned)(p.max_segs * bpg * p.G)), block(kSsmThreads);
  if (split) {
    if (cudaError_t e = launch_after(ssm_scan_kernel<E, V, S, P, 1>, grid, block, 0, s, p, bpg)) return e;
    const int64_t cells = (int64_t)p.D * p.N;
    const dim3 cgrid((unsigned)(((cells + 255) / 256) < 4096 ? (cells + 255) / 256 : 4096), (unsigned)(p.B < 1024 ? p.B : 1024));
    if (cudaError_t e = launch_after(ssm_carry_kernel, cgrid, dim3(256), 0, s, p)) return e;
    *kernels += 2;
  }
  ++*kernels;
  return launch_after(ssm_scan_kernel<E, V, S, P, 0>, grid, block, 0, s, p, bpg);
}

}  // namespace

// Segments for one round of blocks, two to an SM: the outputs' pass takes 255 registers for four channels a
// thread. Narrower threads with more blocks an SM, and twice the segments in two rounds, were both slower. No
// segment is shorter than 32 tokens, where its start and its share of the carry begin to count; at least 128
// tokens instead changes no call above by more than 1 %.
SegmentRule ssm_segments(int64_t T, int B, int D, int G, int N) {
  const int ch = 4 * kSsmThreads / (N <= 16 ? 1 : N <= 32 ? 2 : 4), per_group = D / G;
  const int64_t blocks = (int64_t)((per_group + ch - 1) / ch) * G, fit = kSmCount * 2;
  return segment_rule(T, B, kSsmUnroll, 32, blocks < fit ? fit / blocks : 1);
}

// Four channels a thread where they load at once, else two or one: 16384 tokens x 4096 channels x 32 states 926 us with
// four, 1013 with two. States in a share that they fill, so that none needs a test: 24 states as 12 on two lanes
// 775 us, as 16 and 8 of 16 1668. (20 on the same lanes, with tests, 1158; 32 take 926, 64 2041.)
cudaError_t launch_ssm_extend(const SsmParams& p, const SegmentRule& rule, cudaStream_t s, int* kernels) {
  const int vec = ssm_vec(p, 4, {p.x, p.dt, p.z, p.out}, {p.x_stride, p.dt_stride, p.z ? p.z_stride : 0});
  const bool split = p.T > rule.least;  // some sequence may have two segments
  return with_elem(p.dtype, [&](auto e) {
    using E = decltype(e);
    auto go = [&](auto sc, auto pc) {
      constexpr int S = decltype(sc)::value, P = decltype(pc)::value;
      if (vec == 4) return launch_scan_t<E, 4, S, P>(p, split, s, kernels);
      return vec >= 2 ? launch_scan_t<E, 2, S, P>(p, split, s, kernels) : launch_scan_t<E, 1, S, P>(p, split, s, kernels);
    };
    using std::integral_constant;
    if (p.N <= 8) return go(integral_constant<int, 8>{}, integral_constant<int, 1>{});
    if (p.N <= 16) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (p.N <= 24) return go(integral_constant<int, 12>{}, integral_constant<int, 2>{});
    if (p.N <= 32) return go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  });
}

cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t s) {
  const bool quads = (p.N == 4 || p.N == 8 || p.N == 16 || p.N == 32 || p.N == 64) && aligned_to(p.pool, 16) && aligned_to(p.A, 16);
  const int wps = (p.D + 31) / 32;
  const int64_t warps = (int64_t)p.B * wps;
  const dim3 grid((unsigned)((warps + kSsmThreads / 32 - 1) / (kSsmThreads / 32))), block(kSsmThreads);
  const size_t parts = (size_t)kSsmThreads * (p.N | 1) * sizeof(float);  // of the kernel for any N
  const int size = op_dtype_size(p.dtype);
  const bool bcv = aligned_to(p.Bm, 4 * size) && aligned_to(p.Cm, 4 * size) && p.b_stride % 4 == 0 && p.c_stride % 4 == 0;
  return with_elem(p.dtype, [&](auto e) {
    using E = decltype(e);
    return with_check(p.check, [&](auto check) {
      constexpr int IN = decltype(check)::value;
      auto launch = [&](auto* kernel, size_t smem) {
        if (IN == kCheckBefore) return launch_after(kernel, grid, block, smem, s, p, wps);
        kernel<<<grid, block, smem, s>>>(p, wps);
        return cudaGetLastError();
      };
      if (!quads) return launch(ssm_step_any_kernel<E, IN>, parts);
      auto q = [&](auto qc) {
        constexpr int Q = decltype(qc)::value;
        return bcv ? launch(ssm_step_kernel<E, Q, true, IN>, 0) : launch(ssm_step_kernel<E, Q, false, IN>, 0);
      };
      using std::integral_constant;
      switch (p.N) {
        case 4: return q(integral_constant<int, 1>{});
        case 8: return q(integral_constant<int, 2>{});
        case 16: return q(integral_constant<int, 4>{});
        case 32: return q(integral_constant<int, 8>{});
        default: return q(integral_constant<int, 16>{});
      }
    });
  });
}

}  // namespace gdn
