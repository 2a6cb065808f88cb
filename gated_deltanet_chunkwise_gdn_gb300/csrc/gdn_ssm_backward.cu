// gdn_ssm_backward.cu — gradients of the selective scan (gdn_ssm.cu) for the gradients of its outputs and
// of its final states. With dy the gradient of y (d_out z sigmoid(z), or d_out), u = delta x,
// a_n = exp(delta A_n) and g_n the gradient at h_n of a token, per channel:
//
//   g_n     = dy C_n + (a_n g_n of the next token; d_state at the last)
//   dC_n    = sum over the group's channels of dy h_n         dB_n = ... of g_n u
//   du      = sum_n g_n B_n,     q_n = a_n g_n h_n(before),   w = sum_n q_n A_n
//   dx      = Dskip dy + delta du,   ddt = (x du + w) softplus'(dt + dt_bias)
//   dz      = d_out y silu'(z),  dA_n = sum_t delta q_n,  dDskip = sum_t dy x,  d dt_bias = sum_t ddt
//   d h_0   = a g of the first token
//
// Every sequence is cut into segments, which run side by side:
//   1. ssm_bwd_local_kernel, forward over a segment from a zero state: the end state, the sum of deltas,
//      the gradient that leaves the segment backwards from its own tokens (sum_t exp(A sum_{s<=t} delta_s)
//      dy_t C_t), and the state at every kChunk-th token.
//   2. ssm_bwd_carry_kernel: start states in order, incoming gradients in reverse order, d_state_pool.
//   3. ssm_bwd_main_kernel: the chunks of a segment from its last: the states of a chunk forward from its
//      checkpoint into shared memory, then the chunk backwards.
//   4. ssm_bwd_sum_kernel: dB and dC over the channel blocks, the parameters' gradients over the segments.
// All sums are taken in a fixed order.
//
// The passes are bound by instruction latency and the shared-memory pipe: about 19 operations and 3
// exponentials a state and token, issued in 0.54 of the cycles by 2.7 warps a scheduler, with 0.57 of the
// shared-memory pipe's rate. 3 x 4096 tokens x 2048 channels x 16 states in bf16: local 207 us, main 589, carry
// 12, sum 16 (the rows' bytes alone would take 45). The layout is chosen for the arithmetic: a thread owns CPT channels
// x S states, B and C come as broadcasts from shared memory, sums over states take few shuffles (each lane ends up with
// one channel's sum), and sums over channels are first taken inside the thread in fp32 and then by one tensor-core
// product with a matrix of ones. tf32 holds 11 bits, so a thread's sum goes in as its upper 11 bits and the next 11: the
// last two of fp32's 24 are dropped, an error of at most 2^-22 of a thread's sum, for every type. Where a third product
// would keep them, it would cost as much as either of the two; the sum's own order already moves results by that much.
//
// Where the states do not fill their lanes, an infinite input or output gradient can leave NaN, where the formulas have an
// infinity, in the gradients of its own channel: a padded state multiplies it by zero.
#include "gdn_ssm.cuh"

namespace gdn {

namespace {

constexpr int kChunk = kSsmChunk;  // tokens whose states are in shared memory
constexpr int kWarps = kSsmThreads / 32;

// CPT channels and S states a thread, NL lanes for a channel's states: lane = state lane * CL + channel lane.
template <int CPT_, int S_, int NL_>
struct BwdMap {
  static constexpr int CPT = CPT_, S = S_, NL = NL_;
  static constexpr int CL = 32 / NL;             // channel lanes
  static constexpr int CW = CL * CPT;            // channels of a warp
  static constexpr int kChannels = CW * kWarps;  // of a block
  static constexpr int kStates = S * NL;
  // Blocks on an SM: 168 registers a thread allow three. 3 x 4096 tokens x 2048 channels x 16 states in bf16, forward and
  // backward, take 1040 us with three, 1146 with two. (Four would leave a thread two channels: slower too.) Shared
  // memory allows three up to 8 states, and up to 32 for 16-bit rows read in pairs (sizeof(MainSmem) 54 to 76 KB).
  // For fp32 and for single 16-bit columns it is 92160 bytes with 9 to 16 states and 77824 with 17 to 32, and above 32
  // states 81920 to 86016 for every type: two blocks fit, while the segments are still cut for three.
  static constexpr int kBlocks = 3;
  static_assert(CL >= 4, "the product with ones takes four lanes of one state lane at a time");
};

// Token and channel rows of one warp's chunk: each lane holds IT rows' VEC neighbouring channels.
template <typename M, int VEC>
struct RowMap {
  static constexpr int LPR = M::CW / VEC;  // lanes of a row
  static constexpr int RP = 32 / LPR;      // rows at a time
  static constexpr int IT = kChunk / RP;
  static_assert(LPR <= 32 && RP <= kChunk, "a warp's rows");
};

// The rows x, dt, z and d_out of chunks on their way: two chunks' worth, each lane its own elements.
template <typename E, typename M, int VEC>
using ChunkRing = RowRing<E, VEC, 4, 2 * RowMap<M, VEC>::IT, kSsmThreads, true>;
enum ChunkArray { kRowX = 0, kRowDt = 1, kRowZ = 2, kRowDy = 3 };

// Column d of token `at` of an array.
template <typename E>
__device__ __forceinline__ const E* row_of(const SsmParams& p, int array, int64_t at, int d) {
  switch (array) {
    case kRowX: return static_cast<const E*>(p.x) + at * p.x_stride + d;
    case kRowDt: return static_cast<const E*>(p.dt) + at * p.dt_stride + d;
    case kRowZ: return static_cast<const E*>(p.z) + at * p.z_stride + d;
    default: return static_cast<const E*>(p.d_out) + at * p.d_stride + d;
  }
}

// Rows t0 .. t0 + kChunk - 1 of a segment of n tokens into the chunk's half of the ring (zeros outside).
template <typename E, typename M, int VEC>
__device__ __forceinline__ void fetch_rows(ChunkRing<E, M, VEC>& ring, const SsmParams& p, int64_t first, int t0, int n,
                                           int row, int d, bool in) {
  using R = RowMap<M, VEC>;
  const int half = t0 / kChunk % 2 * R::IT;
#pragma unroll
  for (int i = 0; i < R::IT; ++i) {
    const int t = t0 + row + i * R::RP;
    const bool there = in && t < n;
    const int64_t at = there ? first + t : 0;
    const int col = there ? d : 0;
    ring.copy(half + i, kRowX, row_of<E>(p, kRowX, at, col), there);
    ring.copy(half + i, kRowDt, row_of<E>(p, kRowDt, at, col), there);
    ring.copy(half + i, kRowDy, row_of<E>(p, kRowDy, at, col), there);
    if (p.z) ring.copy(half + i, kRowZ, row_of<E>(p, kRowZ, at, col), there);
  }
  ring_commit();
}

// delta, u = delta x and dy of a warp's chunk, [token][channel of the block].
template <int CH>
struct ChunkScalars {
  float delta[kChunk][CH], u[kChunk][CH], dy[kChunk][CH];
};

// Fills delta, u and dy from the rows; zeros (neutral: a = 1, nothing added) past the segment's tokens.
template <typename E, typename M, int VEC>
__device__ __forceinline__ void fill_scalars(ChunkScalars<M::kChannels>& sc, const ChunkRing<E, M, VEC>& ring,
                                             const SsmParams& p, const float (&bias)[VEC], int64_t first, int t0, int n,
                                             int row, int c, int d, bool in) {
  using R = RowMap<M, VEC>;
  const int half = t0 / kChunk % 2 * R::IT;
#pragma unroll
  for (int i = 0; i < R::IT; ++i) {
    const int t = row + i * R::RP;
    float fx[VEC], fd[VEC], fz[VEC], fo[VEC];
    ring.read(half + i, kRowX, row_of<E>(p, kRowX, first + t0 + t, d)).widen(fx);
    ring.read(half + i, kRowDt, row_of<E>(p, kRowDt, first + t0 + t, d)).widen(fd);
    ring.read(half + i, kRowDy, row_of<E>(p, kRowDy, first + t0 + t, d)).widen(fo);
    if (p.z) ring.read(half + i, kRowZ, row_of<E>(p, kRowZ, first + t0 + t, d)).widen(fz);
#pragma unroll
    for (int v = 0; v < VEC; ++v) fd[v] += bias[v];
    if (p.softplus) softplus_of<VEC>(fd);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float delta = in && t0 + t < n ? fd[v] : 0.f;
      if (p.z) fo[v] *= fz[v] * sigmoid_fast(fz[v]);
      sc.delta[t][c + v] = delta;
      sc.u[t][c + v] = delta * fx[v];
      sc.dy[t][c + v] = fo[v];
    }
  }
}

template <int K>
__device__ __forceinline__ void load_shared(float (&f)[K], const float* s) {
  if constexpr (K % 4 == 0) {
#pragma unroll
    for (int i = 0; i < K / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(s)[i];
      f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < K / 2; ++i) {
      const float2 q = reinterpret_cast<const float2*>(s)[i];
      f[2 * i] = q.x, f[2 * i + 1] = q.y;
    }
  }
}

// B and C of kChunk tokens, widened; zeros past the segment's tokens and the real states. Fetched into
// registers a chunk ahead and stored once the chunk before has been used.
template <typename E, typename M>
struct ChunkBC {
  static constexpr int kEach = kChunk * 2 * M::kStates / kSsmThreads;
  Raw<E, 1> r[kEach];
  __device__ __forceinline__ void fetch(const SsmParams& p, int64_t first, int t0, int n, int group) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = threadIdx.x + i * kSsmThreads, k = at % M::kStates, q = at / M::kStates, t = t0 + (q >> 1);
      r[i].zero();
      if (k < p.N && t < n) {
        const int64_t col = (int64_t)group * p.N + k;
        r[i].load((q & 1) ? static_cast<const E*>(p.Cm) + (first + t) * p.c_stride + col
                          : static_cast<const E*>(p.Bm) + (first + t) * p.b_stride + col);
      }
    }
  }
  __device__ __forceinline__ void store(float (*bc)[2][M::kStates]) const {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      float f[1];
      r[i].widen(f);
      (&bc[0][0][0])[threadIdx.x + i * kSsmThreads] = f[0];
    }
  }
};

// This thread's CPT channels x S states of an array [D, N] as pairs of states; a vector load where the
// rows allow it.
template <typename M>
struct StateTile {
  int64_t at[M::CPT];  // offset of the first state of each channel, -1 outside the group
  int states;          // real states of this lane
  bool vec;            // four states at a time

  __device__ __forceinline__ StateTile(const SsmParams& p, int group, int c0, int nl) {
    const int per_group = p.D / p.G;
#pragma unroll
    for (int i = 0; i < M::CPT; ++i)
      at[i] = c0 + i < per_group ? ((int64_t)group * per_group + c0 + i) * p.N + nl * M::S : -1;
    const int left = p.N - nl * M::S;
    states = left < 0 ? 0 : (left > M::S ? M::S : left);
    vec = states == M::S && p.N % 4 == 0;
  }
  template <bool GUARD_ALIGN = false>
  __device__ __forceinline__ void load(float2 (&f)[M::CPT][M::S / 2], const float* base) const {
#pragma unroll
    for (int i = 0; i < M::CPT; ++i) {
      const float* q = base + at[i];
      if (at[i] >= 0 && vec && !GUARD_ALIGN) {
#pragma unroll
        for (int j = 0; j < M::S / 4; ++j) {
          const float4 x = reinterpret_cast<const float4*>(q)[j];
          f[i][2 * j] = make_float2(x.x, x.y);
          f[i][2 * j + 1] = make_float2(x.z, x.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < M::S / 2; ++j) {
          f[i][j].x = at[i] >= 0 && 2 * j < states ? q[2 * j] : 0.f;
          f[i][j].y = at[i] >= 0 && 2 * j + 1 < states ? q[2 * j + 1] : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void store(float* base, const float2 (&f)[M::CPT][M::S / 2]) const {
#pragma unroll
    for (int i = 0; i < M::CPT; ++i) {
      float* q = base + at[i];
      if (at[i] < 0) continue;
      if (vec) {
#pragma unroll
        for (int j = 0; j < M::S / 4; ++j)
          reinterpret_cast<float4*>(q)[j] = make_float4(f[i][2 * j].x, f[i][2 * j].y, f[i][2 * j + 1].x, f[i][2 * j + 1].y);
      } else {
#pragma unroll
        for (int j = 0; j < M::S / 2; ++j) {
          if (2 * j < states) q[2 * j] = f[i][j].x;
          if (2 * j + 1 < states) q[2 * j + 1] = f[i][j].y;
        }
      }
    }
  }
};

// Index of a segment's chunk in the checkpoint arrays: distinct for every chunk of the batch, since a
// segment of n tokens has at most n / kChunk + 1 of them.
__device__ __forceinline__ int64_t chunk_index(const int4& sg, int seg, int c) { return sg.y / kChunk + seg + c; }

template <typename E, typename M, int VEC>
__global__ void __launch_bounds__(kSsmThreads, M::kBlocks) ssm_bwd_local_kernel(SsmParams p, int blocks_per_group) {
  using R = RowMap<M, VEC>;
  constexpr int S2 = M::S / 2;
  __shared__ __align__(16) ChunkScalars<M::kChannels> sc;
  __shared__ __align__(16) float s_bc[2][kChunk][2][M::kStates];
  __shared__ ChunkRing<E, M, VEC> ring;
  launch_dependents();
  const int nblk = blocks_per_group * p.G;
  const int seg = blockIdx.x / nblk, blk = blockIdx.x % nblk, group = blk / blocks_per_group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cb = (blk % blocks_per_group) * M::kChannels;  // the block's first channel in its group
  const int nl = lane / M::CL, cl = lane % M::CL;
  const int c_own = warp * M::CW + cl * M::CPT;
  const StateTile<M> tile(p, group, cb + c_own, nl);
  const int row = lane / R::LPR, c_row = warp * M::CW + (lane % R::LPR) * VEC;
  const int per_group = p.D / p.G;
  const bool in = cb + c_row < per_group;  // per_group is a multiple of VEC
  const int d_row = group * per_group + cb + c_row;
  float bias[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) bias[v] = p.dt_bias && in ? p.dt_bias[d_row + v] : 0.f;
  float2 A2[M::CPT][S2];
  tile.template load<true>(A2, p.A);
#pragma unroll
  for (int i = 0; i < M::CPT; ++i)
#pragma unroll
    for (int j = 0; j < S2; ++j) A2[i][j].x *= kLog2e, A2[i][j].y *= kLog2e;
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK || seg >= p.plan.status[1]) return;
  const int4 sg = p.plan.seg_tab[seg];
  const int n = sg.z, chunks = (n + kChunk - 1) / kChunk;
  const int64_t cells = (int64_t)p.D * p.N;

  float2 h[M::CPT][S2], gr[M::CPT][S2];
  float sum[M::CPT];
#pragma unroll
  for (int i = 0; i < M::CPT; ++i) {
    sum[i] = 0.f;
#pragma unroll
    for (int j = 0; j < S2; ++j) h[i][j] = gr[i][j] = both(0.f);
  }
  fetch_rows<E, M, VEC>(ring, p, sg.y, 0, n, row, d_row, in);
  ChunkBC<E, M> bc;
  bc.fetch(p, sg.y, 0, n, group);
  bc.store(s_bc[0]);
  __syncthreads();
  for (int c = 0; c < chunks; ++c) {
    const int t0 = c * kChunk;
    if (c + 1 < chunks) {
      fetch_rows<E, M, VEC>(ring, p, sg.y, t0 + kChunk, n, row, d_row, in);
      bc.fetch(p, sg.y, t0 + kChunk, n, group);
      ring_wait<1>();
    } else {
      ring_wait<0>();
    }
    fill_scalars<E, M, VEC>(sc, ring, p, bias, sg.y, t0, n, row, c_row, d_row, in);
    if (c > 0) {  // the state entering this chunk, from the segment's own tokens
      const int64_t at = chunk_index(sg, seg, c);
      tile.store(p.ckpt + at * cells, h);
      if (nl == 0)
#pragma unroll
        for (int i = 0; i < M::CPT; ++i)
          if (cb + c_own + i < per_group) p.ckpt_delta[at * p.D + group * per_group + cb + c_own + i] = sum[i];
    }
    __syncwarp();
#pragma unroll 4
    for (int t = 0; t < kChunk; ++t) {
      float dl[M::CPT], u[M::CPT], dy[M::CPT], Bt[M::S], Ct[M::S];
      load_shared<M::CPT>(dl, &sc.delta[t][c_own]);
      load_shared<M::CPT>(u, &sc.u[t][c_own]);
      load_shared<M::CPT>(dy, &sc.dy[t][c_own]);
      load_shared<M::S>(Bt, &s_bc[c & 1][t][0][nl * M::S]);
      load_shared<M::S>(Ct, &s_bc[c & 1][t][1][nl * M::S]);
#pragma unroll
      for (int i = 0; i < M::CPT; ++i) {
        sum[i] += dl[i];
#pragma unroll
        for (int j = 0; j < S2; ++j) {
          float2 e = mul2(make_float2(dl[i], dl[i]), A2[i][j]);
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          h[i][j] = fma2(e, h[i][j], mul2(make_float2(u[i], u[i]), make_float2(Bt[2 * j], Bt[2 * j + 1])));
          // The decay back to the segment's start from the sum of deltas: a product of the tokens' decays
          // would add up their rounding errors.
          float2 back = mul2(both(sum[i]), A2[i][j]);
          back.x = ex2(back.x);
          back.y = ex2(back.y);
          gr[i][j] = fma2(back, mul2(both(dy[i]), make_float2(Ct[2 * j], Ct[2 * j + 1])), gr[i][j]);
        }
      }
    }
    if (c + 1 < chunks) bc.store(s_bc[(c + 1) & 1]);
    __syncthreads();
  }
  tile.store(p.seg_state + (int64_t)seg * cells, h);
  tile.store(p.seg_grad + (int64_t)seg * cells, gr);
  if (nl == 0)
#pragma unroll
    for (int i = 0; i < M::CPT; ++i)
      if (cb + c_own + i < per_group) p.seg_delta[(int64_t)seg * p.D + group * per_group + cb + c_own + i] = sum[i];
}

// One thread per (sequence, channel, state): the segments' start states in order, then the gradients that
// enter their last states in reverse order; both replace the local values. What leaves the first segment
// is the gradient of the initial state; a sequence without tokens passes its own through.
__global__ void __launch_bounds__(256) ssm_bwd_carry_kernel(SsmParams p) {
  launch_dependents();
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK) return;
  const int64_t per = (int64_t)p.D * p.N;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int j0 = p.plan.seq_off[b], j1 = p.plan.seq_off[b + 1];
    const int64_t slot = p.cache_indices[b] * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < per; i += (int64_t)gridDim.x * 256) {
      const float a = p.A[i] * kLog2e;
      const int64_t d = i / p.N;
      float h = p.pool[slot + i], g = p.d_state ? p.d_state[slot + i] : 0.f;
      for (int j = j0; j < j1; j += kCarryBatch) {
        float own[kCarryBatch], sum[kCarryBatch];
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          const bool there = j + k < j1;
          own[k] = there ? p.seg_state[(int64_t)(j + k) * per + i] : 0.f;
          sum[k] = there ? p.seg_delta[(int64_t)(j + k) * p.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          if (j + k < j1) p.seg_state[(int64_t)(j + k) * per + i] = h;
          h = fmaf(ex2(a * sum[k]), h, own[k]);
        }
      }
      for (int j = j1 - 1; j >= j0; j -= kCarryBatch) {
        float own[kCarryBatch], sum[kCarryBatch];
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          const bool there = j - k >= j0;
          own[k] = there ? p.seg_grad[(int64_t)(j - k) * per + i] : 0.f;
          sum[k] = there ? p.seg_delta[(int64_t)(j - k) * p.D + d] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kCarryBatch; ++k) {
          if (j - k >= j0) {
            p.seg_grad[(int64_t)(j - k) * per + i] = g;
            g = fmaf(ex2(a * sum[k]), g, own[k]);
          }
        }
      }
      p.d_pool[slot + i] = g;
    }
  }
}

// Sums v[0 .. CPT-1] over the NL state lanes; state lane i ends up with the sum of channel i's where CPT >=
// NL (of channel i % CPT, the same in NL / CPT lanes, otherwise). Each step sends half of what is left.
template <typename M>
__device__ __forceinline__ float sum_states(float (&v)[M::CPT], int nl) {
  constexpr int CPT = M::CPT;
  int left = CPT;
#pragma unroll
  for (int o = 1; o < M::NL; o <<= 1) {
    if (left > 1) {
      const bool up = nl & o;
#pragma unroll
      for (int i = 0; i < CPT / 2; ++i)
        if (i < left / 2) {
          // channels are split by their lowest remaining bit, which becomes this lane bit
          const float keep = up ? v[2 * i + 1] : v[2 * i], send = up ? v[2 * i] : v[2 * i + 1];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o * M::CL);
        }
      left /= 2;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * M::CL);
    }
  }
  return v[0];
}

// D += [a0 a1; a0 a1] x [hi; lo]: rows r and r + 8 of the 16 x 8 accumulator get, scaled by a0 and a1, the
// sum over the four lanes of each column of hi + lo.
__device__ __forceinline__ void add_ones_product(float (&d)[4], uint32_t a0, uint32_t a1, float v) {
  const uint32_t hi = __float_as_uint(v) & 0xffffe000u;
  const uint32_t lo = __float_as_uint(v - __uint_as_float(hi));
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %4, %5}, {%6, %7}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(hi), "r"(lo));
}

// The same sum of v into row t, by shuffles: the first column of each state lane's gets all of it.
template <typename M>
__device__ __forceinline__ void add_shuffled(float& even, float& odd, float v, int t, int lane) {
  constexpr int kGroups = M::CL / 4;
#pragma unroll
  for (int o = 1; o < M::CL; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = (lane & 3) * 2;
  const float a = __shfl_sync(0xffffffffu, v, col / kGroups * M::CL);
  const float b = __shfl_sync(0xffffffffu, v, (col + 1) / kGroups * M::CL);
  if ((lane >> 2) == t) {
    if (col % kGroups == 0) even += a;
    if ((col + 1) % kGroups == 0) odd += b;
  }
}

template <typename E, typename M, int VEC>
struct MainSmem {
  ChunkScalars<M::kChannels> sc;
  float y[kChunk][M::kChannels];
  float bc[2][kChunk][2][M::kStates];
  float red[2][kWarps][kChunk][2][M::kStates];
  float4 h[kChunk / 2][M::CPT * M::S / 4][kSsmThreads];  // h[k]: the state before token 2 k, by its thread
  ChunkRing<E, M, VEC> ring;
};

template <typename E, typename M, int VEC>
__global__ void __launch_bounds__(kSsmThreads, M::kBlocks) ssm_bwd_main_kernel(SsmParams p, int blocks_per_group) {
  using R = RowMap<M, VEC>;
  constexpr int CPT = M::CPT, S = M::S, S2 = M::S / 2;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using Smem = MainSmem<E, M, VEC>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  launch_dependents();
  const int nblk = blocks_per_group * p.G;
  const int seg = blockIdx.x / nblk, blk = blockIdx.x % nblk, group = blk / blocks_per_group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cb = (blk % blocks_per_group) * M::kChannels;
  const int nl = lane / M::CL, cl = lane % M::CL;
  const int c_own = warp * M::CW + cl * CPT;
  const StateTile<M> tile(p, group, cb + c_own, nl);
  const int row = lane / R::LPR, c_row = warp * M::CW + (lane % R::LPR) * VEC;
  const int per_group = p.D / p.G;
  const bool in = cb + c_row < per_group;
  const int d_row = group * per_group + cb + c_row;
  float bias[VEC], skip[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    bias[v] = p.dt_bias && in ? p.dt_bias[d_row + v] : 0.f;
    skip[v] = p.Dskip && in ? p.Dskip[d_row + v] : 0.f;
  }
  float2 A2[CPT][S2];
  tile.template load<true>(A2, p.A);
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int j = 0; j < S2; ++j) A2[i][j].x *= kLog2e, A2[i][j].y *= kLog2e;
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK || seg >= p.plan.status[1]) return;
  const int4 sg = p.plan.seg_tab[seg];
  const int n = sg.z, chunks = (n + kChunk - 1) / kChunk;
  const int64_t cells = (int64_t)p.D * p.N;

  float2 gr[CPT][S2], dA[CPT][S2];
  tile.load(gr, p.seg_grad + (int64_t)seg * cells);
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int j = 0; j < S2; ++j) dA[i][j] = make_float2(0.f, 0.f);
  float dskip[VEC], dbias[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) dskip[v] = dbias[v] = 0.f;

  fetch_rows<E, M, VEC>(sm.ring, p, sg.y, (chunks - 1) * kChunk, n, row, d_row, in);
  ChunkBC<E, M> bc;
  bc.fetch(p, sg.y, (chunks - 1) * kChunk, n, group);
  bc.store(sm.bc[(chunks - 1) & 1]);
  __syncthreads();
  for (int c = chunks - 1; c >= 0; --c) {
    const int t0 = c * kChunk;
    // The state before the chunk: what is left of the segment's start state, and what the segment's earlier
    // tokens leave.
    float2 h[CPT][S2];
    tile.load(h, p.seg_state + (int64_t)seg * cells);
    if (c > 0) {
      const int64_t at = chunk_index(sg, seg, c);
      float2 left[CPT][S2];
      tile.load(left, p.ckpt + at * cells);
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        const float since = tile.at[i] >= 0 ? p.ckpt_delta[at * p.D + group * per_group + cb + c_own + i] : 0.f;
#pragma unroll
        for (int j = 0; j < S2; ++j) {
          float2 e = mul2(both(since), A2[i][j]);
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          h[i][j] = fma2(e, h[i][j], left[i][j]);
        }
      }
      if (c > 1) {  // the next chunk's, into L2
#pragma unroll
        for (int i = 0; i < CPT; ++i)
          if (tile.at[i] >= 0) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.ckpt + (at - 1) * cells + tile.at[i]));
      }
    }
    if (c > 0) {
      fetch_rows<E, M, VEC>(sm.ring, p, sg.y, t0 - kChunk, n, row, d_row, in);
      bc.fetch(p, sg.y, t0 - kChunk, n, group);
      ring_wait<1>();
    } else {
      ring_wait<0>();
    }
    fill_scalars<E, M, VEC>(sm.sc, sm.ring, p, bias, sg.y, t0, n, row, c_row, d_row, in);
    __syncwarp();
    // The chunk's states, forward.
#pragma unroll 4
    for (int t = 0; t < kChunk; ++t) {
      float dl[CPT], u[CPT], Bt[S], Ct[S], y[CPT];
      load_shared<CPT>(dl, &sm.sc.delta[t][c_own]);
      load_shared<CPT>(u, &sm.sc.u[t][c_own]);
      load_shared<S>(Bt, &sm.bc[c & 1][t][0][nl * S]);
      load_shared<S>(Ct, &sm.bc[c & 1][t][1][nl * S]);
      if (t % 2 == 0) {
#pragma unroll
        for (int k = 0; k < CPT * S / 4; ++k) {
          const int i = k / (S / 4), j = k % (S / 4) * 2;
          sm.h[t / 2][k][threadIdx.x] = make_float4(h[i][j].x, h[i][j].y, h[i][j + 1].x, h[i][j + 1].y);
        }
      }
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < S2; ++j) {
          float2 e = mul2(make_float2(dl[i], dl[i]), A2[i][j]);
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          h[i][j] = fma2(e, h[i][j], mul2(make_float2(u[i], u[i]), make_float2(Bt[2 * j], Bt[2 * j + 1])));
          y2 = fma2(h[i][j], make_float2(Ct[2 * j], Ct[2 * j + 1]), y2);
        }
        y[i] = y2.x + y2.y;
      }
      if (p.z) {
        const float mine = sum_states<M>(y, nl);
        if (nl < CPT) sm.y[t][c_own + nl] = mine;
      }
    }
    // The chunk backwards; h is the state after token t.
    float acc[S][4];
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;
    // Token t, with the state after it in h and the one before it from before(channel, quad).
    auto token_back = [&](int t, auto&& before_of) {
      float dl[CPT], u[CPT], dy[CPT], Bt[S], Ct[S], du[CPT], w[CPT];
      float2 dB[S2], dC[S2];
      load_shared<CPT>(dl, &sm.sc.delta[t][c_own]);
      load_shared<CPT>(u, &sm.sc.u[t][c_own]);
      load_shared<CPT>(dy, &sm.sc.dy[t][c_own]);
      load_shared<S>(Bt, &sm.bc[c & 1][t][0][nl * S]);
      load_shared<S>(Ct, &sm.bc[c & 1][t][1][nl * S]);
#pragma unroll
      for (int j = 0; j < S2; ++j) dB[j] = dC[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < CPT; ++i) {
        float2 du2 = make_float2(0.f, 0.f), w2 = make_float2(0.f, 0.f);
        const float2 dl2 = make_float2(dl[i], dl[i]), u2 = make_float2(u[i], u[i]), dy2 = make_float2(dy[i], dy[i]);
#pragma unroll
        for (int k = 0; k < S / 4; ++k) {
          const float4 before = before_of(i, k);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int j = 2 * k + m;
            const float2 hb = m == 0 ? make_float2(before.x, before.y) : make_float2(before.z, before.w);
            const float2 g = fma2(dy2, make_float2(Ct[2 * j], Ct[2 * j + 1]), gr[i][j]);
            dC[j] = fma2(dy2, h[i][j], dC[j]);
            dB[j] = fma2(u2, g, dB[j]);
            du2 = fma2(g, make_float2(Bt[2 * j], Bt[2 * j + 1]), du2);
            float2 e = mul2(dl2, A2[i][j]);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            gr[i][j] = mul2(g, e);
            const float2 q = mul2(gr[i][j], hb);
            w2 = fma2(q, A2[i][j], w2);
            dA[i][j] = fma2(dl2, q, dA[i][j]);
            h[i][j] = hb;
          }
        }
        du[i] = du2.x + du2.y;
        w[i] = w2.x + w2.y;
      }
      // An infinite or NaN sum would reach the other tokens' rows as its product with zero, so such a
      // token takes the shuffles instead.
      float2 odd = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < S2; ++j) odd = fma2(dB[j], make_float2(0.f, 0.f), fma2(dC[j], make_float2(0.f, 0.f), odd));
      if (__any_sync(0xffffffffu, !(odd.x + odd.y == 0.f))) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          add_shuffled<M>(acc[j][0], acc[j][1], j % 2 ? dB[j / 2].y : dB[j / 2].x, t, lane);
          add_shuffled<M>(acc[j][2], acc[j][3], j % 2 ? dC[j / 2].y : dC[j / 2].x, t, lane);
        }
      } else {
        const uint32_t one = (lane >> 2) == t ? 0x3f800000u : 0u;  // 1.0 in the accumulator's row t
#pragma unroll
        for (int j = 0; j < S2; ++j) {
          add_ones_product(acc[2 * j], one, 0u, dB[j].x);
          add_ones_product(acc[2 * j + 1], one, 0u, dB[j].y);
          add_ones_product(acc[2 * j], 0u, one, dC[j].x);
          add_ones_product(acc[2 * j + 1], 0u, one, dC[j].y);
        }
      }
      const float du_mine = sum_states<M>(du, nl), w_mine = sum_states<M>(w, nl);
      __syncwarp();
      if (nl < CPT) {  // in the place of u and dy, which every lane has read
        sm.sc.u[t][c_own + nl] = du_mine;
        sm.sc.dy[t][c_own + nl] = w_mine * (1.f / kLog2e);
      }
    };
#pragma unroll 1
    for (int t = kChunk - 2; t >= 0; t -= 2) {
      // Two tokens at a time: the state between them again from the one before both.
      float2 mid[CPT][S2];
      {
        float dl[CPT], u[CPT], Bt[S];
        load_shared<CPT>(dl, &sm.sc.delta[t][c_own]);
        load_shared<CPT>(u, &sm.sc.u[t][c_own]);
        load_shared<S>(Bt, &sm.bc[c & 1][t][0][nl * S]);
#pragma unroll
        for (int i = 0; i < CPT; ++i)
#pragma unroll
          for (int k = 0; k < S / 4; ++k) {
            const float4 q = sm.h[t / 2][i * (S / 4) + k][threadIdx.x];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const int j = 2 * k + m;
              float2 e = mul2(both(dl[i]), A2[i][j]);
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              mid[i][j] = fma2(e, m == 0 ? make_float2(q.x, q.y) : make_float2(q.z, q.w),
                               mul2(both(u[i]), make_float2(Bt[2 * j], Bt[2 * j + 1])));
            }
          }
      }
      token_back(t + 1, [&](int i, int k) {
        return make_float4(mid[i][2 * k].x, mid[i][2 * k].y, mid[i][2 * k + 1].x, mid[i][2 * k + 1].y);
      });
      token_back(t, [&](int i, int k) { return sm.h[t / 2][i * (S / 4) + k][threadIdx.x]; });
    }
    __syncwarp();
    if (c > 0) bc.store(sm.bc[(c - 1) & 1]);
    // dx, ddt and dz of this warp's rows.
    const int half = c % 2 * R::IT;
#pragma unroll
    for (int i = 0; i < R::IT; ++i) {
      const int t = row + i * R::RP;
      if (in && t0 + t < n) {
        float fx[VEC], fd[VEC], fz[VEC], fo[VEC], dx[VEC], ddt[VEC], dz[VEC];
        sm.ring.read(half + i, kRowX, row_of<E>(p, kRowX, sg.y + t0 + t, d_row)).widen(fx);
        sm.ring.read(half + i, kRowDt, row_of<E>(p, kRowDt, sg.y + t0 + t, d_row)).widen(fd);
        sm.ring.read(half + i, kRowDy, row_of<E>(p, kRowDy, sg.y + t0 + t, d_row)).widen(fo);
        if (p.z) sm.ring.read(half + i, kRowZ, row_of<E>(p, kRowZ, sg.y + t0 + t, d_row)).widen(fz);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float du = sm.sc.u[t][c_row + v], w = sm.sc.dy[t][c_row + v], delta = sm.sc.delta[t][c_row + v];
          float dy = fo[v];
          if (p.z) {
            const float sig = sigmoid_fast(fz[v]);
            const float y = fmaf(skip[v], fx[v], sm.y[t][c_row + v]);
            dz[v] = dy * y * sig * fmaf(fz[v], 1.f - sig, 1.f);
            dy *= fz[v] * sig;
          }
          dx[v] = fmaf(skip[v], dy, delta * du);
          ddt[v] = fmaf(fx[v], du, w);
          if (p.softplus) ddt[v] *= sigmoid_fast(fd[v] + bias[v]);
          dskip[v] = fmaf(dy, fx[v], dskip[v]);
          dbias[v] += ddt[v];
        }
        const int64_t at = ((int64_t)sg.y + t0 + t) * p.D + d_row;
        store_vec<E, VEC>(static_cast<E*>(p.dx) + at, dx);
        store_vec<E, VEC>(static_cast<E*>(p.ddt) + at, ddt);
        if (p.z) store_vec<E, VEC>(static_cast<E*>(p.dz) + at, dz);
      }
    }
    // dB and dC of the block's channels. Accumulator row: the token, 8 + the token for dC; column: four
    // lanes' sum, all of one state lane.
    {
      const int t = lane >> 2, q = lane & 3;
      constexpr int kGroups = M::CL / 4;  // columns of a state lane
#pragma unroll
      for (int j = 0; j < S; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float a = acc[j][2 * r], b = acc[j][2 * r + 1];
          if constexpr (kGroups == 1) {
            sm.red[c & 1][warp][t][r][(2 * q) * S + j] = a;
            sm.red[c & 1][warp][t][r][(2 * q + 1) * S + j] = b;
          } else {
            a += b;
            if constexpr (kGroups == 4) a += __shfl_xor_sync(0xffffffffu, a, 1);
            if (kGroups == 2 || (q & 1) == 0) sm.red[c & 1][warp][t][r][(q * 2 / kGroups) * S + j] = a;
          }
        }
    }
    __syncthreads();
    const int kn = min(kChunk, n - t0);
    float* part = p.partial_bc + ((int64_t)blk * p.T + sg.y + t0) * 2 * p.N;
    for (int i = threadIdx.x; i < kn * 2 * p.N; i += kSsmThreads) {
      const int k = i % p.N, r = i / p.N;
      float a = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) a += sm.red[c & 1][v][r >> 1][r & 1][k];
      part[i] = a;
    }
  }

  tile.store(p.partial_A + (int64_t)seg * cells, dA);
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
#pragma unroll
    for (int o = R::LPR; o < 32; o <<= 1) {
      dskip[v] += __shfl_xor_sync(0xffffffffu, dskip[v], o);
      dbias[v] += __shfl_xor_sync(0xffffffffu, dbias[v], o);
    }
    if (in && row == 0) {
      p.partial_par[(int64_t)seg * 2 * p.D + d_row + v] = dskip[v];
      p.partial_par[((int64_t)seg * 2 + 1) * p.D + d_row + v] = dbias[v];
    }
  }
}

// The sums over the other kernels' blocks. Blocks below bc_blocks: dB and dC [T, G, N] over the channel
// blocks, a value a thread. The others: dA [D, N], dD and ddt_bias [D] over the segments, 32 values and
// kSumRows rows of segments a block. All in order.
constexpr int kSumRows = 8;
template <typename E>
__global__ void __launch_bounds__(32 * kSumRows) ssm_bwd_sum_kernel(SsmParams p, int blocks_per_group, int bc_blocks) {
  __shared__ float s[kSumRows][33];
  wait_prerequisite();
  if (p.plan.status[0] != GDN_OK) return;
  if ((int)blockIdx.x < bc_blocks) {
    const int64_t per = p.T * p.N * p.G;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < 2 * per; i += (int64_t)bc_blocks * blockDim.x) {
      const int64_t r = i / p.N, t = r / (2 * p.G);
      const int k = (int)(i - r * p.N), c = (int)(r % 2), g = (int)(r / 2 % p.G);
      const float* q = p.partial_bc + ((((int64_t)g * blocks_per_group) * p.T + t) * 2 + c) * p.N + k;
      const int64_t step = p.T * 2 * p.N;
      float a = 0.f;
#pragma unroll 8
      for (int b = 0; b < blocks_per_group; ++b) a += q[b * step];
      static_cast<E*>(c ? p.dC : p.dB)[(t * p.G + g) * p.N + k] = float_to_elem<E>(a);
    }
    return;
  }
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, n = p.plan.status[1];
  const int64_t cells = (int64_t)p.D * p.N, i = ((int64_t)blockIdx.x - bc_blocks) * 32 + lane;
  const bool of_A = i < cells;
  const float* q = of_A ? p.partial_A + i : p.partial_par + (i - cells);
  const int64_t step = of_A ? cells : 2 * (int64_t)p.D;
  float a = 0.f;
  if (i < cells + 2 * p.D) {
#pragma unroll 4
    for (int j = run; j < n; j += kSumRows) a += q[j * step];
  }
  s[run][lane] = a;
  __syncthreads();
  if (run == 0) {
#pragma unroll
    for (int j = 1; j < kSumRows; ++j) a += s[j][lane];
    if (of_A) {
      p.dA[i] = a;
    } else if (i < cells + p.D) {
      if (p.dD) p.dD[i - cells] = a;
    } else if (i < cells + 2 * p.D) {
      if (p.ddt_bias) p.ddt_bias[i - cells - p.D] = a;
    }
  }
}

template <typename E, typename M, int VEC>
cudaError_t launch_bwd_t(const SsmParams& p, cudaStream_t s, int* kernels) {
  const int per_group = p.D / p.G, bpg = (per_group + M::kChannels - 1) / M::kChannels;
  const dim3 grid((unsigned)(p.max_segs * bpg * p.G)), block(kSsmThreads);
  const int64_t cells = (int64_t)p.D * p.N;
  auto tiles = [](int64_t n, int64_t per, int64_t most) {
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < most ? b : most);
  };
  if (p.T > 0) {
    if (cudaError_t e = launch_after(ssm_bwd_local_kernel<E, M, VEC>, grid, block, 0, s, p, bpg)) return e;
    ++*kernels;
  }
  if (p.B > 0) {
    if (cudaError_t e = launch_after(ssm_bwd_carry_kernel, dim3(tiles(cells, 256, 4096), p.B < 1024 ? p.B : 1024), dim3(256), 0, s, p)) return e;
    ++*kernels;
  }
  if (p.T > 0) {
    constexpr size_t smem = sizeof(MainSmem<E, M, VEC>);
    static std::atomic<uint64_t> allowed{0};
    if (cudaError_t e = allow_shared(ssm_bwd_main_kernel<E, M, VEC>, smem, allowed)) return e;
    if (cudaError_t e = launch_after(ssm_bwd_main_kernel<E, M, VEC>, grid, block, smem, s, p, bpg)) return e;
    ++*kernels;
  }
  ++*kernels;
  const unsigned bc_blocks = p.T > 0 ? tiles(2 * p.T * p.N * p.G, 32 * kSumRows, 1 << 20) : 0;
  const unsigned par_blocks = (unsigned)((cells + 2 * p.D + 31) / 32);
  return launch_after(ssm_bwd_sum_kernel<E>, dim3(bc_blocks + par_blocks), dim3(32 * kSumRows), 0, s, p, bpg, (int)bc_blocks);
}

using Map8 = BwdMap<2, 4, 2>;
using Map16 = BwdMap<4, 4, 4>;
using Map32 = BwdMap<4, 4, 8>;
using Map64 = BwdMap<2, 8, 8>;

}  // namespace

template <typename F>
auto with_map(int N, F&& f) {
  if (N <= 8) return f(Map8{});
  if (N <= 16) return f(Map16{});
  if (N <= 32) return f(Map32{});
  return f(Map64{});
}

int ssm_backward_channels(int N) {
  return with_map(N, [](auto m) { return decltype(m)::kChannels; });
}

// Segments for one round of blocks, of two chunks at least: 1525 tokens of 1002 channels in four sequences, fp32,
// forward and backward: 129 us with at least eight chunks, 109 with four, 100 with two (longer calls fill the
// card with longer segments).
SegmentRule ssm_backward_segments(int64_t T, int B, int D, int G, int N) {
  const int ch = ssm_backward_channels(N), per_group = D / G;
  const int64_t blocks = (int64_t)((per_group + ch - 1) / ch) * G;
  const int64_t fit = kSmCount * with_map(N, [](auto m) { return decltype(m)::kBlocks; });
  return segment_rule(T, B, kChunk, 2 * kChunk, blocks < fit ? fit / blocks : 1);
}

cudaError_t launch_ssm_backward(const SsmParams& p, cudaStream_t s, int* kernels) {
  const int vec = ssm_vec(p, 2, {p.x, p.dt, p.z, p.d_out, p.dx, p.ddt, p.dz},
                          {p.x_stride, p.dt_stride, p.z ? p.z_stride : 0, p.d_stride});
  return with_elem(p.dtype, [&](auto e) {
    using E = decltype(e);
    return with_map(p.N, [&](auto m) {
      using M = decltype(m);
      return vec == 2 ? launch_bwd_t<E, M, 2>(p, s, kernels) : launch_bwd_t<E, M, 1>(p, s, kernels);
    });
  });
}

}  // namespace gdn
