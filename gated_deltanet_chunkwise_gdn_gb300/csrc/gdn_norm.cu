// gdn_norm.cu — layer norm over the last axis, forward and backward, with the reduction of the
// parameters' gradients over the rows.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),  xh = (x - mean) rstd,  out = xh w + b
//   p = dy w,  dx = rstd (p - sum p / n - xh sum(p xh) / n),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: a row is read once and stays in registers, so the variance is taken about the mean (no
// difference of large sums). A block is persistent over rows with the parameters in shared memory and the
// next rows' loads in flight while the current row is reduced; the backward keeps its dw and db sums in
// registers, and writes them once per block.
//
// Measured: norm_kernel 44 us on 14905 rows x 4096 in fp16 (244 MB, 5.5 TB/s, 0.83 of the card's copy rate),
// norm_backward_kernel 78 us on 16384 x 4096 in bf16 (403 MB, 5.1 TB/s, 0.77), norm_reduce_kernel 4 to 8. What
// is left between them and the copy rate is the row's chain: two reductions over its threads forward, one
// of two values backward, with the parameters' shared-memory reads (58 % of that pipe's rate forward).
#include <type_traits>

#include "gdn_ops.cuh"

namespace gdn {

namespace {

constexpr int kNormMaxThreads = 512;  // threads of a row: wider rows go to the re-reading kernels
constexpr int kWideThreads = 256, kWideBlocks = 6;  // of a block of the re-reading kernels; blocks an SM
constexpr size_t kPlainShared = 47 * 1024;  // dynamic shared memory (beside the static) that needs no attribute

// Elements of a row held by one thread: 32 forward, where they are read 16 bytes at a time, so that the
// reduction over the row's threads costs little beside them (14905 rows of 4096: 46 us, 61 with 16); 16 in
// the backward, whose sums of dw and db take two registers an element.
constexpr int kForwardPerThread = 32, kPerThread = 16;
// Threads of one row and rows of one block: whole warps, at least 128 threads a block.
int row_threads(int columns, int per_thread) { return ((columns + per_thread - 1) / per_thread + 31) / 32 * 32; }
bool wide_row(int columns) { return row_threads(columns, kPerThread) > kNormMaxThreads; }  // in the backward
int block_rows(int threads) { return threads >= 128 ? 1 : 128 / threads; }
// Blocks that are resident at once: the launch bounds hold the kernels to 128 registers a thread, so 512
// threads fit on an SM. (Forward rows of 8193 to 16384 columns take 288 to 512 threads, one block an SM, and fill the 512 only
// at the end: 8192 rows of 8192, 8200, 12288 and 16384 columns in bf16 52, 80, 85 and 105 us.)
constexpr int kThreadsPerSm = 512;
int norm_blocks(int64_t rows, int threads) {
  const int r = block_rows(threads);
  const int64_t need = (rows + r - 1) / r, fit = (int64_t)kSmCount * (kThreadsPerSm / (threads * r));
  return (int)(need < fit ? need : fit);
}

// Sum of v over the threads of a row (blockDim.x of them, whole warps), the same in each of them. `buf`
// alternates between two, so one barrier a sum is enough; its places past the row's warps stay zero.
constexpr int kMaxWarps = kNormMaxThreads / 32;
template <int K>
struct RowSums {
  float4 part[2][K][kMaxWarps / 4];  // [which][value][warp of the block]
};
template <int K>
__device__ __forceinline__ void clear_sums(RowSums<K>& buf) {
  float* f = reinterpret_cast<float*>(&buf);
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * K * kMaxWarps; i += blockDim.x * blockDim.y) f[i] = 0.f;
}
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], RowSums<K>& buf, int which, int warps) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_total(v[k]);
  if (warps == 1) return;
  const int first = threadIdx.y * warps;  // a block of several rows has rows of one, two or four warps
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) reinterpret_cast<float*>(buf.part[which][k])[first + (threadIdx.x >> 5)] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (warps == 2) {
      const float2 a = *reinterpret_cast<const float2*>(reinterpret_cast<const float*>(buf.part[which][k]) + first);
      v[k] = a.x + a.y;
    } else {
      v[k] = 0.f;
      for (int i = 0; i < (warps + 3) / 4; ++i) {
        const float4 a = buf.part[which][k][first / 4 + i];
        v[k] += (a.x + a.y) + (a.z + a.w);
      }
    }
  }
}

// A thread's elements of a row come in NV units, each handled as pairs: V neighbouring elements (16 bytes, or
// two), or for V = 1 two single elements a row's threads apart. 16384 rows of 4096 in bf16, forward and
// backward: 50 and 84 us with 16 bytes, 80 and 146 with two elements, 85 and 171 with one.
// FULL: the threads' units cover the row exactly, so none needs a check.
template <int V, bool FULL>
struct Unit {
  static constexpr int kPairs = V == 1 ? 1 : V / 2;
  int c;          // first column
  bool in, both;  // the first (for V > 1: every) element is inside the row; the second of V = 1 too
  __device__ __forceinline__ Unit(int i, int columns) {
    c = V == 1 ? 2 * i * (int)blockDim.x + (int)threadIdx.x : (i * (int)blockDim.x + (int)threadIdx.x) * V;
    in = FULL || c < columns;
    both = FULL || (V > 1 ? in : c + (int)blockDim.x < columns);
  }
  __device__ __forceinline__ int second() const { return c + (int)blockDim.x; }
};

template <typename E, int V, int NV, bool FULL>
struct RowRegs {
  static constexpr int kRaws = V == 1 ? 2 * NV : NV;
  Raw<E, V> r[kRaws];
  __device__ __forceinline__ void load(const E* row, int columns) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Unit<V, FULL> u(i, columns);
      if constexpr (V == 1) {
        if (!FULL) r[2 * i].zero(), r[2 * i + 1].zero();
        if (u.in) r[2 * i].load(row + u.c);
        if (u.both) r[2 * i + 1].load(row + u.second());
      } else {
        if (!FULL) r[i].zero();
        if (u.in) r[i].load(row + u.c);
      }
    }
  }
  __device__ __forceinline__ void widen(float2 (&f)[Unit<V, FULL>::kPairs], int i) const {
    if constexpr (V == 1) {
      float a[1], b[1];
      r[2 * i].widen(a);
      r[2 * i + 1].widen(b);
      f[0] = make_float2(a[0], b[0]);
    } else {
      float x[V];
      r[i].widen(x);
#pragma unroll
      for (int v = 0; v < V / 2; ++v) f[v] = make_float2(x[2 * v], x[2 * v + 1]);
    }
  }
};

template <typename E, int V, bool FULL>
__device__ __forceinline__ void store_unit(E* row, const Unit<V, FULL>& u, const float2 (&f)[Unit<V, FULL>::kPairs]) {
  if constexpr (V == 1) {
    if (u.in) row[u.c] = float_to_elem<E>(f[0].x);
    if (u.both) row[u.second()] = float_to_elem<E>(f[0].y);
  } else if (u.in) {
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = v % 2 ? f[v / 2].y : f[v / 2].x;
    store_vec<E, V>(row + u.c, x);
  }
}

// A parameter in shared memory for the whole block, `other` where there is none. Vectors of 8 are kept as
// two planes of 4, so that a warp's 16-byte reads are of consecutive addresses.
template <int V>
__device__ __forceinline__ void stage_param(float* s, const float* w, int columns, float other) {
  const int n = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  auto place = [&](int c) { return V == 8 ? (c / 4 % 2) * (columns / 2) + c / 8 * 4 + c % 4 : c; };
  if (V >= 4 && w && (reinterpret_cast<uintptr_t>(w) & 15) == 0) {  // (V divides columns)
#pragma unroll 8
    for (int c = tid * 4; c < columns; c += n * 4)
      *reinterpret_cast<float4*>(s + place(c)) = __ldg(reinterpret_cast<const float4*>(w + c));
  } else {
#pragma unroll 8
    for (int c = tid; c < columns; c += n) s[place(c)] = w ? __ldg(w + c) : other;
  }
}
template <int V, bool FULL>
__device__ __forceinline__ void param_unit(float2 (&f)[Unit<V, FULL>::kPairs], const float* s, const Unit<V, FULL>& u, int columns) {
  if constexpr (V == 1) {
    f[0] = make_float2(s[u.c], u.both ? s[u.second()] : 0.f);
  } else if constexpr (V == 2) {
    f[0] = *reinterpret_cast<const float2*>(s + u.c);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(s + (V == 8 ? i * (columns / 2) + u.c / 2 : u.c));
      f[2 * i] = make_float2(q.x, q.y), f[2 * i + 1] = make_float2(q.z, q.w);
    }
  }
}

template <typename E, int V, int NV, bool FULL>
__global__ void __launch_bounds__(kNormMaxThreads) norm_kernel(NormParams p) {
  constexpr int DEPTH = RowRegs<E, V, NV, FULL>::kRaws * Raw<E, V>::kWords <= 16 ? 2 : 1;  // rows in flight
  constexpr int H = Unit<V, FULL>::kPairs;
  extern __shared__ __align__(16) float s_param[];  // weight, bias
  __shared__ __align__(16) RowSums<1> sums;
  const int warps = blockDim.x >> 5;
  const float inv_n = 1.f / (float)p.columns;
  const E* x = static_cast<const E*>(p.x);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowRegs<E, V, NV, FULL> next[DEPTH];
#pragma unroll
  for (int i = 0; i < DEPTH; ++i)
    if (row + i * step < p.rows) next[i].load(x + (row + i * step) * p.x_stride, p.columns);
  const int bias_at = (p.columns + 3) / 4 * 4;
  stage_param<V>(s_param, p.weight, p.columns, 1.f);
  stage_param<V>(s_param + bias_at, p.bias, p.columns, 0.f);
  clear_sums(sums);
  __syncthreads();
  auto one_row = [&](RowRegs<E, V, NV, FULL>& next) {
    float2 f[NV][H], s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) next.widen(f[i], i);
    if (row + DEPTH * step < p.rows) next.load(x + (row + DEPTH * step) * p.x_stride, p.columns);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < H; ++v) s2 = add2(s2, f[i][v]);
    float s[1] = {s2.x + s2.y};
    row_sum<1>(s, sums, 0, warps);
    const float mean = s[0] * inv_n;
    s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Unit<V, FULL> u(i, p.columns);
      if (u.in) {
        const float2 minus = make_float2(-mean, u.both ? -mean : 0.f);  // (a pair's empty half stays zero)
#pragma unroll
        for (int v = 0; v < H; ++v) {
          f[i][v] = add2(f[i][v], minus);
          s2 = fma2(f[i][v], f[i][v], s2);
        }
      }
    }
    s[0] = s2.x + s2.y;
    row_sum<1>(s, sums, 1, warps);
    const float rstd = 1.f / sqrtf(s[0] * inv_n + p.eps);
    if (row < p.rows) {
      E* out = static_cast<E*>(p.out) + row * p.columns;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Unit<V, FULL> u(i, p.columns);
        if (u.in) {
          float2 w[H], b[H];
          param_unit(w, s_param, u, p.columns);
          param_unit(b, s_param + bias_at, u, p.columns);
#pragma unroll
          for (int v = 0; v < H; ++v) f[i][v] = fma2(mul2(f[i][v], both(rstd)), w[v], b[v]);
          store_unit(out, u, f[i]);
        }
      }
      if (p.mean && threadIdx.x == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
    }
    row += step;
  };
  // Each place of `next` by name: moving a row from one to another would wait for its load.
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < p.rows; base += DEPTH * step) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
      if (base + i * step < p.rows) one_row(next[i]);
  }
}

template <typename E, int V, int NV, bool FULL>
__global__ void __launch_bounds__(kNormMaxThreads) norm_backward_kernel(NormParams p) {
  constexpr int DEPTH = RowRegs<E, V, NV, FULL>::kRaws * Raw<E, V>::kWords <= 8 ? 2 : 1;  // rows in flight
  constexpr int H = Unit<V, FULL>::kPairs;
  extern __shared__ __align__(16) float s_param[];  // weight
  __shared__ __align__(16) RowSums<2> sums;
  launch_dependents();
  const int warps = blockDim.x >> 5;
  const float inv_n = 1.f / (float)p.columns;
  float2 dw[NV][H], db[NV][H];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < H; ++v) dw[i][v] = db[i][v] = both(0.f);
  const E *x = static_cast<const E*>(p.x), *dy = static_cast<const E*>(p.d_out);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  RowRegs<E, V, NV, FULL> nx[DEPTH], nd[DEPTH];
  float mean_next[DEPTH], rstd_next[DEPTH];
  auto fetch = [&](int i, int64_t r) {
    if (r < p.rows) {
      nx[i].load(x + r * p.x_stride, p.columns);
      nd[i].load(dy + r * p.d_stride, p.columns);
      mean_next[i] = p.mean[r];
      rstd_next[i] = p.rstd[r];
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) {
    mean_next[i] = rstd_next[i] = 0.f;
    fetch(i, row + i * step);
  }
  stage_param<V>(s_param, p.weight, p.columns, 1.f);
  clear_sums(sums);
  __syncthreads();
  int flip = 0;
  auto one_row = [&](int at) {
    const bool in_row = row < p.rows;
    float2 xh[NV][H], g[NV][H];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[at].widen(xh[i], i);
      nd[at].widen(g[i], i);
    }
    const float mean = mean_next[at], rstd = rstd_next[at];
    fetch(at, row + DEPTH * step);
    float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Unit<V, FULL> u(i, p.columns);
      if (in_row && u.in) {
        float2 w[H];
        param_unit(w, s_param, u, p.columns);
#pragma unroll
        for (int v = 0; v < H; ++v) {  // (dy is zero outside the row)
          xh[i][v] = mul2(add2(xh[i][v], both(-mean)), both(rstd));
          dw[i][v] = fma2(g[i][v], xh[i][v], dw[i][v]);
          db[i][v] = add2(db[i][v], g[i][v]);
          g[i][v] = mul2(g[i][v], w[v]);
          s0 = add2(s0, g[i][v]);
          s1 = fma2(g[i][v], xh[i][v], s1);
        }
      }
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sum<2>(s, sums, flip, warps);
    if (in_row) {
      E* dx = static_cast<E*>(p.dx) + row * p.columns;
      const float2 a = both(-s[0] * inv_n), b = both(-s[1] * inv_n);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Unit<V, FULL> u(i, p.columns);
        if (u.in) {
#pragma unroll
          for (int v = 0; v < H; ++v) g[i][v] = mul2(fma2(xh[i][v], b, add2(g[i][v], a)), both(rstd));
          store_unit(dx, u, g[i]);
        }
      }
    }
    row += step;
    flip ^= 1;
  };
  // Each place of nx and nd by name: moving a row from one to another would wait for its load.
  for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < p.rows; base += DEPTH * step) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i)
      if (base + i * step < p.rows) one_row(i);
  }
  float* part = p.partial + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * 2 * p.columns;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const Unit<V, FULL> u(i, p.columns);
    store_unit(part, u, dw[i]);
    store_unit(part + p.columns, u, db[i]);
  }
}

// dw and db from the partial rows [parts][2][columns], run by run in their order (every block's rows were added one after the
// other before: sums of a fixed order, not a tree): 32 columns and kPartRows runs a block.
constexpr int kPartRows = 16;
__global__ void __launch_bounds__(32 * kPartRows) norm_reduce_kernel(NormParams p, int parts) {
  __shared__ float s[kPartRows][33];
  wait_prerequisite();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t width = 2 * (int64_t)p.columns;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < width)
    for (int i = run; i < parts; i += kPartRows) a += p.partial[i * width + c];
  s[run][lane] = a;
  __syncthreads();
  if (run == 0 && c < width) {
#pragma unroll
    for (int i = 1; i < kPartRows; ++i) a += s[i][lane];
    if (c < p.columns) {
      if (p.dweight) p.dweight[c] = a;
    } else if (p.dbias) {
      p.dbias[c - p.columns] = a;
    }
  }
}

// Sum over a block of kWideThreads.
template <int K>
__device__ __forceinline__ void wide_sum(float (&v)[K], float (*buf)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_total(v[k]);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) buf[threadIdx.x >> 5][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int i = 0; i < kWideThreads / 32; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += buf[i][k];
}

// Rows wider than a block's registers hold (forward 16384 columns, or 8192 without vectors of 16 bytes; backward
// 8192): a block a row, the row read again for each pass over it (from L1 and L2, where it fits), V
// elements at a time. 8192 rows of 8192, 8200 and 16384 columns in bf16, backward: 91 us in registers, 245 and 389 by
// reading again (two kernels, which read x and d_out three times in all).
template <typename E, int V>
__global__ void __launch_bounds__(kWideThreads, kWideBlocks) norm_wide_kernel(NormParams p) {
  __shared__ float s_buf[2][kWideThreads / 32][1];
  const float inv_n = 1.f / (float)p.columns;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const E* x = static_cast<const E*>(p.x) + row * p.x_stride;
    E* out = static_cast<E*>(p.out) + row * p.columns;
    float s[1] = {0.f}, f[V];
#pragma unroll 4
    for (int c = threadIdx.x * V; c < p.columns; c += kWideThreads * V) {
      load_vec<E, V>(f, x + c);
#pragma unroll
      for (int v = 0; v < V; ++v) s[0] += f[v];
    }
    wide_sum<1>(s, s_buf[0]);
    const float mean = s[0] * inv_n;
    s[0] = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x * V; c < p.columns; c += kWideThreads * V) {
      load_vec<E, V>(f, x + c);
#pragma unroll
      for (int v = 0; v < V; ++v) s[0] = fmaf(f[v] - mean, f[v] - mean, s[0]);
    }
    wide_sum<1>(s, s_buf[1]);
    const float rstd = 1.f / sqrtf(s[0] * inv_n + p.eps);
#pragma unroll 4
    for (int c = threadIdx.x * V; c < p.columns; c += kWideThreads * V) {
      load_vec<E, V>(f, x + c);
#pragma unroll
      for (int v = 0; v < V; ++v)
        f[v] = fmaf((f[v] - mean) * rstd, p.weight ? __ldg(p.weight + c + v) : 1.f, p.bias ? __ldg(p.bias + c + v) : 0.f);
      store_vec<E, V>(out + c, f);
    }
    if (p.mean && threadIdx.x == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
  }
}

template <typename E, int V>
__global__ void __launch_bounds__(kWideThreads, kWideBlocks) norm_wide_dx_kernel(NormParams p) {
  __shared__ float s_buf[2][kWideThreads / 32][2];
  launch_dependents();
  const float inv_n = 1.f / (float)p.columns;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const E* x = static_cast<const E*>(p.x) + row * p.x_stride;
    const E* dy = static_cast<const E*>(p.d_out) + row * p.d_stride;
    E* dx = static_cast<E*>(p.dx) + row * p.columns;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.f, 0.f}, g[V], xh[V];
    auto load = [&](int c) {  // dy w and the normalised x
      load_vec<E, V>(g, dy + c);
      load_vec<E, V>(xh, x + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[v] *= p.weight ? __ldg(p.weight + c + v) : 1.f;
        xh[v] = (xh[v] - mean) * rstd;
      }
    };
#pragma unroll 4
    for (int c = threadIdx.x * V; c < p.columns; c += kWideThreads * V) {
      load(c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[0] += g[v];
        s[1] = fmaf(g[v], xh[v], s[1]);
      }
    }
    wide_sum<2>(s, s_buf[flip]);
#pragma unroll 4
    for (int c = threadIdx.x * V; c < p.columns; c += kWideThreads * V) {
      load(c);
#pragma unroll
      for (int v = 0; v < V; ++v) g[v] = rstd * (g[v] - s[0] * inv_n - xh[v] * (s[1] * inv_n));
      store_vec<E, V>(dx + c, g);
    }
  }
}

// dw and db sums of a run of rows, V columns a thread.
template <typename E, int V>
__global__ void __launch_bounds__(256) norm_wide_param_kernel(NormParams p) {
  launch_dependents();
  wait_prerequisite();
  const int c = (blockIdx.x * 256 + threadIdx.x) * V;
  if (c >= p.columns) return;
  float dw[V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = db[v] = 0.f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    float g[V], xv[V];
    load_vec<E, V>(g, static_cast<const E*>(p.d_out) + row * p.d_stride + c);
    load_vec<E, V>(xv, static_cast<const E*>(p.x) + row * p.x_stride + c);
    const float mean = p.mean[row], rstd = p.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      dw[v] = fmaf(g[v], (xv[v] - mean) * rstd, dw[v]);
      db[v] += g[v];
    }
  }
  float* part = p.partial + (int64_t)blockIdx.y * 2 * p.columns;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    part[c + v] = dw[v];
    part[p.columns + c + v] = db[v];
  }
}

constexpr int kWideParts = 64;

int norm_parts(int64_t rows, int columns) {
  if (wide_row(columns)) return (int)(rows < kWideParts ? rows : kWideParts);
  const int threads = row_threads(columns, kPerThread);
  return norm_blocks(rows, threads) * block_rows(threads);
}

// The widest vector that pointers, strides and the row's length allow: 16 bytes, two elements or one.
int row_vector(int dtype, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> strides, int columns) {
  const int size = op_dtype_size(dtype);
  for (int v : {16 / size, 2}) {
    bool ok = columns % v == 0;
    for (const void* q : ptrs) ok = ok && aligned_to(q, (uintptr_t)(v * size));
    for (int64_t st : strides) ok = ok && st % v == 0;
    if (ok) return v;
  }
  return 1;
}

// Calls f(V, NV) for the fewest units a thread of `threads` that cover the row.
template <typename E, typename F>
cudaError_t with_row(int vec, int columns, int threads, F&& f) {
  using std::integral_constant;
  constexpr int V = 16 / (int)sizeof(E);
  if (vec == V) {
    const int need = (columns + threads * V - 1) / (threads * V);
    if (need <= 1) return f(integral_constant<int, V>{}, integral_constant<int, 1>{});
    if (need <= 2) return f(integral_constant<int, V>{}, integral_constant<int, 2>{});
    if (need <= 4) return f(integral_constant<int, V>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, V>{}, integral_constant<int, 32 / V>{});
  }
  const int need = (columns + 2 * threads - 1) / (2 * threads);  // pairs
  auto pairs = [&](auto v) {
    if (need <= 1) return f(v, integral_constant<int, 1>{});
    if (need <= 2) return f(v, integral_constant<int, 2>{});
    return f(v, integral_constant<int, 8>{});
  };
  return vec == 2 ? pairs(integral_constant<int, 2>{}) : pairs(integral_constant<int, 1>{});
}

// The parameters of the longest row that the kernel takes: the limit for all its launches.
template <typename E, int V>
constexpr size_t kMostShared = 2 * sizeof(float) * kNormMaxThreads * (V * sizeof(E) == 16 ? kForwardPerThread : kPerThread);

template <typename E, int V, int NV, bool FULL>
cudaError_t launch_norm_t(const NormParams& p, int threads, cudaStream_t s) {
  const size_t smem = 2 * align_up((size_t)p.columns * sizeof(float), 16);
  if (smem > kPlainShared) {
    static std::atomic<uint64_t> allowed{0};
    if (cudaError_t e = allow_shared(norm_kernel<E, V, NV, FULL>, kMostShared<E, V>, allowed)) return e;
  }
  norm_kernel<E, V, NV, FULL><<<norm_blocks(p.rows, threads), dim3(threads, block_rows(threads)), smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  return with_elem(p.dtype, [&](auto e) {
    using E = decltype(e);
    constexpr int kVec = 16 / (int)sizeof(E);
    const int vec = row_vector(p.dtype, {p.x, p.out}, {p.x_stride}, p.columns);
    const int threads = row_threads(p.columns, vec == kVec ? kForwardPerThread : kPerThread);
    if (threads > kNormMaxThreads) {
      const int64_t fit = kSmCount * kWideBlocks;
      auto* kernel = vec == kVec ? norm_wide_kernel<E, kVec> : norm_wide_kernel<E, 1>;
      kernel<<<(unsigned)(p.rows < fit ? p.rows : fit), kWideThreads, 0, s>>>(p);
      return cudaGetLastError();
    }
    return with_row<E>(vec, p.columns, threads, [&](auto v, auto nv) {
      constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
      if constexpr (V >= 4)  // (a row of single or paired elements is covered exactly only at an odd address)
        if (p.columns == threads * NV * V) return launch_norm_t<E, V, NV, true>(p, threads, s);
      return launch_norm_t<E, V, NV, false>(p, threads, s);
    });
  });
}

size_t norm_backward_workspace(int64_t rows, int columns) {
  const int parts = rows > 0 ? norm_parts(rows, columns) : 0;
  return align_up((size_t)(parts > 0 ? parts : 1) * 2 * columns * sizeof(float), 256);
}

cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t s, int* kernels) {
  const int parts = p.rows > 0 ? norm_parts(p.rows, p.columns) : 0;
  *kernels = 1;
  if (p.rows > 0) {
    cudaError_t err = with_elem(p.dtype, [&](auto e) {
      using E = decltype(e);
      constexpr int kVec = 16 / (int)sizeof(E);
      const int vec = row_vector(p.dtype, {p.x, p.d_out, p.dx}, {p.x_stride, p.d_stride}, p.columns);
      if (wide_row(p.columns)) {
        const int64_t fit = kSmCount * kWideBlocks;
        auto* dx = vec == kVec ? norm_wide_dx_kernel<E, kVec> : norm_wide_dx_kernel<E, 1>;
        dx<<<(unsigned)(p.rows < fit ? p.rows : fit), kWideThreads, 0, s>>>(p);
        if (cudaError_t x = cudaGetLastError()) return x;
        ++*kernels;
        const int units = vec == kVec ? p.columns / kVec : p.columns;
        return launch_after(vec == kVec ? norm_wide_param_kernel<E, kVec> : norm_wide_param_kernel<E, 1>,
                            dim3((units + 255) / 256, parts), dim3(256), 0, s, p);
      }
      const int threads = row_threads(p.columns, kPerThread);
      return with_row<E>(vec, p.columns, threads, [&](auto v, auto nv) {
        constexpr int V = decltype(v)::value, NV = decltype(nv)::value;
        if constexpr (V * NV > kPerThread) {
          return cudaErrorInvalidValue;  // with_row() gives no more than kPerThread elements a thread here
        } else {
          const size_t smem = align_up((size_t)p.columns * sizeof(float), 16);
          auto* kernel = norm_backward_kernel<E, V, NV, false>;
          if constexpr (V >= 4)
            if (p.columns == threads * NV * V) kernel = norm_backward_kernel<E, V, NV, true>;
          kernel<<<norm_blocks(p.rows, threads), dim3(threads, block_rows(threads)), smem, s>>>(p);
          return cudaGetLastError();
        }
      });
    });
    if (err != cudaSuccess) return err;
    ++*kernels;
  }
  return launch_after(norm_reduce_kernel, dim3((unsigned)((2 * (int64_t)p.columns + 31) / 32)), dim3(32 * kPartRows), 0, s, p,
                      parts);
}

}  // namespace gdn
