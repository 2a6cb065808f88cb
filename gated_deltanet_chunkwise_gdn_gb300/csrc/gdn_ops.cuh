// gdn_ops.cuh — shared parts of the sequence-mixer operators beside the delta rule: the short causal
// convolution (gdn_conv.cu), the selective scan (gdn_ssm.cu, gdn_ssm_backward.cu) and layer norm
// (gdn_norm.cu). Launch arguments, element access, activations and the plan kernel that checks a
// packed batch and lays out its work.
#pragma once

#include <atomic>
#include <initializer_list>
#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_decode.cuh"

namespace gdn {

// ----------------------------------------------------------------------------- elements

// V consecutive elements of type E as fp32; V * sizeof(E) is 2, 4, 8, 16 or 32 bytes and the address
// is aligned to the smaller of that and 16.
template <typename E>
__device__ __forceinline__ float elem_to_float(E x) {
  return static_cast<float>(x);
}
template <typename E>
__device__ __forceinline__ E float_to_elem(float x);
template <>
__device__ __forceinline__ bf16 float_to_elem<bf16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ f16 float_to_elem<f16>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ float float_to_elem<float>(float x) {
  return x;
}

// V elements as raw 32-bit words (one 16-bit element: the low half of one word), so that a loop can
// hold loads in flight in few registers and widen them when it uses them.
template <typename E, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(E);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const E* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(E* p) const {
    if constexpr (kBytes == 2) {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void widen(float* f) const {
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      f[0] = ElemT<E>::unpack(w[0]).x;
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 x = ElemT<E>::unpack(w[i]);
        f[2 * i] = x.x, f[2 * i + 1] = x.y;
      }
    }
  }
  __device__ __forceinline__ void narrow(const float* f) {  // round to nearest even
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
      w[0] = ElemT<E>::pack(f[0], 0.f) & 0xffffu;
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = ElemT<E>::pack(f[2 * i], f[2 * i + 1]);
    }
  }
};

template <typename E, int V>
__device__ __forceinline__ void load_vec(float* f, const E* p) {
  Raw<E, V> r;
  r.load(p);
  r.widen(f);
}
template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const float* f) {
  Raw<E, V> r;
  r.narrow(f);
  r.store(p);
}

// Rows on their way from global memory: each thread copies its own V elements of a row into its own place
// in shared memory and reads them back there, so many rows can be in flight without registers and without
// a barrier. ROWS places for each of ARRAYS arrays, THREADS threads. The hardware's asynchronous copies are
// of 4, 8 or 16 bytes. A 2-byte element by itself has two ways, by what its kernel waits for (16384 tokens, rows
// at an odd offset):
// * WORDS: it comes with its aligned word, and the reader gives the row's address again. (The word's other half
//   may be the element before the tensor's first, in the same allocation; never one past its last.) The scan,
//   with few warps, needs the copies in flight: 4096 channels 729 us, 1589 the other way.
// * through a register, loaded and stored at once: the convolution, with warps enough, saves the instructions:
//   8192 channels 156 us, 206 by words.
template <typename E, int V, int ARRAYS, int ROWS, int THREADS, bool WORDS>
struct RowRing {
  static constexpr int kBytes = V * (int)sizeof(E), kCell = kBytes < 4 && WORDS ? 4 : kBytes;
  static_assert(kBytes <= 16, "one copy a row");
  struct __align__(kCell) Cell {
    E e[kCell / sizeof(E)];
  };
  Cell cell[ROWS][ARRAYS][THREADS];

  // Row `place` of array `a` from src; zeros where it is not there.
  __device__ __forceinline__ void copy(int place, int a, const E* src, bool there) {
    const uint32_t to = smem_u32(&cell[place][a][threadIdx.x]);
    if constexpr (kBytes == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(src), "r"(there ? 16 : 0) : "memory");
    } else if constexpr (kBytes >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(to), "l"(src), "n"(kBytes), "r"(there ? kBytes : 0)
                   : "memory");
    } else if constexpr (!WORDS) {
      Raw<E, V> r;
      r.zero();
      if (there) r.load(src);
      r.store(cell[place][a][threadIdx.x].e);
    } else {  // the word up to the element's end
      const uintptr_t at = reinterpret_cast<uintptr_t>(src);
      const uint32_t n = there ? 2 + (uint32_t)(at & 2) : 0;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(to), "l"(at & ~(uintptr_t)3), "r"(n) : "memory");
    }
  }
  // The row that came from `src` (only the address's low bits matter).
  __device__ __forceinline__ Raw<E, V> read(int place, int a, const E* src) const {
    Raw<E, V> r;
    if constexpr (kBytes >= 4 || !WORDS) {
      r.load(cell[place][a][threadIdx.x].e);
    } else {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(&cell[place][a][threadIdx.x]);
      r.w[0] = (word >> (reinterpret_cast<uintptr_t>(src) & 2) * 8) & 0xffffu;
    }
    return r;
  }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {  // all but the last N committed groups have arrived
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// ----------------------------------------------------------------------------- arithmetic

constexpr float kLog2e = 1.4426950408889634f;

// 2^x and 1 / x by the special-function unit, for every type: relative error about 2^-22 and 2^-23, results under 2^-126 zero.
// Beside them stands the argument's own rounding, 2^-24 of it, which the exact functions could not take back. The
// scan forms one exponential a state and token and is bound by them; where a tie of a 16-bit rounding is that near, an
// output falls on its other side (7 of 327680 values of single-token convolutions are not the nearest bf16, and 5 of those of
// elementary torch operations in fp32).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)); exact limits at +-inf (2^(+inf) = inf, 1 / inf = 0).
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// softplus(x) = max(x, 0) + log(1 + t), t = 2^(-|x| log2 e) in [0, 1]. log(1 + t) / t as a polynomial of
// degree 8 through the Chebyshev points of [0, 1]: relative error 1.7e-7 evaluated in fp32, with no
// cancellation for small t. Two values at a time.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 t = make_float2(ex2(-kLog2e * fabsf(x.x)), ex2(-kLog2e * fabsf(x.y)));
  float2 r = make_float2(5.253457930e-03f, 5.253457930e-03f);
  const float c[8] = {-2.958850749e-02f, 7.836166769e-02f, -1.367477030e-01f, 1.911143064e-01f,
                      -2.484436929e-01f, 3.331927061e-01f, -4.999950230e-01f, 1.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) r = fma2(r, t, make_float2(c[i], c[i]));
  return fma2(r, t, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
template <int V>
__device__ __forceinline__ void softplus_of(float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = softplus2(make_float2(x[0], x[0])).x;
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 r = softplus2(make_float2(x[v], x[v + 1]));
      x[v] = r.x, x[v + 1] = r.y;
    }
  }
}

// V values at a time, in pairs where there are any: c += a b, c += a, c *= a, y <- y sigmoid(y).
template <int V>
__device__ __forceinline__ void fma_v(float (&c)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V == 1) {
    c[0] = fmaf(a[0], b[0], c[0]);
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 r = fma2(make_float2(a[v], a[v + 1]), make_float2(b[v], b[v + 1]), make_float2(c[v], c[v + 1]));
      c[v] = r.x, c[v + 1] = r.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void add_v(float (&c)[V], const float (&a)[V]) {
  if constexpr (V == 1) {
    c[0] += a[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 r = add2(make_float2(c[v], c[v + 1]), make_float2(a[v], a[v + 1]));
      c[v] = r.x, c[v + 1] = r.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void mul_v(float (&c)[V], const float (&a)[V]) {
  if constexpr (V == 1) {
    c[0] *= a[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 r = mul2(make_float2(c[v], c[v + 1]), make_float2(a[v], a[v + 1]));
      c[v] = r.x, c[v + 1] = r.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void sigmoid_v(float (&sig)[V], const float (&x)[V]) {
  if constexpr (V == 1) {
    sig[0] = sigmoid_fast(x[0]);
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
      const float2 e = mul2(make_float2(x[v], x[v + 1]), both(-kLog2e));
      const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
      sig[v] = rcp(d.x), sig[v + 1] = rcp(d.y);
    }
  }
}
template <int V>
__device__ __forceinline__ void silu_v(float (&y)[V]) {
  float sig[V];
  sigmoid_v<V>(sig, y);
  mul_v<V>(y, sig);
}

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Programmatic dependent launch. Every kernel launched behind another of the same call with
// launch_after() executes wait_prerequisite() in every thread block before it touches what an
// earlier kernel of the call wrote and before it exits, so that the order is transitive.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_prerequisite() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// item = q n + r; a 64-bit division only where it has to be (it takes a hundred instructions).
__device__ __forceinline__ void split_item(uint64_t item, uint32_t n, int& q, int& r) {
  if (item >> 32 == 0) {
    const uint32_t i = (uint32_t)item, d = i / n;
    q = (int)d, r = (int)(i - d * n);
  } else {
    const uint64_t d = item / n;
    q = (int)d, r = (int)(item - d * n);
  }
}

// How a step's slots are checked (distinct, inside the pool): up to 32 by every warp for itself, up to 256 by
// every block in a hash table of its own (slots of 31 bits), more by a kernel before, and so where the step
// moves so many bytes of state that the GPU is what it waits for: the call without that kernel takes the
// host 1.5 us less, the blocks' own check takes the GPU more the more blocks there are. Scan steps, us a call
// with the blocks' check and with the kernel before: 40 sequences of 4096 channels and 16 states (21 MB)
// 17.0 and 18.7, 128 (67 MB) 18.2 and 18.5, 256 (134 MB) 32.8 and 31.1; 256 of 1024 channels (34 MB) 16.7 and 18.5.
enum SlotCheck : int { kCheckBefore = 0, kCheckWarp = 1, kCheckBlock = 2 };
constexpr int kWarpCheck = 32, kBlockCheck = 256;
inline SlotCheck slot_check(int B, int64_t pool_size, int64_t state_bytes) {
  if (B <= kWarpCheck) return kCheckWarp;
  return B <= kBlockCheck && pool_size < INT32_MAX && state_bytes <= (int64_t)80 << 20 ? kCheckBlock : kCheckBefore;
}

__device__ __forceinline__ bool warp_slots_ok(const int64_t* idx, int B, int64_t pool_size) {
  const int lane = threadIdx.x & 31;
  const int64_t slot = lane < B ? idx[lane] : -1 - lane;
  const bool twice = __popc(__match_any_sync(0xffffffffu, slot)) > 1;
  return !__any_sync(0xffffffffu, lane < B && (twice || slot < 0 || slot >= pool_size));
}

// Open addressing, at most half full, so a probe ends within the table.
__device__ __forceinline__ bool block_slots_ok(const int64_t* idx, int B, int64_t pool_size) {
  constexpr int kPlaces = 2 * kBlockCheck;
  __shared__ int table[kPlaces];
  for (int i = threadIdx.x; i < kPlaces; i += blockDim.x) table[i] = -1;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < B; i += blockDim.x) {
    const int64_t slot = idx[i];
    if (slot < 0 || slot >= pool_size) {
      bad = true;
      continue;
    }
    uint32_t at = (uint32_t)slot * 2654435761u >> 23;  // the upper bits of a multiplicative hash
    static_assert(kPlaces == 512, "nine bits");
    for (int n = 0; n < kPlaces; ++n) {
      const int was = atomicCAS(&table[at], -1, (int)slot);
      if (was == -1) break;
      if (was == (int)slot) {
        bad = true;
        break;
      }
      at = (at + 1) % kPlaces;
    }
  }
  return !__syncthreads_or(bad);
}

// The verdict on a step's slots, in every thread of it: found here, or waited for. A step's kernel calls it in
// every thread before any of them leaves. It may read the pool before: what runs before a step's first
// kernel has finished by then, and the check writes only the status word.
template <int CHECK>
__device__ __forceinline__ bool step_slots_ok(const int64_t* idx, int B, int64_t pool_size, int32_t* status) {
  if constexpr (CHECK == kCheckBefore) {
    wait_prerequisite();
    return *status == GDN_OK;
  } else {
    const bool ok = CHECK == kCheckWarp ? warp_slots_ok(idx, B, pool_size) : block_slots_ok(idx, B, pool_size);
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = ok ? GDN_OK : GDN_ERR_BAD_INDEX;
    return ok;
  }
}

// Calls f with the check's constant.
template <typename F>
auto with_check(SlotCheck c, F&& f) {
  if (c == kCheckWarp) return f(std::integral_constant<int, kCheckWarp>{});
  if (c == kCheckBlock) return f(std::integral_constant<int, kCheckBlock>{});
  return f(std::integral_constant<int, kCheckBefore>{});
}

template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ----------------------------------------------------------------------------- host-side helpers

// Element types of the operators' activations.
inline bool op_dtype_ok(int dtype) { return dtype == GDN_BF16 || dtype == GDN_FP16 || dtype == GDN_FP32; }
inline int op_dtype_size(int dtype) { return dtype == GDN_FP32 ? 4 : 2; }

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Calls f with a value of the dtype's element type.
template <typename F>
cudaError_t with_elem(int dtype, F&& f) {
  switch (dtype) {
    case GDN_BF16: return f(bf16{});
    case GDN_FP16: return f(f16{});
    default: return f(float{});
  }
}

constexpr int kSmCount = 152;  // GB300

// Dynamic shared memory above 48 KB has to be allowed per kernel and device: once, for the largest launch of the
// kernel, since the limit is the kernel's and a launch of another thread may stand between setting it and using it.
// `done`: the devices (by their number's low six bits) that have it, one word per kernel.
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) return e;
  done.fetch_or(bit, std::memory_order_relaxed);
  return cudaSuccess;
}

// ----------------------------------------------------------------------------- plan of a packed batch

// The plan of a call over a packed batch, in the workspace: written by the plan kernel, which checks
// cu_seqlens and cache_indices, and read by the call's later kernels.
struct Plan {
  int32_t* status;   // int32[64]: [0] status code, [1] number of segments
  int32_t* seq_off;  // int32[B+1]: first segment of each sequence
  int4* seg_tab;     // (sequence, first token, length, index in its sequence) of each segment
};

struct PlanLayout {
  size_t status, seq_off, seg_tab, total;
};

// How a batch is cut: into segments of a multiple of `unit` and at least `least` tokens, of a length that is
// chosen on the device from the sequences' lengths so that about `target` segments run side by side.
// target = 0: every segment `least` long.
struct SegmentRule {
  int unit, least, target;
  int64_t max_segs;  // bound of the number of segments, for the grids and the workspace
};
SegmentRule segment_rule(int64_t T, int B, int unit, int least, int64_t target);

inline PlanLayout make_plan_layout(int B, const SegmentRule& rule) {
  PlanLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  L.status = take(64 * sizeof(int32_t));
  L.seq_off = take((size_t)(B + 1) * sizeof(int32_t));
  L.seg_tab = take((size_t)(rule.max_segs > 0 ? rule.max_segs : 1) * sizeof(int4));
  L.total = off;
  return L;
}

inline Plan plan_at(char* ws, const PlanLayout& L) {
  return Plan{reinterpret_cast<int32_t*>(ws + L.status), reinterpret_cast<int32_t*>(ws + L.seq_off),
              reinterpret_cast<int4*>(ws + L.seg_tab)};
}

// Enqueues the plan; *kernels gets the number of kernels launched.
cudaError_t launch_plan(const Plan& plan, const int64_t* cu_seqlens, const int64_t* cache_indices, int B, int64_t T,
                        int64_t pool_size, const SegmentRule& rule, cudaStream_t s, int* kernels);

// ----------------------------------------------------------------------------- convolution

struct ConvParams {
  const void* x;        // [T, D], row stride x_stride
  const float* weight;  // [D, W]
  const float* bias;    // [D] or null
  void* pool;           // [pool, W-1, D] of x's type
  const int64_t* cache_indices;
  const int64_t* cu_seqlens;
  void* out;  // [T, D]
  int64_t T, x_stride;
  int64_t pool_size;
  int B, D, W;
  SlotCheck check;  // of a step
  int silu;
  int dtype;
  int weight_vec;  // weight is 16-byte aligned
  int32_t* status;
  Plan plan;
  // backward
  const void* d_out;       // [T, D], row stride d_stride
  const float* d_state;    // [pool, W-1, D] or null
  void* dx;                // [T, D]
  float* dweight;          // [D, W]
  float* dbias;            // [D] or null
  float* d_pool;           // [pool, W-1, D]
  float* partial;          // [segments, W + 1, D]
  int64_t d_stride;
  int64_t max_segs;
};

SegmentRule conv_segments(int64_t T, int B, int D, bool backward);
cudaError_t launch_conv_extend(const ConvParams& p, cudaStream_t s);
cudaError_t launch_conv_step(const ConvParams& p, cudaStream_t s);
cudaError_t launch_conv_backward(const ConvParams& p, cudaStream_t s, int* kernels);

// ----------------------------------------------------------------------------- selective scan

struct SsmParams {
  const void* x;   // [T, D]
  const void* dt;  // [T, D]
  const void* Bm;  // [T, G, N]
  const void* Cm;  // [T, G, N]
  const void* z;   // [T, D] or null
  const float* A;  // [D, N]
  const float* Dskip;    // [D] or null
  const float* dt_bias;  // [D] or null
  float* pool;           // [pool, D, N]
  const int64_t* cache_indices;
  const int64_t* cu_seqlens;
  void* out;  // [T, D]
  int64_t T;
  int64_t pool_size;
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;  // row strides, in elements
  int B, D, G, N;
  SlotCheck check;  // of a step
  int softplus;
  int dtype;
  int32_t* status;
  Plan plan;
  int64_t max_segs;
  float* seg_state;  // [segments, D, N]: a segment's end state from its own tokens, then its start state
  float* seg_delta;  // [segments, D]: sum of delta over a segment
  // backward
  const void* d_out;  // [T, D], row stride d_stride
  int64_t d_stride;
  const float* d_state;                       // [pool, D, N] or null
  void *dx, *ddt, *dB, *dC, *dz;
  float *dA, *dD, *ddt_bias, *d_pool;
  float* seg_grad;    // [segments, D, N]: gradient leaving a segment backwards, then the one entering its last state
  float* ckpt;        // [chunks, D, N]: state entering a chunk, from its segment's own tokens
  float* ckpt_delta;  // [chunks, D]: sum of delta over the segment's earlier chunks
  float* partial_bc;  // [channel blocks, T, 2, N]
  float* partial_A;   // [segments, D, N]
  float* partial_par; // [segments, 2, D]
};

SegmentRule ssm_segments(int64_t T, int B, int D, int G, int N);
cudaError_t launch_ssm_extend(const SsmParams& p, const SegmentRule& rule, cudaStream_t s, int* kernels);
cudaError_t launch_ssm_step(const SsmParams& p, cudaStream_t s);
constexpr int kSsmChunk = 8;  // tokens of one chunk of the backward
int ssm_backward_channels(int N);  // channels of one block of the backward
SegmentRule ssm_backward_segments(int64_t T, int B, int D, int G, int N);
cudaError_t launch_ssm_backward(const SsmParams& p, cudaStream_t s, int* kernels);

// ----------------------------------------------------------------------------- layer norm

struct NormParams {
  const void* x;  // [rows, columns], row stride x_stride
  const float* weight;
  const float* bias;
  void* out;
  float* mean;  // [rows] or null
  float* rstd;
  int64_t rows, x_stride;
  int columns;
  float eps;
  int dtype;
  // backward
  const void* d_out;  // row stride d_stride
  int64_t d_stride;
  void* dx;
  float* dweight;
  float* dbias;
  float* partial;
};

cudaError_t launch_norm(const NormParams& p, cudaStream_t s);
size_t norm_backward_workspace(int64_t rows, int columns);
cudaError_t launch_norm_backward(const NormParams& p, cudaStream_t s, int* kernels);

}  // namespace gdn
