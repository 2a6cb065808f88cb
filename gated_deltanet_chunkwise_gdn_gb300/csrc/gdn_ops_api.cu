// gdn_ops_api.cu — host side of the convolution, selective scan and layer norm entry points of
// include/gdn.h: argument checks, workspace carve-up and the launch sequences.
#include <nvtx3/nvToolsExt.h>

#include "gdn_ops.cuh"

namespace {

using gdn::align_up;
using gdn::aligned_to;

struct NvtxRange {  // host-side range of one call, for timelines
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr int32_t kMaxStepBatch = 1 << 20;
constexpr int64_t kMaxBlocks = INT32_MAX;

// The kernels count a segment's tokens in 32 bits, up to a tile (64 tokens) past its end.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1024;
bool batch_sizes_ok(int64_t T, int32_t B) { return T >= 0 && T <= kMaxTokens && B >= 0; }

// The kernels count a row's columns in 32 bits, up to a block's share of them past its end.
constexpr int32_t kMaxColumns = 1 << 30;

bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride < ((int64_t)1 << 40); }

bool workspace_ok(const void* ws, size_t have, size_t need) { return ws && have >= need && aligned_to(ws, 256); }

gdn_status done(cudaError_t e, int kernels) {
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  gdn::count_launches(kernels);
  return GDN_OK;
}

// A step: its update kernel, which checks the slots of batches up to gdn::kBlockCheck itself, or a kernel that
// does before it.
template <typename F>
gdn_status run_step(const int64_t* cache_indices, int32_t batch, int64_t pool_size, int32_t* status, gdn::SlotCheck check,
                    cudaStream_t s, F&& update) {
  if (batch == 0 || gdn::decode_check_needs_zeroed_status(batch)) {
    if (cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return GDN_ERR_CUDA;
    if (batch == 0) return GDN_OK;
  }
  if (check != gdn::kCheckBefore) return done(update(), 1);
  gdn::DecodeParams dp{};
  dp.cache_indices = cache_indices;
  dp.pool_size = pool_size;
  dp.B = batch;
  dp.status = status;
  if (gdn::launch_decode_check(dp, s) != cudaSuccess) return GDN_ERR_CUDA;
  return done(update(), 2);
}

// ------------------------------------------------------------------ convolution

bool conv_sizes_ok(int64_t T, int32_t B, int32_t channels, int32_t width) {
  if (!batch_sizes_ok(T, B) || channels <= 0 || width < 2 || width > 4) return false;
  const int64_t segs = gdn::conv_segments(T, B, channels, false).max_segs;  // the backward has fewer
  return segs <= kMaxBlocks && segs * channels / 128 + 1 <= kMaxBlocks;
}

struct ConvLayout {
  gdn::SegmentRule rule;
  gdn::PlanLayout plan;
  size_t partial, total;
};

ConvLayout conv_layout(int64_t T, int32_t B, int32_t channels, int32_t width, bool backward) {
  ConvLayout L{};
  L.rule = gdn::conv_segments(T, B, channels, backward);
  L.plan = gdn::make_plan_layout(B, L.rule);
  L.partial = L.plan.total;
  L.total = L.partial;
  if (backward) L.total += align_up((size_t)L.rule.max_segs * (width + 1) * channels * sizeof(float), 256);
  return L;
}

// ------------------------------------------------------------------ selective scan

// A block of either pass has at least 32 channels.
bool ssm_blocks_ok(const gdn::SegmentRule& rule, int32_t channels, int32_t groups) {
  return rule.max_segs <= kMaxBlocks && rule.max_segs * (((int64_t)channels / groups + 31) / 32 * groups) <= kMaxBlocks;
}
bool ssm_shape_ok(int64_t T, int32_t B, int32_t channels, int32_t groups, int32_t states) {
  return batch_sizes_ok(T, B) && channels > 0 && groups > 0 && channels % groups == 0 && states > 0;
}
bool ssm_shape_built(int32_t states) { return states <= 64; }

struct SsmLayout {
  gdn::SegmentRule rule;
  gdn::PlanLayout plan;
  size_t seg_state, seg_delta, seg_grad, ckpt, ckpt_delta, partial_bc, partial_A, partial_par, total;
};

SsmLayout ssm_layout(int64_t T, int32_t B, int32_t D, int32_t G, int32_t N, bool backward) {
  SsmLayout L{};
  L.rule = backward ? gdn::ssm_backward_segments(T, B, D, G, N) : gdn::ssm_segments(T, B, D, G, N);
  L.plan = gdn::make_plan_layout(B, L.rule);
  size_t off = L.plan.total;
  auto take = [&](size_t floats) {
    const size_t o = off;
    off = align_up(off + floats * sizeof(float), 256);
    return o;
  };
  const size_t segs = (size_t)L.rule.max_segs, cells = (size_t)D * N;
  const bool split = backward || T > L.rule.least;
  L.seg_state = take(split ? segs * cells : 0);
  L.seg_delta = take(split ? segs * D : 0);
  if (backward) {
    const size_t chunks = (size_t)T / gdn::kSsmChunk + segs + 1;
    const int64_t ch = gdn::ssm_backward_channels(N);
    const size_t blocks = (size_t)(((int64_t)D / G + ch - 1) / ch * G);
    L.seg_grad = take(segs * cells);
    L.ckpt = take(chunks * cells);
    L.ckpt_delta = take(chunks * D);
    L.partial_bc = take(blocks * (size_t)T * 2 * N);
    L.partial_A = take(segs * cells);
    L.partial_par = take(segs * 2 * D);
  }
  L.total = off;
  return L;
}

struct SsmArgs {
  const void *x, *dt, *B, *C, *z;
  int64_t x_stride, dt_stride, B_stride, C_stride, z_stride;
  const float *A, *D, *dt_bias;
  int32_t dtype, channels, groups, states, softplus;
};

bool ssm_args_ok(const SsmArgs& a, bool tokens) {
  if (!gdn::op_dtype_ok(a.dtype)) return false;
  if (!a.A || !aligned_to(a.A, 4) || !aligned_to(a.D, 4) || !aligned_to(a.dt_bias, 4)) return false;
  if (!tokens) return true;
  const uintptr_t size = gdn::op_dtype_size(a.dtype);
  const int64_t gn = (int64_t)a.groups * a.states;
  for (const void* q : {a.x, a.dt, a.B, a.C})
    if (!q || !aligned_to(q, size)) return false;
  if (!aligned_to(a.z, size)) return false;
  return stride_ok(a.x_stride, a.channels) && stride_ok(a.dt_stride, a.channels) && stride_ok(a.B_stride, gn) &&
         stride_ok(a.C_stride, gn) && (!a.z || stride_ok(a.z_stride, a.channels));
}

gdn::SsmParams ssm_params(const SsmArgs& a) {
  gdn::SsmParams p{};
  p.x = a.x;
  p.dt = a.dt;
  p.Bm = a.B;
  p.Cm = a.C;
  p.z = a.z;
  p.A = a.A;
  p.Dskip = a.D;
  p.dt_bias = a.dt_bias;
  p.x_stride = a.x_stride;
  p.dt_stride = a.dt_stride;
  p.b_stride = a.B_stride;
  p.c_stride = a.C_stride;
  p.z_stride = a.z_stride;
  p.D = a.channels;
  p.G = a.groups;
  p.N = a.states;
  p.softplus = a.softplus != 0;
  p.dtype = a.dtype;
  return p;
}

}  // namespace

extern "C" {

size_t gdn_conv_workspace_size(int64_t total_tokens, int32_t batch, int32_t channels, int32_t width) {
  return conv_sizes_ok(total_tokens, batch, channels, width) ? conv_layout(total_tokens, batch, channels, width, false).total : 0;
}

size_t gdn_conv_backward_workspace_size(int64_t total_tokens, int32_t batch, int32_t channels, int32_t width) {
  return conv_sizes_ok(total_tokens, batch, channels, width) ? conv_layout(total_tokens, batch, channels, width, true).total : 0;
}

gdn_status gdn_conv_extend(const void* x, int64_t x_stride, gdn_dtype dtype, const float* weight, const float* bias,
                           void* conv_pool, int64_t pool_size, const int64_t* cache_indices, const int64_t* cu_seqlens,
                           int32_t batch, void* out, int64_t total_tokens, int32_t channels, int32_t width, int32_t silu,
                           void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("gdn_conv_extend");
  if (!batch_sizes_ok(total_tokens, batch) || channels <= 0 || width <= 0 || !gdn::op_dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  const uintptr_t size = gdn::op_dtype_size(dtype);
  if (!cu_seqlens || !weight || !aligned_to(weight, 4) || !aligned_to(bias, 4)) return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!conv_pool || !cache_indices || pool_size <= 0 || !aligned_to(conv_pool, size))) return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!x || !out || !aligned_to(x, size) || !aligned_to(out, size) || !stride_ok(x_stride, channels)))
    return GDN_ERR_INVALID_ARG;
  if (!conv_sizes_ok(total_tokens, batch, channels, width)) return GDN_ERR_UNSUPPORTED;
  const ConvLayout L = conv_layout(total_tokens, batch, channels, width, false);
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return GDN_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  gdn::ConvParams p{};
  p.x = x;
  p.weight = weight;
  p.weight_vec = aligned_to(weight, 16);
  p.bias = bias;
  p.pool = conv_pool;
  p.cache_indices = cache_indices;
  p.cu_seqlens = cu_seqlens;
  p.out = out;
  p.T = total_tokens;
  p.x_stride = x_stride;
  p.B = batch;
  p.D = channels;
  p.W = width;
  p.silu = silu != 0;
  p.dtype = dtype;
  p.plan = gdn::plan_at(static_cast<char*>(workspace), L.plan);
  p.max_segs = L.rule.max_segs;
  int kernels = 0;
  if (gdn::launch_plan(p.plan, cu_seqlens, cache_indices, batch, total_tokens, pool_size, L.rule, s, &kernels) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (total_tokens == 0 || batch == 0) return done(cudaSuccess, kernels);
  return done(gdn::launch_conv_extend(p, s), kernels + 1);
}

gdn_status gdn_conv_step(const void* x, int64_t x_stride, gdn_dtype dtype, const float* weight, const float* bias,
                         void* conv_pool, int64_t pool_size, const int64_t* cache_indices, int32_t batch, void* out,
                         int32_t channels, int32_t width, int32_t silu, int32_t* device_status, void* stream) {
  NvtxRange range("gdn_conv_step");
  if (batch < 0 || batch > kMaxStepBatch || channels <= 0 || width <= 0 || !gdn::op_dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  const uintptr_t size = gdn::op_dtype_size(dtype);
  if (!device_status || !aligned_to(device_status, 4) || !weight || !aligned_to(weight, 4) || !aligned_to(bias, 4))
    return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!x || !out || !conv_pool || !cache_indices || pool_size <= 0 || !aligned_to(x, size) ||
                    !aligned_to(out, size) || !aligned_to(conv_pool, size) || !stride_ok(x_stride, channels)))
    return GDN_ERR_INVALID_ARG;
  if (width < 2 || width > 4 || (int64_t)batch * channels / 128 + 1 > kMaxBlocks) return GDN_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  gdn::ConvParams p{};
  p.x = x;
  p.weight = weight;
  p.weight_vec = aligned_to(weight, 16);
  p.bias = bias;
  p.pool = conv_pool;
  p.cache_indices = cache_indices;
  p.out = out;
  p.T = batch;
  p.x_stride = x_stride;
  p.B = batch;
  p.D = channels;
  p.W = width;
  p.silu = silu != 0;
  p.dtype = dtype;
  p.status = device_status;
  p.pool_size = pool_size;
  p.check = gdn::slot_check(batch, pool_size, (int64_t)batch * (width - 1) * channels * size * 2);
  return run_step(cache_indices, batch, pool_size, device_status, p.check, s, [&] { return gdn::launch_conv_step(p, s); });
}

gdn_status gdn_conv_backward(const void* x, int64_t x_stride, gdn_dtype dtype, const float* weight, const float* bias,
                             const void* conv_pool, int64_t pool_size, const int64_t* cache_indices,
                             const int64_t* cu_seqlens, int32_t batch, const void* d_out, int64_t d_out_stride,
                             const float* d_state, void* dx, float* dweight, float* dbias, float* d_conv_pool,
                             int64_t total_tokens, int32_t channels, int32_t width, int32_t silu, void* workspace,
                             size_t workspace_bytes, void* stream) {
  NvtxRange range("gdn_conv_backward");
  if (!batch_sizes_ok(total_tokens, batch) || channels <= 0 || width <= 0 || !gdn::op_dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  const uintptr_t size = gdn::op_dtype_size(dtype);
  if (!cu_seqlens || !weight || !aligned_to(weight, 4) || !aligned_to(bias, 4) || !dweight || !aligned_to(dweight, 4) ||
      !aligned_to(dbias, 4))
    return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!conv_pool || !cache_indices || pool_size <= 0 || !aligned_to(conv_pool, size) || !d_conv_pool ||
                    !aligned_to(d_conv_pool, 4) || !aligned_to(d_state, 4) || d_state == d_conv_pool))
    return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!x || !d_out || !dx || !aligned_to(x, size) || !aligned_to(d_out, size) || !aligned_to(dx, size) ||
                           !stride_ok(x_stride, channels) || !stride_ok(d_out_stride, channels)))
    return GDN_ERR_INVALID_ARG;
  if (!conv_sizes_ok(total_tokens, batch, channels, width)) return GDN_ERR_UNSUPPORTED;
  const ConvLayout L = conv_layout(total_tokens, batch, channels, width, true);
  if (!workspace_ok(workspace, workspace_bytes, L.total)) return GDN_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  gdn::ConvParams p{};
  p.x = x;
  p.weight = weight;
  p.weight_vec = aligned_to(weight, 16);
  p.bias = bias;
  p.pool = const_cast<void*>(conv_pool);  // read only in the backward kernels
  p.cache_indices = cache_indices;
  p.cu_seqlens = cu_seqlens;
  p.T = total_tokens;
  p.x_stride = x_stride;
  p.B = batch;
  p.D = channels;
  p.W = width;
  p.silu = silu != 0;
  p.dtype = dtype;
  p.plan = gdn::plan_at(ws, L.plan);
  p.max_segs = total_tokens > 0 && batch > 0 ? L.rule.max_segs : 0;
  p.d_out = d_out;
  p.d_stride = d_out_stride;
  p.d_state = d_state;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.d_pool = d_conv_pool;
  p.partial = reinterpret_cast<float*>(ws + L.partial);
  int kernels = 0, more = 0;
  if (gdn::launch_plan(p.plan, cu_seqlens, cache_indices, batch, total_tokens, pool_size, L.rule, s, &kernels) != cudaSuccess)
    return GDN_ERR_CUDA;
  const cudaError_t e = gdn::launch_conv_backward(p, s, &more);
  return done(e, kernels + more);
}

size_t gdn_ssm_workspace_size(int64_t total_tokens, int32_t batch, int32_t channels, int32_t groups, int32_t states) {
  if (!ssm_shape_ok(total_tokens, batch, channels, groups, states) || !ssm_shape_built(states)) return 0;
  const SsmLayout L = ssm_layout(total_tokens, batch, channels, groups, states, false);
  return ssm_blocks_ok(L.rule, channels, groups) ? L.total : 0;
}

size_t gdn_ssm_backward_workspace_size(int64_t total_tokens, int32_t batch, int32_t channels, int32_t groups, int32_t states) {
  if (!ssm_shape_ok(total_tokens, batch, channels, groups, states) || !ssm_shape_built(states)) return 0;
  const SsmLayout L = ssm_layout(total_tokens, batch, channels, groups, states, true);
  return ssm_blocks_ok(L.rule, channels, groups) ? L.total : 0;
}

gdn_status gdn_ssm_extend(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, gdn_dtype dtype, const float* A,
                          const void* B, int64_t B_stride, const void* C, int64_t C_stride, const float* D, const void* z,
                          int64_t z_stride, const float* dt_bias, float* state_pool, int64_t pool_size,
                          const int64_t* cache_indices, const int64_t* cu_seqlens, int32_t batch, void* out,
                          int64_t total_tokens, int32_t channels, int32_t groups, int32_t states, int32_t softplus,
                          void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("gdn_ssm_extend");
  if (!ssm_shape_ok(total_tokens, batch, channels, groups, states) || !cu_seqlens) return GDN_ERR_INVALID_ARG;
  const SsmArgs a{x, dt, B, C, z, x_stride, dt_stride, B_stride, C_stride, z_stride, A, D, dt_bias,
                  (int32_t)dtype, channels, groups, states, softplus};
  if (!ssm_args_ok(a, total_tokens > 0)) return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!state_pool || !cache_indices || pool_size <= 0 || !aligned_to(state_pool, 4))) return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!out || !aligned_to(out, gdn::op_dtype_size(dtype)))) return GDN_ERR_INVALID_ARG;
  const size_t need = gdn_ssm_workspace_size(total_tokens, batch, channels, groups, states);
  if (need == 0) return GDN_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const SsmLayout L = ssm_layout(total_tokens, batch, channels, groups, states, false);
  gdn::SsmParams p = ssm_params(a);
  p.pool = state_pool;
  p.cache_indices = cache_indices;
  p.cu_seqlens = cu_seqlens;
  p.out = out;
  p.T = total_tokens;
  p.B = batch;
  p.plan = gdn::plan_at(ws, L.plan);
  p.max_segs = L.rule.max_segs;
  p.seg_state = reinterpret_cast<float*>(ws + L.seg_state);
  p.seg_delta = reinterpret_cast<float*>(ws + L.seg_delta);
  int kernels = 0;
  if (gdn::launch_plan(p.plan, cu_seqlens, cache_indices, batch, total_tokens, pool_size, L.rule, s, &kernels) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (total_tokens == 0 || batch == 0) return done(cudaSuccess, kernels);
  const cudaError_t e = gdn::launch_ssm_extend(p, L.rule, s, &kernels);
  return done(e, kernels);
}

gdn_status gdn_ssm_step(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, gdn_dtype dtype, const float* A,
                        const void* B, int64_t B_stride, const void* C, int64_t C_stride, const float* D, const void* z,
                        int64_t z_stride, const float* dt_bias, float* state_pool, int64_t pool_size,
                        const int64_t* cache_indices, int32_t batch, void* out, int32_t channels, int32_t groups,
                        int32_t states, int32_t softplus, int32_t* device_status, void* stream) {
  NvtxRange range("gdn_ssm_step");
  if (batch > kMaxStepBatch || !ssm_shape_ok(batch, batch, channels, groups, states)) return GDN_ERR_INVALID_ARG;
  const SsmArgs a{x, dt, B, C, z, x_stride, dt_stride, B_stride, C_stride, z_stride, A, D, dt_bias,
                  (int32_t)dtype, channels, groups, states, softplus};
  if (!ssm_args_ok(a, batch > 0)) return GDN_ERR_INVALID_ARG;
  if (!device_status || !aligned_to(device_status, 4)) return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!state_pool || !cache_indices || pool_size <= 0 || !aligned_to(state_pool, 4) || !out ||
                    !aligned_to(out, gdn::op_dtype_size(dtype))))
    return GDN_ERR_INVALID_ARG;
  if (!ssm_shape_built(states) || (int64_t)batch * ((channels + 31) / 32) > kMaxBlocks) return GDN_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  gdn::SsmParams p = ssm_params(a);
  p.pool = state_pool;
  p.cache_indices = cache_indices;
  p.out = out;
  p.T = batch;
  p.B = batch;
  p.status = device_status;
  p.pool_size = pool_size;
  p.check = gdn::slot_check(batch, pool_size, (int64_t)batch * channels * states * 8);
  return run_step(cache_indices, batch, pool_size, device_status, p.check, s, [&] { return gdn::launch_ssm_step(p, s); });
}

gdn_status gdn_ssm_backward(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, gdn_dtype dtype, const float* A,
                            const void* B, int64_t B_stride, const void* C, int64_t C_stride, const float* D, const void* z,
                            int64_t z_stride, const float* dt_bias, const float* state_pool, int64_t pool_size,
                            const int64_t* cache_indices, const int64_t* cu_seqlens, int32_t batch, const void* d_out,
                            int64_t d_out_stride, const float* d_state, void* dx, void* ddt, float* dA, void* dB, void* dC,
                            float* dD, void* dz, float* ddt_bias, float* d_state_pool, int64_t total_tokens, int32_t channels,
                            int32_t groups, int32_t states, int32_t softplus, void* workspace, size_t workspace_bytes,
                            void* stream) {
  NvtxRange range("gdn_ssm_backward");
  if (!ssm_shape_ok(total_tokens, batch, channels, groups, states) || !cu_seqlens) return GDN_ERR_INVALID_ARG;
  const SsmArgs a{x, dt, B, C, z, x_stride, dt_stride, B_stride, C_stride, z_stride, A, D, dt_bias,
                  (int32_t)dtype, channels, groups, states, softplus};
  if (!ssm_args_ok(a, total_tokens > 0)) return GDN_ERR_INVALID_ARG;
  if (!dA || !aligned_to(dA, 4) || !aligned_to(dD, 4) || !aligned_to(ddt_bias, 4)) return GDN_ERR_INVALID_ARG;
  if (batch > 0 && (!state_pool || !cache_indices || pool_size <= 0 || !d_state_pool || !aligned_to(state_pool, 4) ||
                    !aligned_to(d_state, 4) || !aligned_to(d_state_pool, 4)))
    return GDN_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    const uintptr_t size = gdn::op_dtype_size(dtype);
    for (const void* q : {d_out, (const void*)dx, (const void*)ddt, (const void*)dB, (const void*)dC})
      if (!q || !aligned_to(q, size)) return GDN_ERR_INVALID_ARG;
    if ((z != nullptr) != (dz != nullptr) || !aligned_to(dz, size) || !stride_ok(d_out_stride, channels))
      return GDN_ERR_INVALID_ARG;
  }
  const size_t need = gdn_ssm_backward_workspace_size(total_tokens, batch, channels, groups, states);
  if (need == 0) return GDN_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const SsmLayout L = ssm_layout(total_tokens, batch, channels, groups, states, true);
  auto f = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  gdn::SsmParams p = ssm_params(a);
  p.pool = const_cast<float*>(state_pool);  // read only in the backward kernels
  p.cache_indices = cache_indices;
  p.cu_seqlens = cu_seqlens;
  p.T = batch > 0 ? total_tokens : 0;
  p.B = batch;
  p.plan = gdn::plan_at(ws, L.plan);
  p.max_segs = L.rule.max_segs;
  p.seg_state = f(L.seg_state);
  p.seg_delta = f(L.seg_delta);
  p.seg_grad = f(L.seg_grad);
  p.ckpt = f(L.ckpt);
  p.ckpt_delta = f(L.ckpt_delta);
  p.partial_bc = f(L.partial_bc);
  p.partial_A = f(L.partial_A);
  p.partial_par = f(L.partial_par);
  p.d_out = d_out;
  p.d_stride = d_out_stride;
  p.d_state = d_state;
  p.dx = dx;
  p.ddt = ddt;
  p.dB = dB;
  p.dC = dC;
  p.dz = dz;
  p.dA = dA;
  p.dD = dD;
  p.ddt_bias = ddt_bias;
  p.d_pool = d_state_pool;
  int kernels = 0;
  if (gdn::launch_plan(p.plan, cu_seqlens, cache_indices, batch, total_tokens, pool_size, L.rule, s, &kernels) != cudaSuccess)
    return GDN_ERR_CUDA;
  const cudaError_t e = gdn::launch_ssm_backward(p, s, &kernels);
  return done(e, kernels);
}

gdn_status gdn_layer_norm(const void* x, int64_t x_stride, gdn_dtype dtype, const float* weight, const float* bias, void* out,
                          float* mean, float* rstd, int64_t rows, int32_t columns, float eps, void* stream) {
  NvtxRange range("gdn_layer_norm");
  if (rows < 0 || columns <= 0 || !(eps >= 0.f) || !gdn::op_dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  const uintptr_t size = gdn::op_dtype_size(dtype);
  if (!aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return GDN_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !out || !aligned_to(x, size) || !aligned_to(out, size) || !stride_ok(x_stride, columns) ||
                   (mean == nullptr) != (rstd == nullptr)))
    return GDN_ERR_INVALID_ARG;
  if (columns > kMaxColumns) return GDN_ERR_UNSUPPORTED;
  if (rows == 0) return GDN_OK;
  gdn::NormParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.out = out;
  p.mean = mean;
  p.rstd = rstd;
  p.rows = rows;
  p.x_stride = x_stride;
  p.columns = columns;
  p.eps = eps;
  p.dtype = dtype;
  return done(gdn::launch_norm(p, static_cast<cudaStream_t>(stream)), 1);
}

size_t gdn_layer_norm_backward_workspace_size(int64_t rows, int32_t columns) {
  return rows < 0 || columns <= 0 || columns > kMaxColumns ? 0 : gdn::norm_backward_workspace(rows, columns);
}

gdn_status gdn_layer_norm_backward(const void* d_out, int64_t d_out_stride, const void* x, int64_t x_stride, gdn_dtype dtype,
                                   const float* weight, const float* mean, const float* rstd, void* dx, float* dweight,
                                   float* dbias, int64_t rows, int32_t columns, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  NvtxRange range("gdn_layer_norm_backward");
  if (rows < 0 || columns <= 0 || !gdn::op_dtype_ok(dtype)) return GDN_ERR_INVALID_ARG;
  const uintptr_t size = gdn::op_dtype_size(dtype);
  if (!aligned_to(weight, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4)) return GDN_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !d_out || !dx || !mean || !rstd || !aligned_to(x, size) || !aligned_to(d_out, size) ||
                   !aligned_to(dx, size) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !stride_ok(x_stride, columns) ||
                   !stride_ok(d_out_stride, columns)))
    return GDN_ERR_INVALID_ARG;
  if (columns > kMaxColumns) return GDN_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, gdn::norm_backward_workspace(rows, columns))) return GDN_ERR_WORKSPACE;
  gdn::NormParams p{};
  p.x = x;
  p.weight = weight;
  p.mean = const_cast<float*>(mean);  // read only in the backward kernels
  p.rstd = const_cast<float*>(rstd);
  p.rows = rows;
  p.x_stride = x_stride;
  p.columns = columns;
  p.dtype = dtype;
  p.d_out = d_out;
  p.d_stride = d_out_stride;
  p.dx = dx;
  p.dweight = dweight;
  p.dbias = dbias;
  p.partial = static_cast<float*>(workspace);
  int kernels = 0;
  const cudaError_t e = gdn::launch_norm_backward(p, static_cast<cudaStream_t>(stream), &kernels);
  return done(e, kernels);
}

}  // extern "C"
