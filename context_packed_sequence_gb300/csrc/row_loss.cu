// Losses over rows of logits: label log-probabilities, the clipped policy loss
// and distillation from a teacher's top logits, the last two with the
// gradient of the logits in the same pass.
#include <algorithm>

#include "loss_internal.cuh"

namespace thd {
namespace {

constexpr int kPlainThreads = 512;

__device__ __forceinline__ SoftmaxStat block_join(SoftmaxStat t, LogitScale c, SoftmaxStat* tmp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  t = warp_join(t, c);
  if (lane == 0) tmp[wid] = t;
  __syncthreads();
  t = lane < nw ? tmp[lane] : empty_stat();
  t = warp_join(t, c);  // every warp: the same order, the same bits
  __syncthreads();
  return t;
}

__device__ __forceinline__ float block_sum(float v, float* tmp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) tmp[wid] = v;
  __syncthreads();
  v = warp_sum(lane < nw ? tmp[lane] : 0.0f);
  __syncthreads();
  return v;
}

// Any row, one block each: the logits are read twice from memory, element by
// element.  Takes what the kernel above it cannot: rows longer than a
// cluster's shared memory.
template <typename T, int kMode>
__global__ void __launch_bounds__(kPlainThreads) row_plain_kernel(const __grid_constant__ RowArgs a) {
  pdl_wait_then_release();
  __shared__ SoftmaxStat stats[32];
  __shared__ float sums[32];
  __shared__ RowHead head;
  __shared__ int32_t stop;
  __shared__ __align__(16) unsigned char teacher_mem[kMode == ROW_DISTILL ? sizeof(Teacher) : 16];
  Teacher& te = *reinterpret_cast<Teacher*>(teacher_mem);
  const int64_t t = blockIdx.x;
  if (threadIdx.x == 0) {
    stop = status_load(a.status);
    if (!stop) head = row_head<T, kMode>(a, t);
  }
  __syncthreads();
  if (stop) return;
  const RowHead h = head;
  const T* z = static_cast<const T*>(a.logits) + t * a.stride;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
  const uint32_t V = a.vocab, step = blockDim.x;
  if (h.weight == 0.0f) {
    if (threadIdx.x == 0) write_idle_row<kMode>(a, t);
    if (dz)
      for (uint32_t v = threadIdx.x; v < V; v += step) dz[v] = from_float<T>(0.0f);
    return;
  }
  SoftmaxStat st = empty_stat();
  for (uint32_t v = threadIdx.x; v < V; v += step) {
    const float x = to_float(z[v]);
    if (x > st.m) {
      st.s = rescaled(st.m, st.s, x, a.scale);
      st.m = x;
    }
    st.s += exp_scaled(x - softmax_shift(st.m), a.scale);
  }
  if (kMode == ROW_DISTILL && threadIdx.x < 32) load_teacher(a, t, te, true);
  st = block_join(st, a.scale, stats);
  RowGrad g = {};
  if (kMode == ROW_SCORE) {
    if (threadIdx.x == 0) write_score(a, t, h, st);
    return;
  }
  if (kMode == ROW_POLICY) g = policy_row(a, t, h, st, threadIdx.x == 0);
  const RowNorm norm = row_norm(st);
  float fix[kMaxTeacher / kPlainThreads];  // gradients in the entries' places
  if (kMode == ROW_DISTILL) {
    const float gs = a.grad_scale * h.weight * a.scale.tau;
    const bool empty = stat_is_empty(st);
    g.k = empty ? 0.0f : gs * te.mass / st.s;
    float loss = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxTeacher / kPlainThreads; ++j) {
      const int k = threadIdx.x + j * kPlainThreads;
      fix[j] = 0.0f;
      if (k >= a.teacher_count || te.id[k] < 0) continue;
      const Pair lp = entry_logprob(to_float(z[te.id[k]]), empty, norm, a.scale);
      if (te.q[k] != 0.0f) loss += te.q[k] * ((te.lq[k] - lp.hi) - lp.lo);
      float q = 0.0f;  // an id may come more than once
      for (int i = 0; i < a.teacher_count; ++i) q += te.id[i] == te.id[k] ? te.q[i] : 0.0f;
      fix[j] = empty ? 0.0f : gs * (te.mass * expf(lp.hi + lp.lo) - q);
    }
    loss = block_sum(loss, sums);
    if (threadIdx.x == 0)
      a.token_losses[t] = te.mass == 0.0f ? 0.0f : loss * (a.scale.tau * a.scale.tau);
  }
  if (!dz) return;
  for (uint32_t v = threadIdx.x; v < V; v += step) {
    const float x = to_float(z[v]) - norm.shift;
    float d = g.k * ex2(x * a.scale.hi);
    if (kMode == ROW_POLICY && static_cast<int32_t>(v) == h.label) d = g.at_label;
    dz[v] = from_float<T>(d);
  }
  if (kMode == ROW_DISTILL) {
    __syncthreads();  // after the block's own values of the row
#pragma unroll
    for (int j = 0; j < kMaxTeacher / kPlainThreads; ++j) {
      const int k = threadIdx.x + j * kPlainThreads;
      if (k < a.teacher_count && te.id[k] >= 0) dz[te.id[k]] = from_float<T>(fix[j]);
    }
  }
}

template <typename T>
thd_status_t launch_mode(RowMode mode, const RowArgs& a, cudaStream_t s) {
  cudaError_t e;
  const dim3 grid(static_cast<unsigned>(a.rows));
  if (mode == ROW_SCORE) e = launch_pdl(row_plain_kernel<T, ROW_SCORE>, grid, dim3(kPlainThreads), 0, s, a);
  else if (mode == ROW_POLICY) e = launch_pdl(row_plain_kernel<T, ROW_POLICY>, grid, dim3(kPlainThreads), 0, s, a);
  else e = launch_pdl(row_plain_kernel<T, ROW_DISTILL>, grid, dim3(kPlainThreads), 0, s, a);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return THD_ERR_CUDA;
  }
  return THD_OK;
}

// dz_v = g_t (1[v = label] - p_v) / tau from the saved log-sum-exp
template <typename T>
__global__ void __launch_bounds__(kPlainThreads)
    logprobs_backward_kernel(const __grid_constant__ RowArgs a, const float* lse, const float* dlogprobs) {
  pdl_wait_then_release();
  __shared__ int32_t stop;
  const int64_t t = blockIdx.x;
  const uint32_t V = a.vocab, step = blockDim.x;
  const int32_t label = a.labels[t];
  const float up = dlogprobs[t];
  const bool bad = up != 0.0f && (label < 0 || label >= a.vocab);
  if (threadIdx.x == 0) {
    stop = status_load(a.status);
    if (bad && !stop) status_set(a.status, THD_ERR_INDEX_RANGE);
  }
  __syncthreads();
  if (stop) return;
  const T* z = static_cast<const T*>(a.logits) + t * a.stride;
  T* dz = static_cast<T*>(a.dlogits) + t * a.dstride;
  const float l = lse[t];
  if (up == 0.0f || bad || l == -INFINITY) {
    for (uint32_t v = threadIdx.x; v < V; v += step) dz[v] = from_float<T>(0.0f);
    return;
  }
  const float g = up * a.grad_scale * a.scale.inv_tau;
  // z/tau - lse = (z - lse tau)/tau; what rounds off the product goes into the factor
  const float top = l * a.scale.tau;
  const float rest = fabsf(top) < INFINITY ? fmaf(l, a.scale.tau, -top) : 0.0f;
  const float k = g * ex2(-rest * a.scale.hi);
  for (uint32_t v = threadIdx.x; v < V; v += step) {
    const float d = k * exp_scaled(to_float(z[v]) - top, a.scale);
    dz[v] = from_float<T>(static_cast<int32_t>(v) == label ? g - d : -d);
  }
}

}  // namespace

thd_status_t launch_row_loss(RowMode mode, int32_t dtype, const RowArgs& a, cudaStream_t s) {
  if (a.rows == 0) return THD_OK;
  if (dtype == THD_DTYPE_BF16) return launch_mode<__nv_bfloat16>(mode, a, s);
  if (dtype == THD_DTYPE_F16) return launch_mode<__half>(mode, a, s);
  return launch_mode<float>(mode, a, s);
}

thd_status_t launch_logprobs_backward(int32_t dtype, const RowArgs& a, const float* lse, const float* dlogprobs,
                                      cudaStream_t s) {
  if (a.rows == 0) return THD_OK;
  const dim3 grid(static_cast<unsigned>(a.rows)), block(kPlainThreads);
  cudaError_t e;
  if (dtype == THD_DTYPE_BF16) e = launch_pdl(logprobs_backward_kernel<__nv_bfloat16>, grid, block, 0, s, a, lse, dlogprobs);
  else if (dtype == THD_DTYPE_F16) e = launch_pdl(logprobs_backward_kernel<__half>, grid, block, 0, s, a, lse, dlogprobs);
  else e = launch_pdl(logprobs_backward_kernel<float>, grid, block, 0, s, a, lse, dlogprobs);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return THD_ERR_CUDA;
  }
  return THD_OK;
}

}  // namespace thd
