// Losses over rows of logits: label log-probabilities, the clipped policy loss
// and distillation from a teacher's top logits, the last two with the
// gradient of the logits in the same pass.
//
// A row's gradient needs the row's own softmax statistics and a few scalars,
// so a row is read once, kept on the chip until its statistics are known, and
// its gradient written once.  A cluster of 1 to 8 blocks shares a row: each
// holds a slice of it in shared memory, and they exchange their maxima and
// sums through distributed shared memory.
#include <algorithm>

#include "loss_internal.cuh"

namespace thd {
namespace {

// ---------------------------------------------------------------------------
// 16-byte vectors of logits
// ---------------------------------------------------------------------------

// Two floats in one 64-bit register for the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t x) {
  const float2 v = unpack2(x);
  return pack2(ex2(v.x), ex2(v.y));
}

// 32-bit words of a vector by a compile-time index, so that it stays in registers.
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void set_word(uint4& v, int i, uint32_t w) {
  if (i == 0) v.x = w;
  else if (i == 1) v.y = w;
  else if (i == 2) v.z = w;
  else v.w = w;
}

// A vector's pairs of elements as floats, their maximum in the elements' own
// type, and pairs and elements rounded back into it.
template <typename T>
struct Word;

struct Halves {  // two elements a word
  static constexpr int kElems = 8;  // per vector
  static constexpr int kPairs = 4;
  __device__ static __forceinline__ void store_elem(void* p, const uint4& v, int j) {
    *static_cast<uint16_t*>(p) = static_cast<uint16_t>(word(v, j >> 1) >> (16 * (j & 1)));
  }
  // element j (not a constant) of v := the 16 bits
  __device__ static __forceinline__ void set_bits(uint4& v, int j, uint16_t bits) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = word(v, i);
      if ((j >> 1) == i) set_word(v, i, j & 1 ? (w & 0xffffu) | (uint32_t(bits) << 16) : (w & 0xffff0000u) | bits);
    }
  }
};

template <>
struct Word<__nv_bfloat16> : Halves {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static __forceinline__ uint64_t pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static __forceinline__ float top(uint32_t m) {
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ static __forceinline__ void set_pair(uint4& v, int i, uint64_t p) {
    const float2 f = unpack2(p);
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f.y), "f"(f.x));
    set_word(v, i, w);
  }
  __device__ static __forceinline__ void set_elem(uint4& v, int j, float x) {
    set_bits(v, j, __bfloat16_as_ushort(__float2bfloat16_rn(x)));
  }
};

template <>
struct Word<__half> : Halves {
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  __device__ static __forceinline__ uint64_t pair(const uint4& v, int i) {
    const uint32_t w = word(v, i);
    const float2 f = __half22float2(__halves2half2(__ushort_as_half(static_cast<uint16_t>(w)),
                                                   __ushort_as_half(static_cast<uint16_t>(w >> 16))));
    return pack2(f.x, f.y);
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static __forceinline__ float top(uint32_t m) {
    return fmaxf(__half2float(__ushort_as_half(static_cast<uint16_t>(m))),
                 __half2float(__ushort_as_half(static_cast<uint16_t>(m >> 16))));
  }
  __device__ static __forceinline__ void set_pair(uint4& v, int i, uint64_t p) {
    const float2 f = unpack2(p);
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f.y), "f"(f.x));
    set_word(v, i, w);
  }
  __device__ static __forceinline__ void set_elem(uint4& v, int j, float x) {
    set_bits(v, j, __half_as_ushort(__float2half_rn(x)));
  }
};

template <>
struct Word<float> {
  static constexpr int kElems = 4;
  static constexpr int kPairs = 2;
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static __forceinline__ uint64_t pair(const uint4& v, int i) {
    return pack2(__uint_as_float(word(v, 2 * i)), __uint_as_float(word(v, 2 * i + 1)));
  }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static __forceinline__ float top(uint32_t m) { return __uint_as_float(m); }
  __device__ static __forceinline__ void set_pair(uint4& v, int i, uint64_t p) {
    const float2 f = unpack2(p);
    set_word(v, 2 * i, __float_as_uint(f.x));
    set_word(v, 2 * i + 1, __float_as_uint(f.y));
  }
  __device__ static __forceinline__ void store_elem(void* p, const uint4& v, int j) {
    *static_cast<uint32_t*>(p) = word(v, j);
  }
  __device__ static __forceinline__ void set_elem(uint4& v, int j, float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j == i) set_word(v, i, __float_as_uint(x));
  }
};

// Maximum of kVecs vectors, in the elements' type: NaNs are passed over (the
// sum of exponentials shows them).
template <typename T, int kVecs>
__device__ __forceinline__ float vector_max(const uint4 (&v)[kVecs]) {
  uint32_t m = Word<T>::kNegInf;
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
    m = Word<T>::max2(Word<T>::max2(Word<T>::max2(m, v[u].x), Word<T>::max2(v[u].y, v[u].z)), v[u].w);
  return Word<T>::top(m);
}

// A thread's running softmax statistics over batches of logits: the maximum
// of a batch first, so that a rescaling costs one branch a batch.
struct ThreadStat {
  float m = -INFINITY;
  Pair s = {0.0f, 0.0f};

  __device__ __forceinline__ void raise(float to, LogitScale c) {
    if (to > m) {
      s = rescaled(m, s, to, c);
      m = to;
    }
  }
  __device__ __forceinline__ void add_one(float z, LogitScale c) {
    raise(z, c);
    s.hi += exp_scaled(z - softmax_shift(m), c);
  }
  template <typename T, int kVecs>
  __device__ __forceinline__ void add_vectors(const uint4 (&v)[kVecs], LogitScale c) {
    raise(vector_max<T, kVecs>(v), c);
    const float shift = softmax_shift(m);
    const uint64_t neg = pack2(-shift, -shift), hi = pack2(c.hi, c.hi), lo = pack2(c.lo, c.lo);
    uint64_t acc[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
#pragma unroll
      for (int i = 0; i < Word<T>::kPairs; ++i) {
        const uint64_t d = add2(Word<T>::pair(v[u], i), neg);
        acc[i & 1] = add2(acc[i & 1], ex2_2(fma2(d, hi, mul2(d, lo))));
      }
    const float2 t = unpack2(add2(acc[0], acc[1]));
    s.hi += t.x + t.y;
  }
};

__device__ __forceinline__ float warp_max_one(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// The block's statistics, in every thread of its first warp.  `failed` comes
// back true in every thread when it was in any.
__device__ __forceinline__ SoftmaxStat block_stat(ThreadStat t, LogitScale c, float* maxima, Pair* sums, bool* failed) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float m = warp_max_one(t.m);
  if (lane == 0) maxima[wid] = m;
  *failed = __syncthreads_or(*failed);
  m = maxima[0];
  for (int w = 1; w < nw; ++w) m = fmaxf(m, maxima[w]);
  const Pair own = unbiased_sum(t.s.hi);
  Pair s = rescaled(t.m, {t.s.hi, t.s.lo + own.lo}, m, c);
  // high and low parts each on their own: a few roundings of 6e-8 at random
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s.hi += __shfl_xor_sync(kFullMask, s.hi, o);
    s.lo += __shfl_xor_sync(kFullMask, s.lo, o);
  }
  if (lane == 0) sums[wid] = s;
  __syncthreads();
  if (wid == 0) {
    s = {0.0f, 0.0f};
    for (int w = 0; w < nw; ++w) s = add(s, sums[w]);
  }
  return {m, s};
}

// A row's gradient as its threads need it, from the first warp to the block.
struct RowResult {
  SoftmaxStat st;
  RowGrad g;
  float mass;
  bool failed;
};

// kThreads threads; every entry of the teacher is some thread's.
template <int kThreads>
struct EntryFix {
  static constexpr int kPer = (kMaxTeacher + kThreads - 1) / kThreads;
  float at[kPer];  // gradient in the entry's place
};

// Loss terms of the entries for which `mine(id)` and their gradients;
// `logit(id)` reads the row.  Returns this thread's part of the loss / tau^2.
template <int kThreads, class Mine, class Logit>
__device__ __forceinline__ float teacher_entries(const RowArgs& a, const Teacher& te, float weight, const RowResult& r,
                                                 Mine mine, Logit logit, EntryFix<kThreads>& fix) {
  const RowNorm norm = row_norm(r.st);
  const float gs = a.grad_scale * weight * a.scale.tau;
  const bool empty = stat_is_empty(r.st);
  float loss = 0.0f;
#pragma unroll
  for (int j = 0; j < EntryFix<kThreads>::kPer; ++j) {
    const int k = threadIdx.x + j * kThreads;
    fix.at[j] = 0.0f;
    if (k >= a.teacher_count) break;
    const int32_t id = te.id[k];
    if (id < 0 || !mine(id)) continue;
    const Pair lp = entry_logprob(logit(id), empty, norm, a.scale);
    if (te.q[k] != 0.0f) loss += te.q[k] * ((te.lq[k] - lp.hi) - lp.lo);
    fix.at[j] = empty ? 0.0f : gs * (r.mass * expf(lp.hi + lp.lo) - entry_mass(te, id, a.teacher_count));
  }
  return loss;
}

template <typename T, int kThreads, class Mine>
__device__ __forceinline__ void write_entries(const RowArgs& a, const Teacher& te, T* dz, Mine mine,
                                              const EntryFix<kThreads>& fix) {
#pragma unroll
  for (int j = 0; j < EntryFix<kThreads>::kPer; ++j) {
    const int k = threadIdx.x + j * kThreads;
    if (k >= a.teacher_count) break;
    const int32_t id = te.id[k];
    if (id >= 0 && mine(id)) dz[id] = from_float<T>(fix.at[j]);
  }
}

__device__ __forceinline__ float block_sum(float v, float* tmp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  if (lane == 0) tmp[wid] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < nw; ++w) v += tmp[w];
  return v;
}

// ---------------------------------------------------------------------------
// rows shared by a cluster
// ---------------------------------------------------------------------------

constexpr int kVecsPerStep = 4;  // vectors a thread holds in registers at a time
constexpr int kMaxChunks = 16;   // parts of a slice that arrive on their own
constexpr int kMaxCluster = 8;   // largest portable cluster
constexpr int kMaxSlice = 208 * 1024;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every block of the cluster runs, and its barriers are set up, once each has
// arrived (after its fence.mbarrier_init) and this one has waited.  By whole
// warps.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float4 into block `rank`'s shared memory, at this block's addresses of the
// slot and of the barrier that counts its 16 bytes.
__device__ __forceinline__ void cluster_send(const float4* at, const uint64_t* bar, uint32_t rank, float4 v) {
  uint32_t slot, counter;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(slot) : "r"(smem_addr(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(counter) : "r"(smem_addr(bar)), "r"(rank));
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(slot),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(counter)
      : "memory");
}
// Bounded wait for what the cluster sends here (like mbar_wait).
__device__ __forceinline__ bool cluster_receive(uint64_t* bar) {
  for (int it = 0; it < kWaitLimit; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_addr(bar))
        : "memory");
    if (done) return true;
  }
  return false;
}

// A row's slice [first, first + count) of whole 16-byte vectors, counted from
// the row's first 16-byte boundary; the elements before it (head) and after
// the last whole vector (tail) are `edge` elements of the first and the last
// block of the cluster, one thread each.
struct Slice {
  int32_t head;          // elements before the first whole vector of the row
  int32_t first, count;  // this block's vectors
  int32_t edge_at, edge_count;
};

template <typename T>
__device__ __forceinline__ Slice row_slice(const T* z, int32_t V, int32_t rank, int32_t cluster_log2) {
  constexpr int N = Word<T>::kElems;
  Slice s;
  const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) & 15u);
  s.head = min(V, static_cast<int32_t>(((16u - mis) & 15u) / sizeof(T)));
  const int32_t cluster = 1 << cluster_log2;
  const int32_t vecs = static_cast<int32_t>(static_cast<uint32_t>(V - s.head) / N);
  const int32_t per = (vecs + cluster - 1) >> cluster_log2;
  s.first = min(vecs, rank * per);
  s.count = min(vecs, s.first + per) - s.first;
  const int32_t tail = s.head + vecs * N;
  s.edge_at = 0;
  s.edge_count = rank == 0 ? s.head : 0;
  if (rank == cluster - 1 && tail < V) {
    // one block may have both: its edge is then handled as two runs below
    if (s.edge_count == 0) {
      s.edge_at = tail;
      s.edge_count = V - tail;
    } else {
      s.edge_count += V - tail;  // edge_index() skips the vectors between
    }
  }
  return s;
}

// i-th edge element of the block: the head's, then the tail's
__device__ __forceinline__ int32_t edge_index(const Slice& s, int32_t i, int32_t V) {
  if (s.edge_at > 0) return s.edge_at + i;
  return i < s.head ? i : V - (s.edge_count - i);
}

template <typename T, int kMode, int kThreads>
__global__ void __launch_bounds__(kThreads) row_cluster_kernel(const __grid_constant__ RowArgs a, int32_t cluster_log2) {
  constexpr int N = Word<T>::kElems;
  constexpr int kStep = kThreads * kVecsPerStep;  // vectors of a chunk
  constexpr uint32_t kNone = Word<T>::kNegInf;
  extern __shared__ __align__(128) unsigned char dynamic[];
  __shared__ uint64_t bars[kMaxChunks];
  __shared__ uint64_t stat_bar, loss_bar;
  __shared__ float maxima[kThreads / 32];
  __shared__ Pair sums[kThreads / 32];
  __shared__ __align__(16) float4 inbox[kMaxCluster];     // each block's statistics
  __shared__ __align__(16) float4 loss_box[kMaxCluster];  // each block's part of the distillation loss
  __shared__ RowHead head;
  __shared__ RowResult result;
  __shared__ int32_t stop;

  pdl_wait_then_release();
  const int tid = threadIdx.x;
  const int32_t cluster = 1 << cluster_log2;
  const int32_t rank = cluster > 1 ? static_cast<int32_t>(cluster_rank()) : 0;
  const int64_t t = blockIdx.x >> cluster_log2;
  const T* z = static_cast<const T*>(a.logits) + t * a.stride;
  T* dz = a.dlogits ? static_cast<T*>(a.dlogits) + t * a.dstride : nullptr;
  const Slice sl = row_slice(z, a.vocab, rank, cluster_log2);
  uint4* buf = reinterpret_cast<uint4*>(dynamic);
  const int32_t chunks = (sl.count + kStep - 1) / kStep;

  bool loading = false;
  if (tid == 0) {
    const int32_t s = status_load(a.status);
    float w;
    if (kMode == ROW_SCORE) w = (!a.mask || a.mask[t]) ? 1.0f : 0.0f;
    else w = a.weights[t];
    stop = s;
    loading = s == 0 && w != 0.0f;
    for (int i = 0; i < chunks; ++i) mbar_init(&bars[i], 1);
    if (cluster > 1) {
      mbar_init(&stat_bar, 1);
      mbar_init(&loss_bar, 1);
    }
    mbar_init_fence();
    if (loading) {
      const uint4* zv = reinterpret_cast<const uint4*>(z + sl.head) + sl.first;
      for (int i = 0; i < chunks; ++i) {
        const int32_t n = min(kStep, sl.count - i * kStep) * 16;
        mbar_arrive_expect_tx(&bars[i], n);
        bulk_load(buf + i * kStep, zv + i * kStep, n, &bars[i]);
      }
    }
    if (cluster > 1) {
      mbar_arrive_expect_tx(&stat_bar, 16 * cluster);
      if (kMode == ROW_DISTILL && rank == 0) mbar_arrive_expect_tx(&loss_bar, 16 * cluster);
    }
  } else if (tid == 32) {
    head = row_head<T, kMode>(a, t);
  }
  if (cluster > 1) cluster_arrive();
  __syncthreads();
  const RowHead h = head;
  if (cluster > 1) cluster_wait();
  // Every block of the cluster reads the same weight and label, so all of
  // them take this branch or none; the status word may change meanwhile, so
  // a block that saw it set goes on and tells the others.
  if (h.weight == 0.0f) {
    if (loading)  // a bad label: the copies have to land before the block ends
      for (int i = 0; i < chunks; ++i) mbar_wait(&bars[i], 0);
    if (stop) return;
    if (tid == 0 && rank == 0) write_idle_row<kMode>(a, t);
    if (!dz) return;
    const T zero = from_float<T>(0.0f);
    T* dv = dz + sl.head + static_cast<int64_t>(sl.first) * N;
    if ((reinterpret_cast<uintptr_t>(dv) & 15u) == 0) {
#pragma unroll 4
      for (int32_t i = tid; i < sl.count; i += kThreads) reinterpret_cast<uint4*>(dv)[i] = make_uint4(0, 0, 0, 0);
    } else {
      for (int64_t i = tid; i < static_cast<int64_t>(sl.count) * N; i += kThreads) dv[i] = zero;
    }
    if (tid < sl.edge_count) dz[edge_index(sl, tid, a.vocab)] = zero;
    return;
  }

  bool failed = stop != 0;
  const Teacher te = teacher_at(dynamic + static_cast<size_t>(sl.count) * 16, a.teacher_count);
  float mass = 0.0f;
  if (kMode == ROW_DISTILL && tid < 32 && !failed) mass = load_teacher(a, t, te, rank == 0);

  // the slice's statistics, chunk by chunk as they land
  ThreadStat ts;
  if (!failed) {
    const uint4* from = buf + tid;
    for (int i = 0; i < chunks; ++i, from += kStep) {
      if (!mbar_wait(&bars[i], 0)) {
        failed = true;
        break;
      }
      const int32_t left = sl.count - i * kStep;
      uint4 v[kVecsPerStep];
      if (left >= kStep) {
#pragma unroll
        for (int u = 0; u < kVecsPerStep; ++u) v[u] = from[u * kThreads];
      } else {
#pragma unroll
        for (int u = 0; u < kVecsPerStep; ++u)
          v[u] = u * kThreads + tid < left ? from[u * kThreads] : make_uint4(kNone, kNone, kNone, kNone);
      }
      ts.add_vectors<T, kVecsPerStep>(v, a.scale);
    }
    if (tid < sl.edge_count) ts.add_one(to_float(z[edge_index(sl, tid, a.vocab)]), a.scale);
    if (failed) status_set(a.status, THD_ERR_TIMEOUT);
  }
  SoftmaxStat st = block_stat(ts, a.scale, maxima, sums, &failed);
  if (tid < 32) {
    bool off = failed;
    if (cluster > 1) {
      if (tid < cluster)
        cluster_send(&inbox[rank], &stat_bar, tid, make_float4(st.m, st.s.hi, st.s.lo, failed ? 1.0f : 0.0f));
      if (!cluster_receive(&stat_bar)) {
        off = true;
        status_set(a.status, THD_ERR_TIMEOUT);
      }
      float m = inbox[0].x;
      for (int c = 1; c < cluster; ++c) m = fmaxf(m, inbox[c].x);
      Pair s = {0.0f, 0.0f};
      for (int c = 0; c < cluster; ++c) {
        off |= inbox[c].w != 0.0f;
        s = add(s, rescaled(inbox[c].x, {inbox[c].y, inbox[c].z}, m, a.scale));
      }
      st = {m, s};
    }
    RowResult r;
    r.st = st;
    r.mass = mass;
    r.failed = off;
    r.g = {0.0f, 0.0f};
    if (!off) {
      if (kMode == ROW_SCORE) {
        if (tid == 0 && rank == 0) write_score(a, t, h, st);
      } else if (kMode == ROW_POLICY) {
        r.g = policy_row(a, t, h, st, tid == 0 && rank == 0);
      } else if (!stat_is_empty(st)) {
        r.g.k = a.grad_scale * h.weight * a.scale.tau * mass / st.s.hi;
      }
    }
    if (tid == 0) result = r;
    if (off && loading)  // no block of the cluster writes; the copies have to land
      for (int i = 0; i < chunks; ++i) mbar_wait(&bars[i], 0);
  }
  if (kMode == ROW_SCORE) return;
  __syncthreads();
  const RowResult r = result;
  if (r.failed) return;
  const int32_t lo_v = sl.head + sl.first * N, hi_v = lo_v + sl.count * N;  // the slice's elements
  const auto mine = [&](int32_t id) {
    return (id >= lo_v && id < hi_v) || (rank == 0 && id < sl.head) ||
           (rank == cluster - 1 && id >= sl.head + (a.vocab - sl.head) / N * N);
  };
  EntryFix<kThreads> fix;
  if (kMode == ROW_DISTILL) {
    const T* held = reinterpret_cast<const T*>(buf);
    const auto logit = [&](int32_t id) { return to_float(id >= lo_v && id < hi_v ? held[id - lo_v] : z[id]); };
    float part = teacher_entries<kThreads>(a, te, h.weight, r, mine, logit, fix);
    part = block_sum(part, maxima);
    if (cluster > 1) {
      if (tid == 0) cluster_send(&loss_box[rank], &loss_bar, 0, make_float4(part, 0.0f, 0.0f, 0.0f));
    } else if (tid == 0) {
      a.token_losses[t] = part * (a.scale.tau * a.scale.tau);
    }
  }
  if (dz) {
    const float shift = softmax_shift(r.st.m);
    const uint64_t neg = pack2(-shift, -shift), hi = pack2(a.scale.hi, a.scale.hi), k2 = pack2(r.g.k, r.g.k);
    const auto gradient = [&](const uint4& v) {
      uint4 d;
#pragma unroll
      for (int j = 0; j < Word<T>::kPairs; ++j)
        Word<T>::set_pair(d, j, mul2(k2, ex2_2(mul2(add2(Word<T>::pair(v, j), neg), hi))));
      return d;
    };
    T* dv = dz + lo_v;
    if ((reinterpret_cast<uintptr_t>(dv) & 15u) == 0) {
      const uint4* from = buf + tid;
      uint4* to = reinterpret_cast<uint4*>(dv) + tid;
      int32_t left = sl.count - tid;
      for (; left > kStep - kThreads; left -= kStep, from += kStep, to += kStep) {
        uint4 v[kVecsPerStep];
#pragma unroll
        for (int u = 0; u < kVecsPerStep; ++u) v[u] = from[u * kThreads];
#pragma unroll
        for (int u = 0; u < kVecsPerStep; ++u) to[u * kThreads] = gradient(v[u]);
      }
      for (; left > 0; left -= kThreads, from += kThreads, to += kThreads) *to = gradient(*from);
    } else {
      // a gradient laid out to another alignment than the logits
      for (int32_t i = tid; i < sl.count; i += kThreads) {
        const uint4 d = gradient(buf[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) Word<T>::store_elem(dv + static_cast<int64_t>(i) * N + j, d, j);
      }
    }
    if (tid < sl.edge_count) {
      const int32_t e = edge_index(sl, tid, a.vocab);
      dz[e] = from_float<T>(r.g.k * ex2((to_float(z[e]) - shift) * a.scale.hi));
    }
    if (kMode == ROW_POLICY && mine(h.label)) {
      // over the value just written, by the thread that wrote it
      const int32_t in = h.label - lo_v;
      int32_t writer = in / N % kThreads;
      if (in < 0) writer = h.label;                                        // the head
      else if (h.label >= hi_v) writer = sl.edge_count - (a.vocab - h.label);  // the tail
      if (tid == writer) dz[h.label] = from_float<T>(r.g.at_label);
    }
    if (kMode == ROW_DISTILL) {
      __syncthreads();  // after the block's own values of the row
      write_entries<T, kThreads>(a, te, dz, mine, fix);
    }
  }
  if (kMode == ROW_DISTILL && cluster > 1 && rank == 0 && tid == 0) {
    if (!cluster_receive(&loss_bar)) {
      status_set(a.status, THD_ERR_TIMEOUT);
      return;
    }
    float part = 0.0f;
    for (int c = 0; c < cluster; ++c) part += loss_box[c].x;
    a.token_losses[t] = part * (a.scale.tau * a.scale.tau);
  }
}

// ---------------------------------------------------------------------------
// rows longer than a cluster's shared memory
// ---------------------------------------------------------------------------

constexpr int kPlainThreads = 512;

// One block a row; the logits are read twice from memory, element by element.
template <typename T, int kMode>
__global__ void __launch_bounds__(kPlainThreads) row_plain_kernel(const __grid_constant__ RowArgs a) {
  extern __shared__ __align__(128) unsigned char dynamic[];
  __shared__ float maxima[kPlainThreads / 32];
  __shared__ Pair sums[kPlainThreads / 32];
  __shared__ RowHead head;
  __shared__ RowResult result;
  __shared__ int32_t stop;
  pdl_wait_then_release();
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
  const uint32_t V = a.vocab, step = kPlainThreads;
  if (h.weight == 0.0f) {
    if (threadIdx.x == 0) write_idle_row<kMode>(a, t);
    if (dz)
      for (uint32_t v = threadIdx.x; v < V; v += step) dz[v] = from_float<T>(0.0f);
    return;
  }
  const Teacher te = teacher_at(dynamic, a.teacher_count);
  float mass = 0.0f;
  if (kMode == ROW_DISTILL && threadIdx.x < 32) mass = load_teacher(a, t, te, true);
  ThreadStat ts;
  constexpr int kBatch = 16;
  for (uint32_t v0 = threadIdx.x; v0 < V; v0 += kBatch * step) {
    float x[kBatch], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t v = v0 + i * step;
      x[i] = v < V ? to_float(z[v]) : -INFINITY;
      top = fmaxf(top, x[i]);
    }
    ts.raise(top, a.scale);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) sum += exp_scaled(x[i] - softmax_shift(ts.m), a.scale);
    ts.s.hi += sum;
  }
  bool failed = false;
  const SoftmaxStat st = block_stat(ts, a.scale, maxima, sums, &failed);
  if (threadIdx.x < 32) {
    RowResult r;
    r.st = st;
    r.mass = mass;
    r.failed = false;
    r.g = {0.0f, 0.0f};
    if (kMode == ROW_SCORE) {
      if (threadIdx.x == 0) write_score(a, t, h, st);
    } else if (kMode == ROW_POLICY) {
      r.g = policy_row(a, t, h, st, threadIdx.x == 0);
    } else if (!stat_is_empty(st)) {
      r.g.k = a.grad_scale * h.weight * a.scale.tau * mass / st.s.hi;
    }
    if (threadIdx.x == 0) result = r;
  }
  if (kMode == ROW_SCORE) return;
  __syncthreads();
  const RowResult r = result;
  const auto all = [](int32_t) { return true; };
  EntryFix<kPlainThreads> fix;
  if (kMode == ROW_DISTILL) {
    const auto logit = [&](int32_t id) { return to_float(z[id]); };
    const float part = block_sum(teacher_entries<kPlainThreads>(a, te, h.weight, r, all, logit, fix), maxima);
    if (threadIdx.x == 0) a.token_losses[t] = part * (a.scale.tau * a.scale.tau);
  }
  if (!dz) return;
  __syncthreads();  // every entry's logit is read before the gradient may take its place
  const float shift = softmax_shift(r.st.m);
  for (uint32_t v = threadIdx.x; v < V; v += step) {
    float d = r.g.k * ex2((to_float(z[v]) - shift) * a.scale.hi);
    if (kMode == ROW_POLICY && static_cast<int32_t>(v) == h.label) d = r.g.at_label;
    dz[v] = from_float<T>(d);
  }
  if (kMode == ROW_DISTILL) {
    __syncthreads();  // after the block's own values of the row
    write_entries<T, kPlainThreads>(a, te, dz, all, fix);
  }
}

thd_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return THD_OK;
  record_cuda_error(e);
  return THD_ERR_CUDA;
}

// Slices of about kSlice bytes let three blocks share an SM, each in a phase
// of its own: one loads while another writes.
constexpr int64_t kSlice = 76 * 1024;
// Below this a slice is not divided further for want of rows.
constexpr int64_t kSmallestSlice = 8 * 1024;

template <typename T, int kMode, int kThreads>
cudaError_t launch_cluster(const RowArgs& a, int32_t cluster, size_t smem, cudaStream_t s) {
  auto* kernel = row_cluster_kernel<T, kMode, kThreads>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(a.rows) * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  int32_t cluster_log2 = 0;
  while ((1 << cluster_log2) < cluster) ++cluster_log2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, cluster_log2);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename T, int kMode>
thd_status_t launch_mode(const RowArgs& a, cudaStream_t s) {
  const int64_t row = static_cast<int64_t>(a.vocab) * sizeof(T);
  const size_t entries = kMode == ROW_DISTILL ? teacher_bytes(a.teacher_count) : 0;
  const int sms = sm_count();
  int32_t cluster = 1;
  while (cluster < kMaxCluster && row > kSlice * cluster) cluster *= 2;
  while (cluster < kMaxCluster && a.rows * static_cast<int64_t>(cluster) < sms && row > 2 * kSmallestSlice * cluster)
    cluster *= 2;
  const int64_t vecs = (row + 15) / 16;
  const int64_t slice = (vecs + cluster - 1) / cluster * 16;
  if (slice + static_cast<int64_t>(entries) > kMaxSlice || a.rows * static_cast<int64_t>(cluster) > INT32_MAX)
    return done(launch_pdl(row_plain_kernel<T, kMode>, dim3(static_cast<unsigned>(a.rows)), dim3(kPlainThreads), entries,
                           s, a));
  const size_t smem = static_cast<size_t>(slice) + entries;
  if (slice <= 8 * 1024) return done(launch_cluster<T, kMode, 128>(a, cluster, smem, s));
  return done(launch_cluster<T, kMode, 256>(a, cluster, smem, s));
}

template <typename T>
thd_status_t launch_type(RowMode mode, const RowArgs& a, cudaStream_t s) {
  if (mode == ROW_SCORE) return launch_mode<T, ROW_SCORE>(a, s);
  if (mode == ROW_POLICY) return launch_mode<T, ROW_POLICY>(a, s);
  return launch_mode<T, ROW_DISTILL>(a, s);
}

// ---------------------------------------------------------------------------
// gradient from saved log-sum-exps
// ---------------------------------------------------------------------------

constexpr int kBackThreads = 256;
constexpr int kBackTile = 2 * kBackThreads * kVecsPerStep;  // vectors of a block

// dz_v = g_t (1[v = label] - p_v) / tau, elementwise: a block takes one tile of
// one row.  Rows go from the last to the first, since those that the forward
// pass read last are still in the L2.  No barriers: every thread reads the
// row's scalars itself.
template <typename T>
__global__ void __launch_bounds__(kBackThreads)
    logprobs_backward_kernel(const __grid_constant__ RowArgs a, const float* lse, const float* dlogprobs, int32_t tiles) {
  constexpr int N = Word<T>::kElems;
  constexpr int kStep = kBackThreads * kVecsPerStep;
  pdl_wait_then_release();
  const int tid = threadIdx.x;
  const uint32_t from_last = blockIdx.x / static_cast<uint32_t>(tiles);
  const int64_t t = a.rows - 1 - static_cast<int32_t>(from_last);
  const int32_t tile = static_cast<int32_t>(blockIdx.x - from_last * tiles);
  const int32_t label = a.labels[t];
  const float up = dlogprobs[t], l = lse[t];
  if (status_load(a.status) != 0) return;
  const T* z = static_cast<const T*>(a.logits) + t * a.stride;
  T* dz = static_cast<T*>(a.dlogits) + t * a.dstride;
  const Slice row = row_slice(z, a.vocab, 0, 0);
  const int32_t first = tile * kBackTile, count = min(kBackTile, row.count - first);
  const int32_t lo_v = row.head + first * N, hi_v = lo_v + max(count, 0) * N;
  const bool bad = up != 0.0f && (label < 0 || label >= a.vocab);
  if (bad && tid == 0) status_set(a.status, THD_ERR_INDEX_RANGE);
  // a row that takes no part: zeros, and its logits are not read
  const bool idle = up == 0.0f || bad || l == -INFINITY;
  const float g = up * a.grad_scale * a.scale.inv_tau;
  // z/tau - lse = (z - top)/tau; what lse tau rounds off goes into the factor
  const float top = l * a.scale.tau;
  const float rest = fabsf(top) < INFINITY ? fmaf(-top, a.scale.inv_tau, l) : 0.0f;
  const float k = -g * ex2(-rest * 1.44269504f);
  // the label's element is written again by the thread that wrote it, from
  // the logit read before
  int32_t writer = -1;
  if (!idle) {
    if (label >= lo_v && label < hi_v) writer = (label - lo_v) / N % kBackThreads;
    else if (tile == 0 && label < row.head) writer = label;
    else if (tile == 0 && label >= row.head + row.count * N) writer = row.edge_count - (a.vocab - label);
  }
  const float z_label = tid == writer ? to_float(z[label]) : 0.0f;

  const uint64_t neg = pack2(-top, -top), hi = pack2(a.scale.hi, a.scale.hi), k2 = pack2(k, k);
  const auto gradient = [&](const uint4& v) {
    uint4 d;
#pragma unroll
    for (int j = 0; j < Word<T>::kPairs; ++j)
      Word<T>::set_pair(d, j, mul2(k2, ex2_2(mul2(add2(Word<T>::pair(v, j), neg), hi))));
    return d;
  };
  const uint4 zeros = make_uint4(0, 0, 0, 0);
  T* dv = dz + lo_v;
  if ((reinterpret_cast<uintptr_t>(dv) & 15u) == 0) {
    const uint4* from = reinterpret_cast<const uint4*>(z + lo_v) + tid;
    uint4* to = reinterpret_cast<uint4*>(dv) + tid;
    int32_t left = count - tid;
    for (; left > kStep - kBackThreads; left -= kStep, from += kStep, to += kStep) {
      uint4 v[kVecsPerStep];
#pragma unroll
      for (int u = 0; u < kVecsPerStep; ++u) v[u] = idle ? zeros : from[u * kBackThreads];
#pragma unroll
      for (int u = 0; u < kVecsPerStep; ++u) to[u * kBackThreads] = idle ? zeros : gradient(v[u]);
    }
    for (; left > 0; left -= kBackThreads, from += kBackThreads, to += kBackThreads)
      *to = idle ? zeros : gradient(*from);
  } else {
    // a gradient laid out to another alignment than the logits
    const uint4* from = reinterpret_cast<const uint4*>(z + lo_v);
    for (int32_t i = tid; i < count; i += kBackThreads) {
      const uint4 d = idle ? zeros : gradient(from[i]);
#pragma unroll
      for (int j = 0; j < N; ++j) Word<T>::store_elem(dv + static_cast<int64_t>(i) * N + j, d, j);
    }
  }
  if (tile == 0 && tid < row.edge_count) {
    const int32_t e = edge_index(row, tid, a.vocab);
    dz[e] = from_float<T>(idle ? 0.0f : k * ex2((to_float(z[e]) - top) * a.scale.hi));
  }
  if (tid == writer) dz[label] = from_float<T>(g + k * exp_scaled(z_label - top, a.scale));
}

template <typename T>
thd_status_t launch_backward(const RowArgs& a, const float* lse, const float* dlogprobs, cudaStream_t s) {
  const int64_t vecs = static_cast<int64_t>(a.vocab) * sizeof(T) / 16;
  const int64_t tiles = std::max<int64_t>(1, (vecs + kBackTile - 1) / kBackTile);
  // a grid has at most 2^31 - 1 blocks: rows in parts
  const int64_t most = std::max<int64_t>(1, INT32_MAX / tiles);
  for (int64_t done_rows = 0; done_rows < a.rows; done_rows += most) {
    RowArgs part = a;
    part.rows = static_cast<int32_t>(std::min(most, a.rows - done_rows));
    part.labels = a.labels + done_rows;
    part.logits = static_cast<const T*>(a.logits) + done_rows * a.stride;
    part.dlogits = static_cast<T*>(a.dlogits) + done_rows * a.dstride;
    const cudaError_t e =
        launch_pdl(logprobs_backward_kernel<T>, dim3(static_cast<unsigned>(part.rows * tiles)), dim3(kBackThreads), 0, s,
                   part, lse + done_rows, dlogprobs + done_rows, static_cast<int32_t>(tiles));
    if (e != cudaSuccess) return done(e);
  }
  return THD_OK;
}

}  // namespace

thd_status_t launch_row_loss(RowMode mode, int32_t dtype, const RowArgs& a, cudaStream_t s) {
  if (a.rows == 0) return THD_OK;
  if (dtype == THD_DTYPE_BF16) return launch_type<__nv_bfloat16>(mode, a, s);
  if (dtype == THD_DTYPE_F16) return launch_type<__half>(mode, a, s);
  return launch_type<float>(mode, a, s);
}

thd_status_t launch_logprobs_backward(int32_t dtype, const RowArgs& a, const float* lse, const float* dlogprobs,
                                      cudaStream_t s) {
  if (a.rows == 0) return THD_OK;
  if (dtype == THD_DTYPE_BF16) return launch_backward<__nv_bfloat16>(a, lse, dlogprobs, s);
  if (dtype == THD_DTYPE_F16) return launch_backward<__half>(a, lse, dlogprobs, s);
  return launch_backward<float>(a, lse, dlogprobs, s);
}

}  // namespace thd
