// Tokens sorted by expert and back, with their gradients, for GB300 (sm_103a).
//
//   dora_expert_sort        expert[T, k] -> order, inverse, offsets
//   dora_expert_send        xs[inverse[t, j]] = x[t]
//   dora_expert_return      y[t] = sum_j weight[t, j] ys[inverse[t, j]]
//   dora_expert_return_bwd  d_ys[inverse[t, j]] = weight[t, j] dy[t],
//                           d_weight[t, j] = <dy[t], ys[inverse[t, j]]>
//   dora_expert_clear       zeros in the rows that no expert has
//
// The gradient of send is return without weights.  An entry whose expert is
// outside [0, experts) goes to no expert: its row lies behind the last expert's,
// where nothing is read or written, its weight counts for nothing and gets the
// gradient 0.  All of them are stable and add in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "stream.cuh"
#include "tc_ptx.cuh"

namespace {

// ---------------------------------------------------------------------------
// the sort: one cluster of CTAs per expert, and one for the entries of none, each CTA
// and each of its warps a stretch of the input.  A cluster counts the entries of lower
// experts, which is where its rows start, and its own in every stretch, and then
// numbers its own in order.  No cluster waits for another; the input is read from L2.
// It is bound by its instructions, about 20 an entry, expert and lane: 65536 entries of
// 64 experts 10 us (one CTA an expert 16), 378 of 60 2.
// ---------------------------------------------------------------------------
constexpr int kSortWarps = 32;
constexpr int kMaxSortCtas = 8;

__device__ __forceinline__ int bin_of(int32_t v, int experts) {
  return static_cast<int>(min(static_cast<uint32_t>(v), static_cast<uint32_t>(experts)));
}
__device__ __forceinline__ int bin_of(int64_t v, int experts) {
  return static_cast<int>(min(static_cast<unsigned long long>(v), static_cast<unsigned long long>(experts)));
}
__device__ __forceinline__ int2 ld_cluster_s32x2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <typename Idx, bool MANY>
__global__ void __launch_bounds__(32 * kSortWarps)
expert_sort_kernel(const Idx *__restrict__ expert, int n, int experts, int many, int *__restrict__ order,
                   int *__restrict__ inverse, int *__restrict__ offsets) {
  __shared__ int2 counts[kSortWarps];                  // of lower experts, of this one
  __shared__ int2 total;
  const int ctas = MANY ? many : 1;
  const int e = static_cast<int>(blockIdx.x) / ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x) - e * ctas;
  // each warp a stretch of whole 32s
  const int64_t all = static_cast<int64_t>(32 * kSortWarps) * ctas, per = (n + all - 1) / all * 32;
  const int64_t i0 = per * (rank * kSortWarps + warp), i1 = i0 + per < n ? i0 + per : n;
  int lt = 0, eq = 0;
#pragma unroll 8
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int b = bin_of(expert[i], experts);
    lt += b < e;
    eq += b == e;
  }
  lt = __reduce_add_sync(0xffffffffu, lt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) counts[warp] = make_int2(lt, eq);
  __syncthreads();
  int start = __reduce_add_sync(0xffffffffu, counts[lane].x);
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? counts[lane].y : 0);
  if (MANY) {
    const int own = __reduce_add_sync(0xffffffffu, counts[lane].y);
    if (threadIdx.x == 0) total = make_int2(start, own);
    __syncwarp();
    cluster_sync();
    start = 0;
    for (int c = 0; c < ctas; ++c) {
      const int2 v = ld_cluster_s32x2(mapa_shared(smem_u32(&total), static_cast<uint32_t>(c)));
      start += v.x;
      at += c < rank ? v.y : 0;
    }
  }
  at += start;
  if (threadIdx.x == 0 && rank == 0) offsets[e] = start;
  if (counts[warp].y != 0) {
    const uint32_t lower = (1u << lane) - 1;
#pragma unroll 4
    for (int64_t i = i0; i < i1; i += 32) {
      const bool mine = i + lane < i1 && bin_of(expert[i + lane], experts) == e;
      const uint32_t same = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int p = at + __popc(same & lower);
        order[p] = static_cast<int>(i) + lane;
        inverse[i + lane] = p;
      }
      at += __popc(same);
    }
  }
  __syncwarp();
  if (MANY) cluster_sync();                        // no CTA leaves while another reads its counts
}

// ---------------------------------------------------------------------------
// rows there and back.  The threads of a token hold VEC columns each and walk
// its row; a block holds kThreads / tpt tokens.  Bound by memory: 8192 tokens at 8 experts
// each, 4096 columns of bf16, send 103 us, return 91, its gradient 176 (at the copy
// bandwidth 90, 90 and 171).
// ---------------------------------------------------------------------------
struct RouteParams {
  int64_t T, cols;
  int k, tpt;                  // rows a token has, threads a token has
  uint32_t rows;               // T k
  const int *inverse;          // [T, k]
  const int *end;              // rows that belong to an expert
};
// no row past the T k of the arrays, whatever the offsets say
__device__ __forceinline__ uint32_t rows_sent(const RouteParams &p) {
  return min(static_cast<uint32_t>(max(*p.end, 0)), p.rows);
}

template <typename Act, int VEC>
__global__ void __launch_bounds__(kThreads)
expert_send_kernel(const Act *__restrict__ x, const RouteParams p, Act *__restrict__ xs) {
  using IO = Io<Act, VEC>;
  const int per = kThreads / p.tpt, c0 = static_cast<int>(threadIdx.x % p.tpt) * VEC;
  const uint32_t end = rows_sent(p);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.tpt; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int *row = p.inverse + t * p.k;
    for (int64_t c = c0; c < p.cols; c += static_cast<int64_t>(p.tpt) * VEC) {
      const typename IO::Raw v = IO::load(x, t * p.cols + c);
      for (int j = 0; j < p.k; ++j) {
        const uint32_t r = static_cast<uint32_t>(row[j]);
        if (r < end) IO::store(xs, static_cast<int64_t>(r) * p.cols + c, v);
      }
    }
  }
}

template <typename Act, int VEC>
__global__ void __launch_bounds__(kThreads)
expert_return_kernel(const Act *__restrict__ ys, const float *__restrict__ weight, const RouteParams p,
                     Act *__restrict__ y) {
  using IO = Io<Act, VEC>;
  constexpr int kAhead = 4;
  const int per = kThreads / p.tpt, c0 = static_cast<int>(threadIdx.x % p.tpt) * VEC;
  const uint32_t end = rows_sent(p);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / p.tpt; t < p.T;
       t += static_cast<int64_t>(gridDim.x) * per) {
    const int *row = p.inverse + t * p.k;
    for (int64_t c = c0; c < p.cols; c += static_cast<int64_t>(p.tpt) * VEC) {
      float acc[VEC] = {};
      for (int j = 0; j < p.k; j += kAhead) {
        typename IO::Raw raw[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          const uint32_t r = j + a < p.k ? static_cast<uint32_t>(row[j + a]) : 0xffffffffu;
          live[a] = r < end;
          raw[a] = live[a] ? IO::load(ys, static_cast<int64_t>(r) * p.cols + c) : typename IO::Raw{};
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (!live[a]) continue;
          const float w = weight ? weight[t * p.k + j + a] : 1.0f;
          float v[VEC];
          IO::unpack(raw[a], v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, v[i], acc[i]);
        }
      }
      IO::store(y, t * p.cols + c, IO::pack(acc));
    }
  }
}

template <typename Act, int VEC>
__global__ void __launch_bounds__(kThreads)
expert_return_bwd_kernel(const Act *__restrict__ dy, const Act *__restrict__ ys, const float *__restrict__ weight,
                         const RouteParams p, Act *__restrict__ d_ys, float *__restrict__ d_weight) {
  using IO = Io<Act, VEC>;
  constexpr int kAhead = 4;
  __shared__ float part[kAhead][kThreads / 32];
  const int per = kThreads / p.tpt, c0 = static_cast<int>(threadIdx.x % p.tpt) * VEC;
  const uint32_t end = rows_sent(p);
  // every thread takes part in the sums, whether its token exists or not
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * per; t0 < p.T; t0 += static_cast<int64_t>(gridDim.x) * per) {
    const int64_t t = t0 + threadIdx.x / p.tpt;
    const bool in = t < p.T;
    for (int j = 0; j < p.k; j += kAhead) {
      uint32_t r[kAhead];
      float w[kAhead], dot[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const bool has = in && j + a < p.k;
        r[a] = has ? static_cast<uint32_t>(p.inverse[t * p.k + j + a]) : 0xffffffffu;
        w[a] = has ? weight[t * p.k + j + a] : 0.0f;
        dot[a] = 0.0f;
      }
      if (in)
        for (int64_t c = c0; c < p.cols; c += static_cast<int64_t>(p.tpt) * VEC) {
          const typename IO::Raw draw = IO::load(dy, t * p.cols + c);
          typename IO::Raw raw[kAhead];
#pragma unroll
          for (int a = 0; a < kAhead; ++a)
            raw[a] = r[a] < end ? IO::load(ys, static_cast<int64_t>(r[a]) * p.cols + c) : typename IO::Raw{};
          float d[VEC];
          IO::unpack(draw, d);
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            if (r[a] >= end) continue;
            float v[VEC], o[VEC];
            IO::unpack(raw[a], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              dot[a] = fmaf(d[i], v[i], dot[a]);
              o[i] = w[a] * d[i];
            }
            IO::store(d_ys, static_cast<int64_t>(r[a]) * p.cols + c, IO::pack(o));
          }
        }
      // the token's threads: within a warp, then its warps in order
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        for (int o = min(p.tpt, 32) / 2; o > 0; o >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
      const int lead = threadIdx.x % p.tpt;
      if (p.tpt > 32) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
          if (threadIdx.x % 32 == 0) part[a][threadIdx.x / 32] = dot[a];
        __syncthreads();
        if (lead == 0)
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            float s = 0.0f;
            for (int v = 0; v < p.tpt / 32; ++v) s += part[a][threadIdx.x / 32 + v];
            dot[a] = s;
          }
        __syncthreads();
      }
      if (lead == 0)
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
          if (in && j + a < p.k) d_weight[t * p.k + j + a] = r[a] < end ? dot[a] : 0.0f;
    }
  }
}

// rows [rows, cols] of no expert: before the first's and behind the last's.  `Word`
// divides a row
template <typename Word>
__global__ void __launch_bounds__(kThreads)
expert_clear_kernel(Word *__restrict__ x, int64_t rows, int64_t words, const int *__restrict__ offsets, int experts) {
  const int64_t first = min(static_cast<int64_t>(max(offsets[0], 0)), rows),
                end = min(max(static_cast<int64_t>(offsets[experts]), first), rows);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads, i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t i = i0; i < first * words; i += step) x[i] = Word{};
  for (int64_t i = end * words + i0; i < rows * words; i += step) x[i] = Word{};
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int64_t kMaxExperts = 4096;

bool bad_rows(int64_t T, int64_t k, int64_t cols, int64_t experts) {
  return T < 0 || k < 1 || cols < 0 || experts < 1 || experts > kMaxExperts || cols >= (1ll << 31) ||
         T >= (1ll << 31) || k >= (1ll << 31) || T * k >= (1ll << 31) - 1024;
}

// as many threads a token as its row has pieces, up to the block
unsigned plan(RouteParams *p, int vec, int resident, int sms) {
  const int64_t pieces = dora::ceil_div(p->cols, vec);
  p->tpt = 1;
  while (p->tpt < kThreads && p->tpt < pieces) p->tpt *= 2;
  const int64_t all = dora::ceil_div(p->T, kThreads / p->tpt), most = static_cast<int64_t>(sms) * resident;
  return static_cast<unsigned>(all < most ? all : most);
}

template <typename Act>
dora_status run_send(const void *x, RouteParams p, void *xs, int device, int sms, cudaStream_t cs) {
  constexpr int V = 16 / sizeof(Act);
  if (vector_ok<Act>(p.cols, {x, xs})) {
    const unsigned g = plan(&p, V, resident_blocks<expert_send_kernel<Act, V>>(device), sms);
    expert_send_kernel<Act, V><<<g, kThreads, 0, cs>>>(static_cast<const Act *>(x), p, static_cast<Act *>(xs));
  } else {
    const unsigned g = plan(&p, 1, resident_blocks<expert_send_kernel<Act, 1>>(device), sms);
    expert_send_kernel<Act, 1><<<g, kThreads, 0, cs>>>(static_cast<const Act *>(x), p, static_cast<Act *>(xs));
  }
  dora::count_launches(1);
  return dora::launch_status();
}

template <typename Act>
dora_status run_return(const void *ys, const float *w, RouteParams p, void *y, int device, int sms, cudaStream_t cs) {
  constexpr int V = 16 / sizeof(Act);
  if (vector_ok<Act>(p.cols, {ys, y})) {
    const unsigned g = plan(&p, V, resident_blocks<expert_return_kernel<Act, V>>(device), sms);
    expert_return_kernel<Act, V><<<g, kThreads, 0, cs>>>(static_cast<const Act *>(ys), w, p, static_cast<Act *>(y));
  } else {
    const unsigned g = plan(&p, 1, resident_blocks<expert_return_kernel<Act, 1>>(device), sms);
    expert_return_kernel<Act, 1><<<g, kThreads, 0, cs>>>(static_cast<const Act *>(ys), w, p, static_cast<Act *>(y));
  }
  dora::count_launches(1);
  return dora::launch_status();
}

template <typename Act>
dora_status run_return_bwd(const void *dy, const void *ys, const float *w, RouteParams p, void *d_ys, float *dw,
                           int device, int sms, cudaStream_t cs) {
  constexpr int V = 16 / sizeof(Act);
  const auto *pd = static_cast<const Act *>(dy), *py = static_cast<const Act *>(ys);
  if (vector_ok<Act>(p.cols, {dy, ys, d_ys})) {
    const unsigned g = plan(&p, V, resident_blocks<expert_return_bwd_kernel<Act, V>>(device), sms);
    expert_return_bwd_kernel<Act, V><<<g, kThreads, 0, cs>>>(pd, py, w, p, static_cast<Act *>(d_ys), dw);
  } else {
    const unsigned g = plan(&p, 1, resident_blocks<expert_return_bwd_kernel<Act, 1>>(device), sms);
    expert_return_bwd_kernel<Act, 1><<<g, kThreads, 0, cs>>>(pd, py, w, p, static_cast<Act *>(d_ys), dw);
  }
  dora::count_launches(1);
  return dora::launch_status();
}

RouteParams params(const int32_t *inverse, const int32_t *offsets, int64_t T, int64_t k, int64_t cols, int64_t experts) {
  RouteParams p = {};
  p.T = T;
  p.cols = cols;
  p.k = static_cast<int>(k);
  p.rows = static_cast<uint32_t>(T * k);
  p.inverse = inverse;
  p.end = offsets + experts;
  return p;
}

bool bad_elem(dora_dtype act, const void *p) { return !dora::aligned(p, act == DORA_BF16 ? 2 : 4); }

}  // namespace

template <typename Idx>
static dora_status run_sort(const void *expert, int n, int E, int sms, int32_t *order, int32_t *inverse, int32_t *offsets,
                            cudaStream_t cs) {
  // as many CTAs an expert as are resident at two an SM, each with at least four
  // entries a thread
  int ctas = 1;
  while (ctas < kMaxSortCtas && 2 * ctas * (E + 1) <= 2 * sms && n / (2 * ctas) >= 4 * 32 * kSortWarps) ctas *= 2;
  const auto *ex = static_cast<const Idx *>(expert);
  if (ctas == 1) {
    expert_sort_kernel<Idx, false><<<E + 1, 32 * kSortWarps, 0, cs>>>(ex, n, E, 1, order, inverse, offsets);
    return dora::launch_status();
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(ctas);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((E + 1) * ctas));
  cfg.blockDim = dim3(32 * kSortWarps);
  cfg.stream = cs;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, expert_sort_kernel<Idx, true>, ex, n, E, ctas, order, inverse, offsets) !=
      cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  return DORA_OK;
}

extern "C" dora_status dora_expert_sort(int index_bytes, const void *expert, int64_t T, int64_t k, int64_t experts,
                                        int32_t *order, int32_t *inverse, int32_t *offsets, dora_stream_t stream) {
  if (index_bytes != 4 && index_bytes != 8) return DORA_ERR_DTYPE;
  if (bad_rows(T, k, 0, experts)) return DORA_ERR_SHAPE;
  if (!offsets || (T > 0 && (!expert || !order || !inverse))) return DORA_ERR_NULL;
  if (!dora::aligned(expert, index_bytes) || !dora::aligned(order, 4) || !dora::aligned(inverse, 4) ||
      !dora::aligned(offsets, 4))
    return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  const dora_status st = dora::current_device(&info, nullptr);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(T * k), E = static_cast<int>(experts);
  const dora_status done = index_bytes == 4 ? run_sort<int32_t>(expert, n, E, info.sms, order, inverse, offsets, cs)
                                            : run_sort<int64_t>(expert, n, E, info.sms, order, inverse, offsets, cs);
  if (done != DORA_OK) return done;
  dora::count_launches(1);
  return DORA_OK;
}

extern "C" dora_status dora_expert_send(dora_dtype act, const void *x, const int32_t *inverse, const int32_t *offsets,
                                        int64_t T, int64_t k, int64_t cols, int64_t experts, void *xs,
                                        dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_rows(T, k, cols, experts)) return DORA_ERR_SHAPE;
  if (T == 0 || cols == 0) return DORA_OK;
  if (!x || !inverse || !offsets || !xs) return DORA_ERR_NULL;
  if (bad_elem(act, x) || bad_elem(act, xs) || !dora::aligned(inverse, 4) || !dora::aligned(offsets, 4))
    return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  const dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const RouteParams p = params(inverse, offsets, T, k, cols, experts);
  return act == DORA_BF16 ? run_send<__nv_bfloat16>(x, p, xs, device, info.sms, cs)
                          : run_send<float>(x, p, xs, device, info.sms, cs);
}

extern "C" dora_status dora_expert_return(dora_dtype act, const void *ys, const int32_t *inverse, const int32_t *offsets,
                                          const float *weight, int64_t T, int64_t k, int64_t cols, int64_t experts,
                                          void *y, dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_rows(T, k, cols, experts)) return DORA_ERR_SHAPE;
  if (T == 0 || cols == 0) return DORA_OK;
  if (!ys || !inverse || !offsets || !y) return DORA_ERR_NULL;
  if (bad_elem(act, ys) || bad_elem(act, y) || !dora::aligned(inverse, 4) || !dora::aligned(offsets, 4) ||
      !dora::aligned(weight, 4))
    return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  const dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const RouteParams p = params(inverse, offsets, T, k, cols, experts);
  return act == DORA_BF16 ? run_return<__nv_bfloat16>(ys, weight, p, y, device, info.sms, cs)
                          : run_return<float>(ys, weight, p, y, device, info.sms, cs);
}

extern "C" dora_status dora_expert_return_bwd(dora_dtype act, const void *dy, const void *ys, const int32_t *inverse,
                                              const int32_t *offsets, const float *weight, int64_t T, int64_t k,
                                              int64_t cols, int64_t experts, void *d_ys, float *d_weight,
                                              dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_rows(T, k, cols, experts)) return DORA_ERR_SHAPE;
  if (T == 0) return DORA_OK;
  if (!inverse || !offsets || !weight || !d_weight || (cols > 0 && (!dy || !ys || !d_ys))) return DORA_ERR_NULL;
  if (bad_elem(act, dy) || bad_elem(act, ys) || bad_elem(act, d_ys) || !dora::aligned(inverse, 4) ||
      !dora::aligned(offsets, 4) || !dora::aligned(weight, 4) || !dora::aligned(d_weight, 4))
    return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  const dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const RouteParams p = params(inverse, offsets, T, k, cols, experts);
  return act == DORA_BF16 ? run_return_bwd<__nv_bfloat16>(dy, ys, weight, p, d_ys, d_weight, device, info.sms, cs)
                          : run_return_bwd<float>(dy, ys, weight, p, d_ys, d_weight, device, info.sms, cs);
}

extern "C" dora_status dora_expert_clear(dora_dtype act, void *x, const int32_t *offsets, int64_t rows, int64_t cols,
                                         int64_t experts, dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_rows(rows, 1, cols, experts)) return DORA_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DORA_OK;
  if (!x || !offsets) return DORA_ERR_NULL;
  if (bad_elem(act, x) || !dora::aligned(offsets, 4)) return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  const dora_status st = dora::current_device(&info, nullptr);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int64_t bytes = cols * (act == DORA_BF16 ? 2 : 4);
  const bool wide = bytes % 16 == 0 && dora::aligned(x, 16);
  const int64_t words = wide ? bytes / 16 : bytes / 2, all = dora::ceil_div(rows * words, kThreads), most = 4 * info.sms;
  const unsigned grid = static_cast<unsigned>(all < most ? all : most);
  if (wide)
    expert_clear_kernel<uint4><<<grid, kThreads, 0, cs>>>(static_cast<uint4 *>(x), rows, words, offsets, static_cast<int>(experts));
  else
    expert_clear_kernel<uint16_t><<<grid, kThreads, 0, cs>>>(static_cast<uint16_t *>(x), rows, words, offsets,
                                                             static_cast<int>(experts));
  dora::count_launches(1);
  return dora::launch_status();
}
