// A weight in 4 bits (see q4.cuh for the form), for GB300 (sm_103a).
//
//   dora_q4_store, dora_q4_load   a matrix into the 4-bit form and back
//
// Rows are whole groups of 32 columns, so the form is flat: group i of the
// matrix, in memory order, is 16 bytes of q and one of scale.  A thread holds 8
// neighbouring elements, four threads a group, whose maximum is two shuffles.  Both
// are bound by memory: 14336 x 4096 store 42 us from fp32 and 27 from bf16, load 45 and
// 27 (at the copy bandwidth 40 and 22); 512 x 512 2, a launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q4.cuh"
#include "stream.cuh"

#include <type_traits>

namespace {

constexpr int kPer = 8;            // elements a thread holds
constexpr int kRows = 4;           // pieces in flight a thread

template <typename Act> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  using IO = Io<__nv_bfloat16, 8>;
  struct Raw {
    IO::Raw a;
  };
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p, int64_t e) { return {IO::load(p, e)}; }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[8]) { IO::unpack(r.a, v); }
};
template <> struct Eight<float> {
  using IO = Io<float, 4>;
  struct Raw {
    IO::Raw a, b;
  };
  static __device__ __forceinline__ Raw load(const float *p, int64_t e) { return {IO::load(p, e), IO::load(p, e + 4)}; }
  static __device__ __forceinline__ void unpack(const Raw &r, float (&v)[8]) {
    v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
    v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
  }
};

// `pieces` of 8 elements, a multiple of 4
template <typename Act>
__global__ void __launch_bounds__(kThreads)
q4_store_kernel(const Act *__restrict__ x, int64_t pieces, uint32_t *__restrict__ q, uint8_t *__restrict__ scale) {
  using E = Eight<Act>;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads; base < pieces; base += kRows * step) {
    typename E::Raw raw[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t i = base + r * step + threadIdx.x;
      raw[r] = i < pieces ? E::load(x, i * kPer) : typename E::Raw{};
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t i = base + r * step + threadIdx.x;
      float v[kPer];
      E::unpack(raw[r], v);
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kPer; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t b = q4_scale_byte(m);
      const float inv = q4_inverse(b);
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < kPer; k += 2) w |= q4_quant2(v[k], v[k + 1], inv) << (4 * k);
      if (i < pieces) {
        __stcs(q + i, b == kQ4Nan ? 0u : w);
        if ((threadIdx.x & 3) == 0) scale[i / 4] = static_cast<uint8_t>(b);
      }
    }
  }
}

// A load writes pieces of 16 bytes: 8 elements of bf16, 4 of fp32 (of 8, a thread's two
// stores would each leave gaps: 14336 x 4096 63.9 us)
template <typename Act>
__global__ void __launch_bounds__(kThreads)
q4_load_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t pieces, Act *__restrict__ x) {
  constexpr int V = 16 / sizeof(Act), kFlight = 2 * kRows;
  using IO = Io<Act, V>;
  using Q = typename std::conditional<V == 8, uint32_t, uint16_t>::type;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads; base < pieces; base += kFlight * step) {
    uint32_t w[kFlight], b[kFlight];
#pragma unroll
    for (int r = 0; r < kFlight; ++r) {
      const int64_t i = base + r * step + threadIdx.x;
      w[r] = i < pieces ? __ldcs(reinterpret_cast<const Q *>(q) + i) : 0u;
      b[r] = i < pieces ? scale[i / (kQ4Group / V)] : 0u;
    }
#pragma unroll
    for (int r = 0; r < kFlight; ++r) {
      const int64_t i = base + r * step + threadIdx.x;
      const float s = q4_scale(b[r]);
      float v[V];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 f = q4_value2((w[r] >> (4 * k)) & 0xffu);
        v[k] = f.x * s;
        v[k + 1] = f.y * s;
      }
      if (i < pieces) IO::store(x, i * V, IO::pack(v));
    }
  }
}

dora_status check(dora_dtype act, const void *q, const void *scale, int64_t rows, int64_t cols, const void *x) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (rows < 0 || cols < 0 || rows >= (1ll << 31) || cols >= (1ll << 31)) return DORA_ERR_SHAPE;
  if (cols % kQ4Group != 0) return DORA_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DORA_OK;
  if (!q || !scale || !x) return DORA_ERR_NULL;
  if (!dora::aligned(x, 16) || !dora::aligned(q, 16)) return DORA_ERR_ALIGN;
  return DORA_OK;
}

template <auto *KERNEL>
unsigned blocks(int64_t pieces, int device, int sms) {
  const int64_t all = dora::ceil_div(pieces, kThreads), most = static_cast<int64_t>(sms) * resident_blocks<KERNEL>(device);
  return static_cast<unsigned>(all < most ? all : most);
}

}  // namespace

extern "C" dora_status dora_q4_store(dora_dtype act, const void *x, int64_t rows, int64_t cols, void *q, void *scale,
                                     dora_stream_t stream) {
  dora_status st = check(act, q, scale, rows, cols, x);
  if (st != DORA_OK || rows == 0 || cols == 0) return st;
  dora::DeviceInfo info;
  int device = 0;
  st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  const int64_t pieces = rows * (cols / kPer);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  auto *pq = static_cast<uint32_t *>(q);
  auto *ps = static_cast<uint8_t *>(scale);
  if (act == DORA_BF16)
    q4_store_kernel<__nv_bfloat16><<<blocks<q4_store_kernel<__nv_bfloat16>>(pieces, device, info.sms), kThreads, 0, cs>>>(
        static_cast<const __nv_bfloat16 *>(x), pieces, pq, ps);
  else
    q4_store_kernel<float><<<blocks<q4_store_kernel<float>>(pieces, device, info.sms), kThreads, 0, cs>>>(
        static_cast<const float *>(x), pieces, pq, ps);
  dora::count_launches(1);
  return dora::launch_status();
}

extern "C" dora_status dora_q4_load(dora_dtype act, const void *q, const void *scale, int64_t rows, int64_t cols, void *x,
                                    dora_stream_t stream) {
  dora_status st = check(act, q, scale, rows, cols, x);
  if (st != DORA_OK || rows == 0 || cols == 0) return st;
  dora::DeviceInfo info;
  int device = 0;
  st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  auto *pq = static_cast<const uint8_t *>(q);
  auto *ps = static_cast<const uint8_t *>(scale);
  if (act == DORA_BF16) {
    const int64_t pieces = rows * (cols / 8);
    q4_load_kernel<__nv_bfloat16><<<blocks<q4_load_kernel<__nv_bfloat16>>(pieces, device, info.sms), kThreads, 0, cs>>>(
        pq, ps, pieces, static_cast<__nv_bfloat16 *>(x));
  } else {
    const int64_t pieces = rows * (cols / 4);
    q4_load_kernel<float><<<blocks<q4_load_kernel<float>>(pieces, device, info.sms), kThreads, 0, cs>>>(
        pq, ps, pieces, static_cast<float *>(x));
  }
  dora::count_launches(1);
  return dora::launch_status();
}
