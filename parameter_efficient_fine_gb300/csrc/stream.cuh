// What the kernels that stream [T, out] matrices share (compose.cu, q8.cu):
// the thread layout, the vector accesses, the d_mag reduction and the grid
// plan.  Each translation unit gets its own internal copy (anonymous namespace).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <initializer_list>
#include <mutex>

#include "common.cuh"

namespace {

constexpr int kBX = 32;     // column groups per block
constexpr int kBY = 8;      // token lanes per block
constexpr int kThreads = kBX * kBY;
constexpr int kMaxSMs = 256;             // workspace bound: any device up to this size
constexpr int kMaxBlocksPerSM = 2048 / kThreads;

// ---------------------------------------------------------------------------
// Vector I/O: Raw is what one access moves; unpack/pack convert to fp32.
// ---------------------------------------------------------------------------
template <typename Act, int VEC> struct Io;

template <> struct Io<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p, int64_t e) {
    return __ldcs(reinterpret_cast<const uint4 *>(p + e));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, int64_t e, Raw r) {
    __stcs(reinterpret_cast<uint4 *>(p + e), r);
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <> struct Io<float, 4> {
  using Raw = float4;
  static __device__ __forceinline__ Raw load(const float *p, int64_t e) {
    return __ldcs(reinterpret_cast<const float4 *>(p + e));
  }
  static __device__ __forceinline__ void store(float *p, int64_t e, Raw r) {
    __stcs(reinterpret_cast<float4 *>(p + e), r);
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[4]) {
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  static __device__ __forceinline__ Raw pack(const float (&v)[4]) { return make_float4(v[0], v[1], v[2], v[3]); }
};

template <> struct Io<__nv_bfloat16, 1> {
  using Raw = unsigned short;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p, int64_t e) {
    return __ldcs(reinterpret_cast<const unsigned short *>(p + e));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, int64_t e, Raw r) {
    __stcs(reinterpret_cast<unsigned short *>(p + e), r);
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[1]) { v[0] = __uint_as_float(uint32_t(r) << 16); }
  static __device__ __forceinline__ Raw pack(const float (&v)[1]) {
    __nv_bfloat16 h = __float2bfloat16_rn(v[0]);
    return *reinterpret_cast<unsigned short *>(&h);
  }
};

template <> struct Io<float, 1> {
  using Raw = float;
  static __device__ __forceinline__ Raw load(const float *p, int64_t e) { return __ldcs(p + e); }
  static __device__ __forceinline__ void store(float *p, int64_t e, Raw r) { __stcs(p + e, r); }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[1]) { v[0] = r; }
  static __device__ __forceinline__ Raw pack(const float (&v)[1]) { return v[0]; }
};

// d_mag[j] = (sum over partial rows in increasing order) / norm[j]
__global__ void __launch_bounds__(256)
dmag_reduce_kernel(const float *__restrict__ part, int64_t rows, int64_t out,
                   const float *__restrict__ norm, float *__restrict__ d_mag) {
  const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= out) return;
  float sum = 0.0f;
  int64_t k = 0;
  for (; k + 4 <= rows; k += 4) {
    const float a0 = part[(k + 0) * out + j], a1 = part[(k + 1) * out + j];
    const float a2 = part[(k + 2) * out + j], a3 = part[(k + 3) * out + j];
    sum += a0;
    sum += a1;
    sum += a2;
    sum += a3;
  }
  for (; k < rows; ++k) sum += part[k * out + j];
  d_mag[j] = sum / norm[j];
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// resident blocks per SM of one kernel.  The kernel is the template's argument,
// not its type: the forms of a kernel for whole pieces and for ragged rows
// have one type and each its own number
template <auto *KERNEL>
int resident_blocks(int device) {
  static std::mutex mu;
  static int cache[64] = {};
  if (device < 0 || device >= 64) return 1;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[device] == 0) {
    int b = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, KERNEL, kThreads, 0) != cudaSuccess || b <= 0) b = 1;
    cache[device] = b;
  }
  return cache[device];
}

struct Grid {
  int64_t gx, gy;
};

Grid plan_grid(int64_t T, int64_t ncg, int64_t target_blocks) {
  Grid gr;
  gr.gx = dora::ceil_div(ncg, kBX);
  // as many grid rows as the resident blocks fill, rounded DOWN: every block
  // has the same work, so a block beyond the resident ones would run alone
  // in a second wave (bf16, out = 14336 on 152 SMs x 4 blocks: 56 x 11 = 616
  // blocks took 269 us for the forward at T = 16384, 56 x 10 take 215 us)
  int64_t gy = target_blocks / gr.gx;
  const int64_t gy_max = dora::ceil_div(T, kBY);
  if (gy > gy_max) gy = gy_max;
  if (gy < 1) gy = 1;
  if (gy > 65535) gy = 65535;
  gr.gy = gy;
  return gr;
}

int64_t bwd_rows_bound(int64_t T, int64_t out) {
  // the widest vector (8 bf16) gives the fewest column groups and so the
  // most grid rows; any narrower path launches no more rows than this
  const int64_t gx_min = dora::ceil_div(dora::ceil_div(out, 8), kBX);
  Grid gr = plan_grid(T, gx_min * kBX, (int64_t)kMaxSMs * kMaxBlocksPerSM);
  return gr.gy;
}

bool valid_dtype(dora_dtype act) { return act == DORA_F32 || act == DORA_BF16; }

template <typename Act>
bool vector_ok(int64_t out, std::initializer_list<const void *> ptrs) {
  constexpr int vec = 16 / sizeof(Act);
  if (out % vec != 0) return false;
  for (const void *p : ptrs)
    if (!dora::aligned(p, 16)) return false;
  return true;
}

}  // namespace
