// The gradient of A from the 8-bit x (see q8.cuh for the form) for GB300
// (sm_103a): dora_lora_grad_q8, dA = dxa^T x, dxa [T, r] bf16, x [T, in].
//
// 64 x 64 tiles of the result on the CUDA cores, operands decoded into shared
// memory in fp32, 16 tokens at a time, a 4 x 4 block a thread, sums in chains
// of 256 tokens that are added up apart (a chain's rounding error grows with
// its length).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kTile = 64;
constexpr int kStep = 16;
constexpr int kChain = 256;
constexpr int64_t kMaxDim = (1ll << 31) - 1;

enum Mode { kMatmul, kMatmulT, kLoraGrad };

struct Operands {
  const uint8_t *q, *scale;      // x or dy: [T, kx], one scale per 128 columns
  const uint8_t *wq, *wscale;    // W [out, in], one scale per 128 x 128
  const __nv_bfloat16 *dxa;      // [T, r]
  int64_t T, out, in, r;
};

__device__ __forceinline__ float q8_at(const uint8_t *q, const uint8_t *scale, int64_t row, int64_t col, int64_t cols,
                                       int rows_per) {
  const int64_t nsc = (cols + kQBlock - 1) / kQBlock;
  return dequant2(q[row * cols + col], scale_value(scale[row / rows_per * nsc + col / kQBlock])).x;
}

// element (i, k) of the left operand and (j, k) of the right one
template <Mode M>
__device__ __forceinline__ float left(const Operands &o, int64_t i, int64_t k) {
  if (M == kLoraGrad) return __bfloat162float(o.dxa[k * o.r + i]);
  return q8_at(o.q, o.scale, i, k, M == kMatmul ? o.in : o.out, 1);
}
template <Mode M>
__device__ __forceinline__ float right(const Operands &o, int64_t j, int64_t k) {
  if (M == kMatmul) return q8_at(o.wq, o.wscale, j, k, o.in, kQBlock);
  if (M == kMatmulT) return q8_at(o.wq, o.wscale, k, j, o.in, kQBlock);
  return q8_at(o.q, o.scale, k, j, o.in, 1);
}

template <Mode M, typename Out>
__global__ void __launch_bounds__(256) q8_tile_kernel(const Operands o, int64_t m, int64_t n, int64_t kk,
                                                      Out *__restrict__ d) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int64_t ntn = (n + kTile - 1) / kTile;
  const int64_t i0 = blockIdx.x / ntn * kTile, j0 = blockIdx.x % ntn * kTile;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  float sum[4][4] = {}, acc[4][4] = {};
  for (int64_t k0 = 0; k0 < kk; k0 += kStep) {
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      // neighbouring threads read neighbouring addresses
      const int ka = M == kLoraGrad ? e / kTile : e % kStep, ia = M == kLoraGrad ? e % kTile : e / kStep;
      sa[ka][ia] = i0 + ia < m && k0 + ka < kk ? left<M>(o, i0 + ia, k0 + ka) : 0.0f;
      const int kb = M == kMatmul ? e % kStep : e / kTile, jb = M == kMatmul ? e / kStep : e % kTile;
      sb[kb][jb] = j0 + jb < n && k0 + kb < kk ? right<M>(o, j0 + jb, k0 + kb) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sa[k][ti + 16 * a], sb[k][tj + 16 * b], acc[a][b]);
    __syncthreads();
    if (k0 % kChain == kChain - kStep || k0 + kStep >= kk)
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          sum[a][b] += acc[a][b];
          acc[a][b] = 0.0f;
        }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int64_t i = i0 + ti + 16 * a, j = j0 + tj + 16 * b;
      if (i < m && j < n) d[i * n + j] = static_cast<Out>(sum[a][b]);
    }
}

template <Mode M, typename Out>
dora_status run_tiles(const Operands &o, int64_t m, int64_t n, int64_t k, void *d, dora_stream_t stream) {
  dora::DeviceInfo info;
  dora_status st = dora::current_device(&info, nullptr);
  if (st != DORA_OK) return st;
  const int64_t tiles = dora::ceil_div(m, kTile) * dora::ceil_div(n, kTile);
  if (tiles > kMaxDim) return DORA_ERR_SHAPE;
  q8_tile_kernel<M, Out><<<(unsigned)tiles, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(o, m, n, k,
                                                                                              static_cast<Out *>(d));
  dora::count_launches(1);
  return dora::launch_status();
}

bool bad_size(int64_t v, int64_t least) { return v < least || v > kMaxDim; }

}  // namespace

extern "C" size_t dora_lora_grad_q8_workspace(int64_t T, int64_t in, int64_t r) {
  if (bad_size(T, 0) || bad_size(in, 0) || r < 1 || r > 1024) return 0;
  return 256;
}

extern "C" dora_status dora_lora_grad_q8(const void *dxa, const void *xq, const void *xscale, int64_t T, int64_t in,
                                         int64_t r, float *dA, void *workspace, size_t workspace_bytes,
                                         dora_stream_t stream) {
  if (bad_size(T, 0) || bad_size(in, 0) || r < 1 || r > 1024) return DORA_ERR_SHAPE;
  if (in == 0) return DORA_OK;
  if (!dA || (T > 0 && (!dxa || !xq || !xscale))) return DORA_ERR_NULL;
  // TMA: 16-byte aligned bases and row strides
  if (in % 16 != 0 || r % 8 != 0) return DORA_ERR_ALIGN;
  if (!dora::aligned(dA, 16) || (T > 0 && (!dora::aligned(dxa, 16) || !dora::aligned(xq, 16)))) return DORA_ERR_ALIGN;
  if (!workspace || !dora::aligned(workspace, 256) || workspace_bytes < dora_lora_grad_q8_workspace(T, in, r))
    return DORA_ERR_WORKSPACE;
  const Operands o = {static_cast<const uint8_t *>(xq), static_cast<const uint8_t *>(xscale), nullptr, nullptr,
                      static_cast<const __nv_bfloat16 *>(dxa), T, 0, in, r};
  return run_tiles<kLoraGrad, float>(o, r, in, T, dA, stream);
}
