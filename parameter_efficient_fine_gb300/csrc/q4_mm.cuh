// What the two kernels of a product with a 4-bit weight share: the call's
// parameters and the tiles of it.  Each translation unit gets its own internal copy
// (anonymous namespace).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "q4.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int64_t kMaxExperts = 4096;

struct Q4Params {
  int T, out, in;
  int nfeat, kdim;                  // features of the result, k
  int experts;
  const int *offsets;               // null: one weight, all rows
  int ntok;                         // tokens per tile
  int xrows;                        // rows of a box of x (q4_mm.cu)
  int ftiles, parts;                // feature tiles; parts that k is cut into
  int tiles;                        // no more than these
  const uint8_t *scale;
  __nv_bfloat16 *y;
  float *partial;                   // results of the parts [parts, T, nfeat]
  Guard guard;
};

// feature tiles per tile-order group, for reuse in L2
constexpr int kGroupF = 8;

// what a tile works on
struct Tile {
  int e, ft;                        // expert, feature tile
  int t0, t1;                       // its tokens
};

// Tile `t`, or false past the last.  All lanes of the warp call it.  Experts: the
// tokens' tiles of all experts in order, the feature tiles of each in turn.
__device__ __forceinline__ bool find_tile(const Q4Params &p, int t, Tile *o) {
  if (!p.offsets) {
    if (t >= p.tiles) return false;
    const int ntiles = p.tiles / p.ftiles, per = kGroupF * ntiles, g = t / per, f0 = g * kGroupF,
              gf = min(kGroupF, p.ftiles - f0), r = t - g * per, tt = r / gf;
    o->e = 0;
    o->ft = f0 + r - tt * gf;
    o->t0 = tt * p.ntok;
    o->t1 = min(p.T, o->t0 + p.ntok);
    return true;
  }
  const int lane = threadIdx.x & 31;
  const int tt = t / p.ftiles;
  int64_t before = 0;                                  // token tiles of the experts before this 32
  for (int e0 = 0; e0 < p.experts; e0 += 32) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < p.experts) {
      a = min(max(p.offsets[e], 0), p.T);
      b = min(max(p.offsets[e + 1], a), p.T);
    }
    const int own = (b - a + p.ntok - 1) / p.ntok;
    int64_t upto = own;                                // tiles of this 32, up to and with this expert's
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > tt);
    if (past) {
      const int who = __ffs(past) - 1;
      const int64_t first = __shfl_sync(0xffffffffu, upto - own, who);
      a = __shfl_sync(0xffffffffu, a, who);
      b = __shfl_sync(0xffffffffu, b, who);
      o->e = e0 + who;
      o->ft = t - tt * p.ftiles;
      o->t0 = a + static_cast<int>(tt - before - first) * p.ntok;
      o->t1 = min(b, o->t0 + p.ntok);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// this thread's writes to shared memory before the tensor core's reads
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// the stack of weights [experts, out, in / 2 bytes] in boxes of 128 rows x 64 bytes, 64-byte swizzle
inline bool map_w(CUtensorMap *map, const void *base, int64_t experts, int64_t out, int64_t in) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(in / 2), static_cast<cuuint64_t>(out), static_cast<cuuint64_t>(experts)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(in / 2), static_cast<cuuint64_t>(in / 2) * static_cast<cuuint64_t>(out)};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace dora {

// The tokens that a tile of q4_few.cu is made for.  Experts: twice their mean, for uneven loads,
// whose second tile of an expert would read its weight again (32 experts of 2048 x 4096, us
// by twice the mean and by the mean; uneven: squares of even numbers, up to three times the mean: 256
// tokens 40, 62; 512 47, 59; even loads 40, 48; 47, 45; one expert with half of the tokens 49, 62; 59, 58)
inline int64_t q4_tile(int64_t T, int64_t experts) {
  const int64_t per = experts < T ? ceil_div(T, experts) : 1;
  return (experts > 1 ? 2 : 1) * per;
}
// x W^T by q4_few.cu: where a tile is made for so many at most; where rows of W are no whole blocks of
// 128, for half (us, that kernel / pairs: 32 x 8192 x 8192 17 / 19, 32 x 14336 x 4096 16.4 / 18.1, 32 x 4096 x
// 4096 10.8 / 9.6, 512 tokens at 32 experts of 2048 x 4096 47 / 59, 768 at 32, tiles of 32, 65 / 59; with 64 in a
// tile, whose third and fourth pieces leave room for one CTA an SM, 37 x 14336 x 4096 21.9 / 18.2, 64 x 8192 x 8192 25 / 19.5.
// 8224 columns: 16 tokens 18.7 / 20.1, 20 22.6 / 20.2; 16 x 1024 x 4128 9.1 / 8.1)
inline bool q4_few(int64_t T, int64_t in, int64_t experts) { return q4_tile(T, experts) <= (in % 128 == 0 ? 32 : 16); }
size_t q4_few_workspace(int64_t T, int64_t in, int64_t experts);
dora_status matmul_q4_few(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T,
                          int64_t out, int64_t in, int64_t experts, void *y, void *workspace, cudaStream_t cs);

}  // namespace dora
