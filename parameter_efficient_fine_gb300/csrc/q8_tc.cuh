// What the tensor-core kernels of the 8-bit operators share: the wait limits
// and hooks, the tensor map of an 8-bit matrix, tensor-memory loads.  Each
// translation unit gets its own internal copy (anonymous namespace).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1024;   // a tile past it is still an int
constexpr int kSmemMax = 232448;
constexpr unsigned long long kWaitNs = 2000000000ull;

// the device error word, and the test hook that withholds loads
struct Guard {
  int *err;
  const int *stall;
  const unsigned long long *limit_ns;
};

// bounded wait.  The clock that bounds it is slow to read (hundreds of cycles),
// so it is started only after a few tries
__device__ __forceinline__ bool guard_wait(uint32_t bar, uint32_t parity, SharedCtl *ctl, const Guard &g, int code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return wait_bounded_ns(bar, parity, ctl, g.err, code, *reinterpret_cast<const volatile unsigned long long *>(g.limit_ns));
}
__device__ __forceinline__ bool loads_withheld(const Guard &g) {
  return *reinterpret_cast<const volatile int *>(g.stall) != 0;
}

// this thread's warp, as a value that the compiler knows to be the same in all
// of its lanes
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}
// one lane of a converged warp.  The MMA warp runs its loop as a whole and
// issues under this, so the operands of its instructions stay warp-uniform
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// C consecutive fp32 columns of this thread's tensor-memory lane
template <int C> __device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[C]);
template <> __device__ __forceinline__ void tmem_ld<32>(uint32_t taddr, float (&v)[32]) { tmem_ld32(taddr, v); }
template <> __device__ __forceinline__ void tmem_ld<16>(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <> __device__ __forceinline__ void tmem_ld<8>(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// D (+)= A B with a power-of-two scale per row of A and per row of B, 8-bit or
// smaller operands in shared memory, scale words in tensor memory
__device__ __forceinline__ void mma_q8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// instruction descriptor: E4M3 x E4M3, E8M0 scales, fp32 accumulator, M = m,
// N = n, `byte` of the scale words on both sides, A transposed (M-major) or not
__device__ __forceinline__ uint32_t idesc_q8(int m, int n, uint32_t byte, bool a_mmajor) {
  return (byte << 4)                                  // B's scale byte
         | (a_mmajor ? 1u << 15 : 0u)
         | (static_cast<uint32_t>(n >> 3) << 17)
         | (1u << 23)                                 // E8M0 scales
         | (static_cast<uint32_t>(m >> 4) << 24)
         | (byte << 29);                              // A's scale byte
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// loads that stay where they are written (the compiler would move them down to
// their use, past the wait that they are to overlap)
__device__ __forceinline__ uint32_t load_now(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_now(const uint8_t *p) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// arrive on an mbarrier of the pair where what it hands over is tensor memory
// only: the tcgen05 fence before it orders that, and a release at cluster scope
// (a memory fence of about 1500 cycles here) would order nothing more
__device__ __forceinline__ void mbar_arrive_pair_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// a place in a ring of n
struct Ring {
  int n, i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int size) : n(size) {}
  __device__ __forceinline__ void next() {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// bytes [rows, cols] (cols a multiple of 16) with a [box_rows x 128] box, 128-byte
// swizzle; `promotion` is how much a fetch from memory brings into L2
inline bool map_q8(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int box_rows,
                   CUtensorMapL2promotion promotion) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the device's error word and hooks; once per context, the shared-memory limit of `kernels`
inline dora_status tc_init(int device, Guard *g, const void *const *kernels, int nkernels) {
  static std::mutex mu;
  static uint64_t done_ctx[64] = {};
  static Guard known[64] = {};
  if (device < 0 || device >= 64) return DORA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  const uint64_t ctx = dora::context_id();
  if (ctx == 0 || ctx != done_ctx[device]) {
    int *stall = nullptr;
    unsigned long long *limit = nullptr;
    dora_status st = dora::error_word(device, &known[device].err);
    if (st == DORA_OK) st = dora::test_hooks(&stall, &limit);
    if (st != DORA_OK) return st;
    known[device].stall = stall;
    known[device].limit_ns = limit;
    for (int k = 0; k < nkernels; ++k)
      if (cudaFuncSetAttribute(kernels[k], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
        return DORA_ERR_CUDA;
    done_ctx[device] = dora::context_id();
  }
  *g = known[device];
  return DORA_OK;
}

inline bool bad_size(int64_t v, int64_t least) { return v < least || v > kMaxDim; }

}  // namespace
