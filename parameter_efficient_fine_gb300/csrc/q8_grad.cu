// The gradient of A from the 8-bit x (see q8.cuh for the form) for GB300
// (sm_103a): dora_lora_grad_q8, dA = dxa^T x with dxa [T, r] in bf16 and x
// [T, in] in 8 bits.
//
// Every value of an 8-bit form is exact in bf16, so the product runs as
// kind::f16 bf16 MMAs with exact products: 128 features of x on the M side, up
// to 256 columns of dxa on the N side, the tokens as k.  Both operands lie in
// memory token by token, so both are M-/N-major: no transposed copy is made.
//
// The tensor core's fp32 sum rounds toward zero, so its error grows with the
// length of a chain of MMAs.  A window of 256 tokens is one chain (16 MMAs of
// k = 16); the windows are added up in registers with ordinary rounding.
//
// Work: a tile of the result is 128 features x N columns of r; its windows
// are units, and each CTA (one per SM) takes an equal run of units over all
// tiles.  A CTA that has a whole tile writes dA; otherwise it writes its part
// to the workspace and grad_join_kernel adds the parts of a tile in order
// (bitwise reproducible).
//   warp 0      TMA producer: per stage (64 tokens) the x bytes of the tile's
//               128 features (8 KB) and the dxa boxes (8 KB per 64 columns)
//   warp 1      tensor memory (two window accumulators), MMA issue
//   warps 2-9   bytes -> bf16 in shared memory, one stage after another;
//               window w - 1 out of tensor memory while window w runs
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q8.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kTok = 64;                         // tokens per stage
constexpr int kWin = 256;                        // tokens per window
constexpr int kWorkers = 8;                      // conversion warps
constexpr int kThreadsG = 64 + 32 * kWorkers;
constexpr unsigned kRawBytes = kTok * 128;       // 8 KB of x
constexpr unsigned kABytesG = kTok * 128 * 2;    // 16 KB of bf16: two halves of 64 features
constexpr unsigned kBox = kTok * 128;            // 64 tokens x 64 columns of dxa
constexpr int kMaxR = 1024;
constexpr int kMaxCtasG = 256;
constexpr int kMaxStagesG = 8;

struct GradParams {
  int T, in, r;
  int mtiles, ntiles, windows;     // tiles are m fastest; windows per tile
  int ncols;                       // columns of r per tile (N of the MMA)
  int boxes;                       // dxa boxes per stage
  int stages;
  unsigned stage_bytes;
  int nsx;
  const uint8_t *scale;
  float *dA;
  float *part;                     // [2 per CTA][columns][128]
  Guard guard;
};

// first unit of CTA i of n
__host__ __device__ __forceinline__ int64_t first_unit(int64_t units, int i, int n) { return units * i / n; }

// shared-memory descriptor of an operand whose rows are k: 64 values (one
// 128-byte swizzled row) of the M or N side, 8-row groups 1024 bytes apart,
// the next 64 values `lead` bytes on
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr, uint32_t lead) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// Four E4M3 bytes times the scale as bf16, in the order 0, 2, 1, 3.  The
// exponent and mantissa bits of an E4M3 value, four places up in a bf16, are
// that value times 2^-120 (subnormals too: their bits become a bf16
// subnormal's), so one product with 2^120 scale finishes it, exactly.
// `up` is that factor twice; it is a bf16 as long as the scale is at most 2^7
__device__ __forceinline__ uint2 decode4(uint32_t w, uint32_t up) {
  const uint32_t even = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u);
  const uint32_t odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
  return make_uint2(mul_bf16x2(even, up), mul_bf16x2(odd, up));
}
// the same through fp32, for larger scales and for NaN bytes
__device__ __noinline__ uint2 decode4_any(uint32_t w, uint32_t byte) {
  const float s = scale_value(byte);
  const float2 a = dequant2(w & 0xffffu, s), b = dequant2(w >> 16, s);
  return make_uint2(pack_bf16x2(a.x, b.x), pack_bf16x2(a.y, b.y));
}
// feature of a tile at M row m: the order of decode4
__device__ __forceinline__ int feature_of(int m) { return (m & ~3) | ((m & 1) << 1) | ((m >> 1) & 1); }

// NC: columns of a tile per worker warp (half of the tile's, rounded up)
template <int NC>
__global__ void __launch_bounds__(kThreadsG, 1)
lora_grad_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mD, const GradParams p) {
  constexpr int kN = 2 * NC;                             // columns of one window accumulator
  constexpr int kCols = kN <= 16 ? 32 : kN <= 32 ? 64 : kN <= 64 ? 128 : kN <= 128 ? 256 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(S) * p.stage_bytes);
  // barriers: loaded[S], converted[S], free[S], window done[2], window read[2]
  const uint32_t full0 = smem_u32(bars), conv0 = full0 + 8u * S, empty0 = conv0 + 8u * S, done0 = empty0 + 8u * S,
                 read0 = done0 + 16, fin = read0 + 16;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 3 * S + 5);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(conv0 + 8u * s, kWorkers);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(done0 + 8u * b, 1);
      mbar_init(read0 + 8u * b, kWorkers);
    }
    mbar_init(fin, 1);
    ctl->abort = 0;
    fence_barrier_init();
    prefetch_map(&mX);
    prefetch_map(&mD);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_u32(&ctl->tmem_base), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.windows;
  const int64_t u0 = first_unit(units, blockIdx.x, gridDim.x), u1 = first_unit(units, blockIdx.x + 1, gridDim.x);
  // stages of a window
  auto nstages = [&](int w) { return min(kWin, p.T - w * kWin + kTok - 1) / kTok; };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      bool ok = !loads_withheld(p.guard);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int64_t u = u0; u < u1 && ok; ++u) {
        const int tile = static_cast<int>(u / p.windows), w = static_cast<int>(u % p.windows);
        const int mt = tile % p.mtiles, nt = tile / p.mtiles;
        const int ns = nstages(w);
        for (int k = 0; k < ns; ++k) {
          if (!guard_wait(empty0 + 8u * stage, phase ^ 1u, ctl, p.guard, 31)) {
            ok = false;
            break;
          }
          const uint32_t fb = full0 + 8u * stage;
          const uint32_t at = smem_u32(smem + static_cast<size_t>(stage) * p.stage_bytes);
          const int t0 = w * kWin + k * kTok;
          mbar_expect_tx(fb, kRawBytes + p.boxes * kBox);
          tma_load_2d(at + kABytesG, &mX, mt * kTcM, t0, fb);
          for (int b = 0; b < p.boxes; ++b)
            tma_load_2d(at + kABytesG + kRawBytes + b * kBox, &mD, nt * p.ncols + 64 * b, t0, fb);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok)
        for (int k = 0; k < S && k < issued; ++k) {   // copies in flight
          if (--stage < 0) {
            stage = S - 1;
            phase ^= 1u;
          }
          wait_drain_ns(full0 + 8u * stage, phase, kWaitNs);
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------------------- MMA issuer
      // bf16, fp32 accumulator, both operands transposed (M- and N-major)
      const uint32_t idesc = idesc_bf16(p.ncols) | (1u << 15) | (1u << 16);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int wi = 0;
      for (int64_t u = u0; u < u1 && ok; ++u, ++wi) {
        const int ns = nstages(static_cast<int>(u % p.windows));
        const uint32_t d = tmem + static_cast<uint32_t>((wi & 1) * kN);
        if (!guard_wait(read0 + 8u * (wi & 1), (static_cast<uint32_t>(wi >> 1) & 1u) ^ 1u, ctl, p.guard, 32)) break;
        for (int k = 0; k < ns; ++k) {
          if (!guard_wait(conv0 + 8u * stage, phase, ctl, p.guard, 33)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = smem_u32(smem + static_cast<size_t>(stage) * p.stage_bytes);
          const uint32_t bt = at + kABytesG + kRawBytes;
#pragma unroll
          for (int j = 0; j < kTok / 16; ++j)   // 16 tokens: 16 rows of 128 bytes
            mma_bf16_ss(d, mn_desc(at + 2048u * j, kABytesG / 2), mn_desc(bt + 2048u * j, kBox), idesc,
                        k != 0 || j != 0 ? 1u : 0u);
          mma_commit(empty0 + 8u * stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma_commit(done0 + 8u * (wi & 1));
      }
      mma_commit(fin);
      wait_drain_ns(fin, 0, kWaitNs);
    }
  } else {
    // ---------------------------------------------------------------- workers
    const int wk = warp - 2, tid = threadIdx.x - 64;
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    const int nh = wk >> 2;                              // which half of the columns
    const uint32_t lane_addr = tmem + ((quad * 32u) << 16) + static_cast<uint32_t>(nh * NC);
    constexpr int C = NC % 32 == 0 ? 32 : NC % 16 == 0 ? 16 : 8;
    float sum[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[j] = 0.0f;
    // this thread's pieces of a stage: 16 features of rows `row` and row + 32
    const int row = tid >> 3, ch = tid & 7;
    const uint32_t half = static_cast<uint32_t>(ch >> 2) * (kABytesG / 2);
    const uint32_t first = static_cast<uint32_t>(ch >> 2);   // the halves write their two 16-byte chunks in opposite order
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int wi = 0;
    auto flush = [&](int k) {   // window number k of this CTA into `sum`
      const bool got = guard_wait(done0 + 8u * (k & 1), static_cast<uint32_t>(k >> 1) & 1u, ctl, p.guard, 34);
      if (!__all_sync(0xffffffffu, got)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NC; c += C) {
        float v[C];
        tmem_ld<C>(lane_addr + static_cast<uint32_t>((k & 1) * kN + c), v);
#pragma unroll
        for (int j = 0; j < C; ++j) sum[c + j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(read0 + 8u * (k & 1));
      return true;
    };
    int seg0 = 0;   // first window of the current run within one tile
    for (int64_t u = u0; u < u1 && ok; ++u, ++wi) {
      const int tile = static_cast<int>(u / p.windows), w = static_cast<int>(u % p.windows);
      const int mt = tile % p.mtiles, nt = tile / p.mtiles;
      const int ns = nstages(w);
      const uint8_t *sp = p.scale + mt;
      auto scale_at = [&](int t) {
        return t < p.T ? static_cast<uint32_t>(__ldg(sp + static_cast<int64_t>(t) * p.nsx)) : 127u;
      };
      uint32_t b0 = scale_at(w * kWin + row), b1 = scale_at(w * kWin + row + 32);
      for (int k = 0; k < ns; ++k) {
        const uint32_t c0 = b0, c1 = b1;
        if (k + 1 < ns) {
          b0 = scale_at(w * kWin + (k + 1) * kTok + row);
          b1 = scale_at(w * kWin + (k + 1) * kTok + row + 32);
        }
        const bool got = guard_wait(full0 + 8u * stage, phase, ctl, p.guard, 35);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        uint8_t *at = smem + static_cast<size_t>(stage) * p.stage_bytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rr = row + 32 * h;
          const uint32_t byte = h ? c1 : c0;
          const uint4 raw = *reinterpret_cast<const uint4 *>(at + kABytesG + rr * 128 + ((ch ^ (rr & 7)) << 4));
          const uint32_t in4[4] = {raw.x, raw.y, raw.z, raw.w};
          uint2 o[4];
          // a byte of 0x7f in any sign
          uint32_t nan = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) nan |= (in4[i] & 0x7f7f7f7fu) + 0x01010101u;
          if ((nan & 0x80808080u) == 0 && byte <= 134) {
            const uint32_t e = (byte + 120u) << 7;          // 2^(byte - 7) in bf16
            const uint32_t up = e | (e << 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = decode4(in4[i], up);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = decode4_any(in4[i], byte);
          }
          uint8_t *dst = at + half + rr * 128;
          const uint32_t ca = 2u * (ch & 3);
          const uint4 lo = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y), hi = make_uint4(o[2].x, o[2].y, o[3].x, o[3].y);
          const uint32_t x = static_cast<uint32_t>(rr & 7);
          *reinterpret_cast<uint4 *>(dst + (((ca + first) ^ x) << 4)) = first ? hi : lo;
          *reinterpret_cast<uint4 *>(dst + (((ca + 1 - first) ^ x) << 4)) = first ? lo : hi;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(conv0 + 8u * stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
        // the window before this one, once this one keeps the tensor core fed
        if (k == min(2, ns - 1) && wi > seg0 && !flush(wi - 1)) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      if (w + 1 == p.windows || u + 1 == u1) {
        // the end of this CTA's run of the tile
        if (!flush(wi)) break;
        const bool whole = w + 1 == p.windows && wi - seg0 + 1 == p.windows;
        const bool from_start = w - (wi - seg0) == 0;
        const int m = static_cast<int>(quad) * 32 + lane;
        if (whole) {
          const int f = mt * kTcM + feature_of(m);
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            const int n = nh * NC + j, col = nt * p.ncols + n;
            if (n < p.ncols && col < p.r && f < p.in) p.dA[static_cast<int64_t>(col) * p.in + f] = sum[j];
          }
        } else {
          // slot 0: the run began inside the tile; slot 1: at its start
          float *dst = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (from_start ? 1 : 0)) * p.ncols * kTcM + m;
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (nh * NC + j < p.ncols) dst[(nh * NC + j) * kTcM] = sum[j];
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) sum[j] = 0.0f;
        seg0 = wi + 1;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kCols);
  }
}

// dA of the tiles that more than one CTA worked on: their parts in CTA order.
// One block: one tile, 8 of its columns
__global__ void __launch_bounds__(256) grad_join_kernel(const GradParams p, int ctas) {
  const int chunks = (p.ncols + 7) / 8;
  const int tile = blockIdx.x / chunks;
  const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.windows;
  // the CTA that holds a unit: first_unit(i) <= unit < first_unit(i + 1)
  auto owner = [&](int64_t unit) {
    int i = static_cast<int>(unit * ctas / units);
    while (first_unit(units, i + 1, ctas) <= unit) ++i;
    while (first_unit(units, i, ctas) > unit) --i;
    return i;
  };
  const int i0 = owner(static_cast<int64_t>(tile) * p.windows), i1 = owner(static_cast<int64_t>(tile + 1) * p.windows - 1);
  if (i0 == i1) return;
  const int mt = tile % p.mtiles, nt = tile / p.mtiles;
  const int m = threadIdx.x % kTcM, f = mt * kTcM + feature_of(m);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = (blockIdx.x % chunks) * 8 + 2 * j + threadIdx.x / kTcM, col = nt * p.ncols + n;
    if (n >= p.ncols || col >= p.r || f >= p.in) continue;
    const int64_t at = static_cast<int64_t>(n) * kTcM + m, slot = static_cast<int64_t>(p.ncols) * kTcM;
    float s = p.part[(static_cast<int64_t>(i0) * 2 + 1) * slot + at];
    for (int i = i0 + 1; i <= i1; ++i) s += p.part[static_cast<int64_t>(i) * 2 * slot + at];
    p.dA[static_cast<int64_t>(col) * p.in + f] = s;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// columns of r per tile: as few tiles as hold it at 256 each, of equal width
int tile_columns(int64_t r) {
  const int64_t tiles = dora::ceil_div(r, 256);
  return static_cast<int>(dora::round_up(dora::ceil_div(r, tiles), 16));
}

template <int NC>
dora_status launch_grad(const CUtensorMap &mX, const CUtensorMap &mD, GradParams p, int ctas, cudaStream_t cs) {
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + 512;
  lora_grad_kernel<NC><<<static_cast<unsigned>(ctas), kThreadsG, smem, cs>>>(mX, mD, p);
  dora::count_launches(1);
  if (cudaGetLastError() != cudaSuccess) return DORA_ERR_CUDA;
  // no tile is cut when every CTA's run is a whole number of tiles
  const int64_t tiles = static_cast<int64_t>(p.mtiles) * p.ntiles;
  if (tiles % ctas != 0) {
    const int64_t blocks = tiles * dora::ceil_div(p.ncols, 8);
    grad_join_kernel<<<static_cast<unsigned>(blocks), 256, 0, cs>>>(p, ctas);
    dora::count_launches(1);
  }
  return dora::launch_status();
}

}  // namespace

extern "C" size_t dora_lora_grad_q8_workspace(int64_t T, int64_t in, int64_t r) {
  if (bad_size(T, 0) || bad_size(in, 0) || r < 1 || r > kMaxR) return 0;
  if (T == 0 || in == 0) return 256;
  // two parts per CTA, for up to kMaxCtasG CTAs
  const int64_t units = dora::ceil_div(in, kTcM) * dora::ceil_div(r, tile_columns(r)) * dora::ceil_div(T, kWin);
  const int64_t ctas = units < kMaxCtasG ? units : kMaxCtasG;
  return static_cast<size_t>(2 * ctas) * tile_columns(r) * kTcM * sizeof(float);
}

extern "C" dora_status dora_lora_grad_q8(const void *dxa, const void *xq, const void *xscale, int64_t T, int64_t in,
                                         int64_t r, float *dA, void *workspace, size_t workspace_bytes,
                                         dora_stream_t stream) {
  if (bad_size(T, 0) || bad_size(in, 0) || r < 1 || r > kMaxR) return DORA_ERR_SHAPE;
  if (in == 0) return DORA_OK;
  if (!dA || (T > 0 && (!dxa || !xq || !xscale))) return DORA_ERR_NULL;
  // TMA: 16-byte aligned bases and row strides
  if (in % 16 != 0 || r % 8 != 0) return DORA_ERR_ALIGN;
  if (!dora::aligned(dA, 16) || (T > 0 && (!dora::aligned(dxa, 16) || !dora::aligned(xq, 16)))) return DORA_ERR_ALIGN;
  if (!workspace || !dora::aligned(workspace, 256) || workspace_bytes < dora_lora_grad_q8_workspace(T, in, r))
    return DORA_ERR_WORKSPACE;
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(dA, 0, static_cast<size_t>(r) * in * sizeof(float), cs) == cudaSuccess ? DORA_OK
                                                                                                  : DORA_ERR_CUDA;
  GradParams p = {};
  static const void *const kernels[] = {
      (const void *)lora_grad_kernel<8>,  (const void *)lora_grad_kernel<16>, (const void *)lora_grad_kernel<32>,
      (const void *)lora_grad_kernel<48>, (const void *)lora_grad_kernel<64>, (const void *)lora_grad_kernel<96>,
      (const void *)lora_grad_kernel<128>};
  st = tc_init(device, &p.guard, kernels, sizeof(kernels) / sizeof(kernels[0]));
  if (st != DORA_OK) return st;
  p.T = static_cast<int>(T);
  p.in = static_cast<int>(in);
  p.r = static_cast<int>(r);
  p.ncols = tile_columns(r);
  p.boxes = static_cast<int>(dora::ceil_div(p.ncols, 64));
  p.mtiles = static_cast<int>(dora::ceil_div(in, kTcM));
  p.ntiles = static_cast<int>(dora::ceil_div(r, p.ncols));
  p.windows = static_cast<int>(dora::ceil_div(T, kWin));
  p.stage_bytes = kABytesG + kRawBytes + p.boxes * kBox;
  p.stages = static_cast<int>((kSmemMax - 1536) / p.stage_bytes);
  if (p.stages > kMaxStagesG) p.stages = kMaxStagesG;
  p.nsx = static_cast<int>(dora::ceil_div(in, kQBlock));
  p.scale = static_cast<const uint8_t *>(xscale);
  p.dA = dA;
  p.part = static_cast<float *>(workspace);
  CUtensorMap mX, mD;
  if (!map_q8(&mX, xq, T, in, kTok) || !make_map(&mD, dxa, true, T, r, r, kTok, 128)) return DORA_ERR_CUDA;
  const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.windows;
  const int sms = info.sms < kMaxCtasG ? info.sms : kMaxCtasG;
  const int ctas = units < sms ? static_cast<int>(units) : sms;
  const int half = p.ncols / 2;
  if (half <= 8) return launch_grad<8>(mX, mD, p, ctas, cs);
  if (half <= 16) return launch_grad<16>(mX, mD, p, ctas, cs);
  if (half <= 32) return launch_grad<32>(mX, mD, p, ctas, cs);
  if (half <= 48) return launch_grad<48>(mX, mD, p, ctas, cs);
  if (half <= 64) return launch_grad<64>(mX, mD, p, ctas, cs);
  if (half <= 96) return launch_grad<96>(mX, mD, p, ctas, cs);
  return launch_grad<128>(mX, mD, p, ctas, cs);
}
