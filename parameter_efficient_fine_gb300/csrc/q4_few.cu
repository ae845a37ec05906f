// x W^T of few tokens with a weight in 4 bits (see q4.cuh for the form) on the
// tensor cores of GB300 (sm_103a), without turning W into anything.
//
// tcgen05.mma kind::mxf8f6f4 takes E2M1 beside E4M3 and multiplies every 32 k of a
// row of either operand by a power of two, which is W's form.  x, a bf16, becomes
// two E4M3 pieces with a scale per 32 columns: h = E4M3(x / s), s the power of two
// that brings the group's largest magnitude to at most 448, and E4M3((x / s - h) 16)
// with the scale s / 16.  8 bits less the 4 of h leave 4, so x / s is their sum
// exactly down to 2^-6, and within 2^-14 below: an error of at most 2^-21 of the
// group's largest magnitude, as the fp32 sum itself makes.
//
// The features are the M side, the tokens' pieces the N side (NT first pieces, NT
// second ones).  A tile of 128 features and up to NT tokens is a cluster of CTAs
// that share its k range and meet in distributed shared memory, summed in rank
// order.
//   warps 0-7   x into pieces, in place, scale words into tensor memory (each warp
//               its lane quadrant), two groups of four taking turns; then the
//               result out of it
//   warp 8      tensor memory, MMA issue (four 32-wide steps per 128 k)
//   warps 9-10  copies of W, its scales and x.  W: 16 values, 8 bytes, to every 16
//               bytes of shared memory, the layout that the tensor core takes 4-bit
//               values in.  TMA does that (BOX) where rows are whole blocks of 128;
//               other rows come by asynchronous copies of 8 bytes
// Every wait on a shared-memory barrier is bounded; a wait that gives up records
// a code in the library's device error word and all roles leave.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q4.cuh"
#include "q4_mm.cuh"
#include "q8.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kKB = 128;                    // k per stage
constexpr unsigned kWBytes = kTcM * kKB;    // 16 KB of shared memory, 8 of W
constexpr int kGroups = 2, kTokWarps = 4;   // turns, warps of each
constexpr int kMmaWarp = kGroups * kTokWarps, kWWarps = 2;
constexpr int kFewThreads = 32 * (kMmaWarp + 1 + kWWarps);
constexpr int kMaxCluster = 8;              // the portable limit
constexpr int kFewCols = 128, kSfCol = 64, kSfStride = 8;   // tensor memory: scale words, 4 columns of W's and 2 of x's a stage

template <int NT> constexpr unsigned kXBytes = 2 * NT * kKB;
template <int NT> constexpr unsigned kStage = kWBytes + kXBytes<NT>;
// two CTAs an SM: half of the shared memory each.  Each group visits every use of its slots
template <int NT> constexpr int kFewStages = NT == 8 ? 6 : 4;
static_assert(kFewStages<8> % kGroups == 0 && kFewStages<32> % kGroups == 0, "slots of a group");

// 4, 8 or 16 bytes into shared memory, zeros where `bytes` is 0
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// an arrival on `bar` once this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// barrier `id` of `THREADS` threads, and whether `v` holds in all of them
template <int THREADS> __device__ __forceinline__ bool all_of(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.b32 a, %1, 0;\n\t"
      "bar.red.and.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "n"(THREADS)
      : "memory");
  return r != 0;
}

template <int NT, bool BOX>
__global__ void __launch_bounds__(kFewThreads, 2)
q4_few_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const Q4Params p,
              const __nv_bfloat16 *x, const uint8_t *wq) {
  constexpr int S = kFewStages<NT>, N = 2 * NT;
  constexpr int kMine = NT / kTokWarps;     // tokens a warp splits
  constexpr int kXCols = (N + 31) / 32;
  static_assert(NT % 8 == 0 && kXCols <= 2 && S * kSfStride + kSfCol <= kFewCols, "tensor memory");
  static_assert(NT * kTcM * 4 <= S * kStage<NT>, "the parts lie in the stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t *wscale = reinterpret_cast<uint32_t *>(smem + S * kStage<NT>);  // W's scale words, [S][128]
  uint32_t *words = wscale + S * kTcM;                                     // x's, [S][N]
  uint64_t *bars = reinterpret_cast<uint64_t *>(words + S * N);
  const uint32_t wfull0 = smem_u32(bars), xfull0 = wfull0 + 8u * S, empty0 = xfull0 + 8u * S, accf = empty0 + 8u * S;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 3 * S + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(wfull0 + 8u * s, 33 * kWWarps + (BOX ? 1 : 0));   // every thread's copies, every warp; boxes
      mbar_init(xfull0 + 8u * s, kTokWarps);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(accf, 1);
    ctl->abort = 0;
    fence_barrier_init();
    if (BOX) {
      prefetch_map(&mW);
      prefetch_map(&mX);
    }
  }
  for (int i = threadIdx.x; i < S * N; i += kFewThreads) words[i] = 0x7f7f7f7fu;
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(smem_u32(&ctl->tmem_base), kFewCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const uint32_t rank = cluster_ctarank();
  pdl_trigger();
  pdl_wait();       // the set-up above overlaps the end of the launch before

  Tile o = {};
  const bool work = find_tile(p, blockIdx.x / csize, &o);   // all of a cluster alike
  const int blocks = (p.kdim + kKB - 1) / kKB;
  // at least one block: a cluster has no more CTAs than there are
  const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / csize);
  const int kb1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / csize);
  const int ntok = o.t1 - o.t0, f0 = o.ft * kTcM;
  bool ok = true;

  if (!work) {
    // no tile for this cluster
  } else if (warp > kMmaWarp) {
    // ---------------------------------------------------------------- W
    const int i = threadIdx.x - 32 * (kMmaWarp + 1);
    const int G = p.in / kQ4Group;
    const bool words4 = G % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scale) & 3) == 0;
    ok = !loads_withheld(p.guard);
    Ring st(S);
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = guard_wait(empty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 71);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t at = smem_u32(smem) + st.i * kStage<NT>, xs = at + kWBytes;
      // x as it is: the 256 bytes of token t where its two pieces go, rows t and NT + t
      if (BOX) {
        if (warp == kMmaWarp + 1 && elect_one()) {
          const uint32_t fb = wfull0 + 8u * st.i;
          mbar_expect_tx(fb, kWBytes / 2 + kXBytes<NT>);      // a box counts the bytes it reads
          tma_load_3d(at, &mW, kb * kKB, f0, o.e, fb);
          tma_load_2d(xs, &mX, kb * kKB, o.t0, fb);
          tma_load_2d(xs + NT * 128u, &mX, kb * kKB + 64, o.t0, fb);
        }
        __syncwarp();
      } else {
        const int r = i / 8, c = i % 8;                       // first row, piece of 16 values
        const int64_t ld = p.in / 2;
        const uint8_t *src = wq + (static_cast<int64_t>(o.e) * p.out + f0 + r) * ld + kb * (kKB / 2) + 8 * c;
        const uint32_t dst = at + r * 128u + static_cast<uint32_t>((c ^ r) * 16);
        const int live = kb * kKB + 16 * c < p.in ? p.out - f0 - r : 0;      // rows from r that exist
#pragma unroll
        for (int j = 0; j < kTcM / 8; ++j) copy8(dst + j * 1024u, 8 * j < live ? src + 8 * j * ld : wq, 8 * j < live ? 8u : 0u);
#pragma unroll
        for (int j = 0; j < NT / 4; ++j) {
          const int t = 4 * j + i / 16, d = i % 16, k = kb * kKB + 8 * d;
          const bool has = t < ntok && k < p.in;
          copy16(xs + static_cast<uint32_t>(t + (d >= 8 ? NT : 0)) * 128u + static_cast<uint32_t>(d & 7) * 16u,
                 has ? x + static_cast<int64_t>(o.t0 + t) * p.in + k : x, has ? 16u : 0u);
        }
      }
      const uint32_t sc = smem_u32(wscale + st.i * kTcM);
#pragma unroll
      for (int j = 0; j < kTcM / (32 * kWWarps); ++j) {
        const int f = 32 * kWWarps * j + i;
        const bool has = f0 + f < p.out;
        const uint8_t *row = p.scale + (static_cast<int64_t>(o.e) * p.out + f0 + f) * G + 4 * kb;
        if (words4) {
          copy4(sc + 4u * f, has ? row : p.scale, has ? 4u : 0u);
        } else {
          uint32_t w = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) w |= (has && 4 * kb + q < G ? load_now(row + q) : 127u) << (8 * q);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc + 4u * f), "r"(w) : "memory");
        }
      }
      // the stage is full when the copies of all producing threads have landed and
      // their plain stores are out.  The threads that wait for it order both before
      // the tensor core's reads: a proxy fence here would wait for the copies
      copies_arrive(wfull0 + 8u * st.i);
      __syncwarp();
      if (lane == 0) mbar_arrive(wfull0 + 8u * st.i);
      st.next();
    }
    copies_wait();
    if (BOX && !ok && warp == kMmaWarp + 1) {
      // boxes in flight, whose barrier may never complete after an abort: they land
      // within microseconds, wait 1 ms
      const unsigned long long c0 = globaltimer();
      while (globaltimer() - c0 < 1000000ull) {
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    Ring st(S);
    for (int kb = kb0; kb < kb1; ++kb) {
      // after x's pieces come W, whose copies the pieces waited for
      ok = guard_wait(xfull0 + 8u * st.i, st.phase, ctl, p.guard, 72);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem) + st.i * kStage<NT>;
      const uint64_t a = sdesc<32>(at), b = sdesc<32>(at + kWBytes);
      const uint32_t sf = tmem + kSfCol + kSfStride * st.i;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_q8(tmem, a + 2u * k, b + 2u * k, idesc_q8(kTcM, N, k, false) | 5u << 7 /* A: E2M1 */, sf, sf + 4,
                 kb != kb0 || k != 0 ? 1u : 0u);
        mma_commit(empty0 + 8u * st.i);
      }
      __syncwarp();
      st.next();
    }
    if (elect_one()) {
      mma_commit(accf);
      wait_drain_ns(accf, 0, kWaitNs);   // every MMA issued is done before this CTA's memory is given back
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- x and the scales
    const int group = warp / kTokWarps, own = warp % kTokWarps;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(own) * 32u << 16);
    Ring st(S);
    if (group == 1) st.next();
    // a place without a token keeps what it holds: its column of the result is not read
    const int mine = own < ntok ? (ntok - own + kTokWarps - 1) / kTokWarps : 0;
    for (int kb = kb0 + group; kb < kb1; kb += kGroups, st.next(), st.next()) {
      ok = guard_wait(wfull0 + 8u * st.i, st.phase, ctl, p.guard, 74);
      uint8_t *xs = smem + st.i * kStage<NT> + kWBytes;
      uint8_t *ws = reinterpret_cast<uint8_t *>(words + st.i * N);
      uint2 raw[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j)
        raw[j] = *reinterpret_cast<const uint2 *>(xs + (own + kTokWarps * j + (lane >= 16 ? NT : 0)) * 128 + (lane & 15) * 8);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        if (j >= mine) break;
        float v[4] = {__uint_as_float(raw[j].x << 16), __uint_as_float(raw[j].x & 0xffff0000u),
                      __uint_as_float(raw[j].y << 16), __uint_as_float(raw[j].y & 0xffff0000u)};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, finite_bits(v[i]));
        // the group's 8 lanes
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
        const uint32_t b = scale_byte(m);
        const float inv = scale_inverse(b);
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = inf_to_nan(v[i]) * inv;
        const uint32_t h = quant4(v, 1.0f);
        dequant4(h, 1.0f, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v[i] - f[i];
        const uint32_t l = quant4(f, 16.0f);
        const int t = own + kTokWarps * j, at = ((lane >> 2) ^ (t & 7)) * 16 + (lane & 3) * 4;
        *reinterpret_cast<uint32_t *>(xs + t * 128 + at) = h;
        *reinterpret_cast<uint32_t *>(xs + (NT + t) * 128 + at) = l;      // NT % 8 == 0: the same swizzle
        if ((lane & 7) == 0) {
          ws[4 * t + (lane >> 3)] = static_cast<uint8_t>(b);
          ws[4 * (NT + t) + (lane >> 3)] = static_cast<uint8_t>(b - 4u);
        }
      }
      fence_async_proxy();
      // all scale words are there; the four warps go on or leave together
      ok = all_of<32 * kTokWarps>(1 + group, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t *sw = wscale + st.i * kTcM + lane;
      const uint32_t w0 = N >= 32 || lane < N ? words[st.i * N + lane] : 0x7f7f7f7fu;
      const uint32_t w1 = kXCols > 1 ? words[st.i * N + 32 + lane] : 0x7f7f7f7fu;
      const uint32_t all[8] = {sw[0], sw[32], sw[64], sw[96], w0, w1, 0u, 0u};
      tmem_st8(lane_addr + kSfCol + kSfStride * st.i, all);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(xfull0 + 8u * st.i);
    }
    // ---------------------------------------------------------------- result
    // into shared memory as [token][feature]: the stages are free once the
    // last MMA is done
    const bool got = guard_wait(accf, 0, ctl, p.guard, 75);
    ok = __all_sync(0xffffffffu, got) && ok;
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);
    const int f = own * 32 + lane;
#pragma unroll
    for (int c = 0; c < NT; c += 8) {
      if (c < ntok && (c / 8) % kGroups == group) {
        float a[8], b[8];
        tmem_ld<8>(lane_addr + c, a);
        tmem_ld<8>(lane_addr + NT + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[(c + i) * kTcM + f] = ok ? a[i] + b[i] : 0.0f;
      }
    }
  }
  tc_fence_before();
  if (csize > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (work) {
    // the parts of the cluster in rank order, one rounding to bf16: four
    // features a thread, neighbouring threads on neighbouring features
    const int quads = ntok * 32;
    const uint32_t base = smem_u32(smem);
    for (int i = static_cast<int>(rank) * kFewThreads + threadIdx.x; i < quads; i += static_cast<int>(csize) * kFewThreads) {
      float4 s = ld_cluster_f32x4(mapa_shared(base + 16u * i, 0));
      for (uint32_t c = 1; c < csize; ++c) {
        const float4 v = ld_cluster_f32x4(mapa_shared(base + 16u * i, c));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const int t = o.t0 + i / 32, f = f0 + 4 * (i % 32);
      if (f < p.nfeat)
        *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(t) * p.nfeat + f) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
  }
  if (csize > 1) cluster_sync();   // no CTA leaves while another reads its part
  else __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tmem, kFewCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// a stack of weights [experts, out, in] in boxes of 128 x 128 values, 8 bytes of every 16 of the result
bool map_w4(CUtensorMap *map, const void *base, int64_t experts, int64_t out, int64_t in) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(in), static_cast<cuuint64_t>(out), static_cast<cuuint64_t>(experts)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(in / 2), static_cast<cuuint64_t>(in / 2) * static_cast<cuuint64_t>(out)};
  cuuint32_t box[3] = {kKB, kTcM, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// x [T, in] in boxes of NT rows x 64 columns, unswizzled
bool map_x(CUtensorMap *map, const void *base, int64_t T, int64_t in, int nt) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(in), static_cast<cuuint64_t>(T)};
  cuuint64_t strides[1] = {2 * static_cast<cuuint64_t>(in)};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(nt)};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool BOX>
dora_status launch(const void *x, const void *wq, Q4Params p, int cluster, cudaStream_t cs) {
  constexpr auto kern = &q4_few_kernel<NT, BOX>;
  CUtensorMap mW = {}, mX = {};
  if (BOX && (!map_w4(&mW, wq, p.experts, p.out, p.in) || !map_x(&mX, x, p.T, p.in, NT))) return DORA_ERR_CUDA;
  constexpr size_t smem = 1024 + kFewStages<NT> * (kStage<NT> + 4 * kTcM + 8 * NT) + 8 * (3 * kFewStages<NT> + 1) + sizeof(SharedCtl);
  static_assert(2 * (smem + 1024) <= kSmemMax + 1024, "two CTAs an SM, each with 1 KB of the system's");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles * cluster));
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, mW, mX, p, static_cast<const __nv_bfloat16 *>(x), static_cast<const uint8_t *>(wq)) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

}  // namespace

namespace dora {

dora_status matmul_q4_few(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T,
                          int64_t out, int64_t in, int64_t experts, void *y, cudaStream_t cs) {
  DeviceInfo info;
  int device = 0;
  dora_status st = current_device(&info, &device);
  if (st != DORA_OK) return st;
  static const void *const kernels[] = {
      (const void *)q4_few_kernel<8, false>,  (const void *)q4_few_kernel<8, true>,  (const void *)q4_few_kernel<16, false>,
      (const void *)q4_few_kernel<16, true>, (const void *)q4_few_kernel<32, false>, (const void *)q4_few_kernel<32, true>};
  Q4Params p = {};
  st = tc_init(device, &p.guard, kernels, sizeof(kernels) / sizeof(kernels[0]));
  if (st != DORA_OK) return st;
  p.T = static_cast<int>(T);
  p.out = static_cast<int>(out);
  p.in = static_cast<int>(in);
  p.nfeat = p.out;
  p.kdim = p.in;
  p.experts = static_cast<int>(experts);
  p.offsets = offsets;
  p.scale = static_cast<const uint8_t *>(wscale);
  p.y = static_cast<__nv_bfloat16 *>(y);
  const int64_t groups = offsets ? (experts < T ? experts : T) : 1, per = ceil_div(T, groups);
  p.ntok = per <= 8 ? 8 : per <= 16 ? 16 : 32;
  p.ftiles = static_cast<int>(ceil_div(out, kTcM));
  p.tiles = p.ftiles * (offsets ? T / p.ntok + groups : ceil_div(T, p.ntok));
  // the k range over as many CTAs as keep all clusters resident at two CTAs an SM
  int cluster = 1;
  const int64_t blocks = ceil_div(in, kKB);
  while (cluster < kMaxCluster && p.tiles * cluster * 2 <= 2 * info.sms && cluster * 2 <= blocks) cluster *= 2;
  if (p.tiles * cluster > kMaxDim) return DORA_ERR_SHAPE;
  // boxes of 4-bit values take whole blocks of 128 and 32-byte rows
  const bool box = in % kKB == 0 && aligned(wq, 32);
  switch (p.ntok) {
    case 8: return box ? launch<8, true>(x, wq, p, cluster, cs) : launch<8, false>(x, wq, p, cluster, cs);
    case 16: return box ? launch<16, true>(x, wq, p, cluster, cs) : launch<16, false>(x, wq, p, cluster, cs);
  }
  return box ? launch<32, true>(x, wq, p, cluster, cs) : launch<32, false>(x, wq, p, cluster, cs);
}

}  // namespace dora
