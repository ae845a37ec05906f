// Products of two 8-bit matrices (see q8.cuh for the form) on the tensor cores
// of GB300 (sm_103a).
//
//   dora_matmul_q8     y  = x W^T      x [T, in], W [out, in]
//   dora_matmul_q8_t   dx = dy W       dy [T, out], the same W
//
// One k block is 128 wide, the width of a scale block, so the scales of a k
// block are one byte per token and one byte per 128 features.  The tensor core
// applies them itself: tcgen05.mma kind::mxf8f6f4 with block scaling multiplies
// every 32-wide step of k by a power of two per row of either operand, read
// from tensor memory; the four steps of a k block name the same byte.  The
// bytes of four consecutive k blocks form the 32-bit words that tensor memory
// holds them in, and the instruction picks one of the four.
//
// The features are the M side (128 rows of the tile are 128 features, whose
// scale is one byte), the tokens the N side, so a few tokens cost a narrow
// MMA and not a wide one mostly idle.  W is read as it is stored in both
// products: for x W^T a k block of a tile is 128 features x 128 bytes along k
// (K-major), for dy W it is 128 rows of k x 128 bytes along the features
// (M-major, the transpose bit of the instruction).
//
// q8_split_kernel: up to 128 tokens, one tile of 128 features x NT of them per
// cluster of CTAs, which share its k range; each CTA streams its part through
// a ring of TMA stages, and the parts meet in distributed shared memory,
// summed in rank order (bitwise reproducible, no workspace).  It has to read W
// once and is bound by that and by what lies around it: the launch, the first
// loads' latency and the joining of the parts are 3 us of the 13.2 that 1 x
// 8192 x 8192 takes (9.9 to read W at the copy bandwidth; 5100 GB/s), so its
// set-up and the first boxes of W into L2 overlap the end of the launch
// before.  37 x 14336 x 4096: 13.7 us (8.8); 128 x 8192 x 8192: 18.6 (10.3),
// where the token box is as large as W's.  dy W: 13.6, 14.2, 18.7.
//   warp 0     TMA producer: per k block the W box (16 KB) and the token box
//   warp 1     tensor memory, MMA issue (four 32-wide steps per k block)
//   warps 2-5  scale words into tensor memory, four k blocks at a time, each
//              warp its lane quadrant; then the result out of it
// q8_pair_kernel: for many tokens, tiles of 256 features x up to 256 tokens on CTA
// pairs (tcgen05.mma.cta_group::2, M = 256), one pair per two SMs, tile after
// tile.  Each CTA stages its 128 features and half of the tokens, so an SM loads
// half of what a single CTA's tile would; the scale words of all tokens of the
// tile are written in both CTAs.  Up to 224 tokens, two accumulators and the
// scale words fill tensor memory and a tile's result leaves while the next
// tile's MMAs run; a tile of more tokens has one accumulator.  It is bound by
// the tensor cores: their pipe is active in 83% of the cycles (8192^3), and
// over longer calls the power limit lowers the clock (15360 x 8192 x 8192: 605
// to 660 us, 3.1 to 3.4 PFLOP/s; 8192 x 4096 x 4096: 94 to 98 us; 512 x 8192 x 8192:
// 27 us; dy W 655 to 695 and 28 us).  A pair walks all of k alone, so a call of few
// tiles takes as long as one tile does: 129 x 256 x 14336 24 us, 129 x 4096 x 14336 29,
// 200 x 8192 x 8192 19 (10.6 to read and write).
//   warp 0      TMA producer (each CTA its own boxes, on the even CTA's barrier)
//   warp 1      tensor memory, MMA issue (even CTA).  A stage is two k blocks: waiting
//               for one and issuing its MMAs takes this warp about 600 cycles,
//               more than the 512 that the MMAs of one k block run
//   warps 2-5   scale words into tensor memory
//   warps 6-13  the result: out of tensor memory into registers as bf16 (the
//               next tile's MMAs may start), then 32 features a warp and token
//               straight to memory, 64 contiguous bytes
// Every wait on a shared-memory barrier is bounded; a wait that gives up
// records a code in the library's device error word and all roles leave.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "q8.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kKB = 128;                    // k per block: one 128-byte swizzled row, one scale
constexpr unsigned kWBytes = kTcM * kKB;    // 16 KB
constexpr int kSfSlots = 4;                 // scale words in flight, in groups of four k blocks
constexpr int kSplitThreads = 192;
constexpr int kSplitTok = 128;              // most tokens of q8_split_kernel (one tile of them)
constexpr int kMaxCluster = 8;              // the portable limit

struct MmParams {
  int T, nfeat, kdim;               // tokens, features of the result, k
  int kblocks;
  int ntiles, tiles;                // token tiles (pairs), all tiles
  int ntok;                         // tokens per tile (pairs)
  int stages;
  int nsx, nsw;                     // scale bytes per row of x, of W
  const uint8_t *xscale, *wscale;
  __nv_bfloat16 *y;
  Guard guard;
};

// a box's 128-byte rows are fetched with their neighbours' (128 x 8192 x 8192:
// 18.6 us, 19.0 without)
constexpr CUtensorMapL2promotion kPromote = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;

// D (+)= A B with a power-of-two scale per row of A and per row of B, E4M3
// operands in shared memory, scale words in tensor memory
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
// a box into L2
__device__ __forceinline__ void prefetch_box_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
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
// the scale bytes of k blocks 4 g .. 4 g + 3 of one row of an activation, a
// byte each; 1 past the last k block
__device__ __forceinline__ uint32_t token_word(const uint8_t *row, int g, int kblocks, bool words) {
  if (words) return load_now(reinterpret_cast<const uint32_t *>(row) + g);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (4 * g + i < kblocks ? load_now(row + 4 * g + i) : 127u) << (8 * i);
  return w;
}
// the same of 128 features of W: along a row of its scales, or down a column
template <bool TRANS>
__device__ __forceinline__ uint32_t weight_word(const MmParams &p, int mt, int g) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kb = 4 * g + i;
    const int64_t at = TRANS ? static_cast<int64_t>(kb) * p.nsw + mt : static_cast<int64_t>(mt) * p.nsw + kb;
    w |= (kb < p.kblocks ? load_now(p.wscale + at) : 127u) << (8 * i);
  }
  return w;
}

template <int NT, bool TRANS>
__global__ void __launch_bounds__(kSplitThreads, 1)
q8_split_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const MmParams p) {
  static_assert(NT % 16 == 0 && NT <= 128, "one chunk of scale words");
  constexpr unsigned kXBytes = NT * kKB;
  constexpr unsigned kStage = kWBytes + kXBytes;
  constexpr int kSfCol = NT < 32 ? 32 : NT;          // first column of the scale words
  constexpr int kCols = NT <= 32 ? 64 : NT == 64 ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(S) * kStage);
  // barriers: full[S], empty[S], scales full and empty [kSfSlots], accumulator
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S, sff0 = empty0 + 8u * S, sfe0 = sff0 + 8u * kSfSlots,
                 accf = sfe0 + 8u * kSfSlots;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 2 * S + 2 * kSfSlots + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(sff0 + 8u * s, 4);
      mbar_init(sfe0 + 8u * s, 1);
    }
    mbar_init(accf, 1);
    ctl->abort = 0;
    fence_barrier_init();
    prefetch_map(&mW);
    prefetch_map(&mX);
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

  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const uint32_t rank = cluster_ctarank();
  const int mt = static_cast<int>(blockIdx.x / csize);
  // at least one k block: a cluster has no more CTAs than there are
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / csize);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / csize);
  bool ok = true;
  // the launch before this one may still run.  Until it has ended nothing is
  // read or written here, but the first boxes of W are on their way into L2
  pdl_trigger();
  if (warp == 0 && elect_one())
    for (int kb = kb0; kb < kb1 && kb < kb0 + S; ++kb) {
      if (TRANS) prefetch_box_2d(&mW, mt * kTcM, kb * kKB);
      else prefetch_box_2d(&mW, kb * kKB, mt * kTcM);
    }
  pdl_wait();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    ok = !loads_withheld(p.guard);
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = guard_wait(empty0 + 8u * stage, phase ^ 1u, ctl, p.guard, 21);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t fb = full0 + 8u * stage;
      const uint32_t at = smem_u32(smem) + static_cast<uint32_t>(stage) * kStage;
      if (elect_one()) {
        mbar_expect_tx(fb, kStage);
        if (TRANS) tma_load_2d(at, &mW, mt * kTcM, kb * kKB, fb);
        else tma_load_2d(at, &mW, kb * kKB, mt * kTcM, fb);
        tma_load_2d(at + kWBytes, &mX, kb * kKB, 0, fb);
      }
      __syncwarp();
      ++issued;
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
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
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    bool up = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int grp = kb / 4 - kb0 / 4, slot = grp % kSfSlots;
      if (kb == kb0 || kb % 4 == 0)
        up = guard_wait(sff0 + 8u * slot, static_cast<uint32_t>(grp / kSfSlots) & 1u, ctl, p.guard, 22);
      up = up && guard_wait(full0 + 8u * stage, phase, ctl, p.guard, 23);
      if (!__all_sync(0xffffffffu, up)) break;
      tc_fence_after();
      const uint32_t at = smem_u32(smem) + static_cast<uint32_t>(stage) * kStage;
      const uint64_t a = sdesc<32>(at), b = sdesc<32>(at + kWBytes);
      const uint32_t idesc = idesc_q8(kTcM, NT, static_cast<uint32_t>(kb & 3), TRANS);
      const uint32_t sf = tmem + kSfCol + 8u * slot;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          // 32 k: 32 bytes along a K-major row; 32 rows of 128 bytes M-major
          // (descriptors count 16 bytes)
          mma_q8(tmem, a + (TRANS ? 256u : 2u) * k, b + 2u * k, idesc, sf, sf + 4, kb != kb0 || k != 0 ? 1u : 0u);
        mma_commit(empty0 + 8u * stage);
        if (kb % 4 == 3) mma_commit(sfe0 + 8u * slot);
      }
      __syncwarp();
      if (++stage == S) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (elect_one()) {
      mma_commit(accf);
      wait_drain_ns(accf, 0, kWaitNs);   // every MMA issued is done before this CTA's memory is given back
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- scales
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    const uint32_t lane_addr = tmem + ((quad * 32u) << 16);
    const bool words = p.nsx % 4 == 0 && (reinterpret_cast<uintptr_t>(p.xscale) & 3) == 0;
    const int g0 = kb0 / 4, g1 = (kb1 - 1) / 4 + 1;
    for (int g = g0; g < g1; ++g) {
      uint32_t w[8];
      w[0] = w[1] = w[2] = w[3] = weight_word<TRANS>(p, mt, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 32 * j + lane;
        w[4 + j] = 32 * j < NT && t < p.T ? token_word(p.xscale + static_cast<int64_t>(t) * p.nsx, g, p.kblocks, words)
                                          : 0x7f7f7f7fu;
      }
      const int slot = (g - g0) % kSfSlots;
      const bool got = guard_wait(sfe0 + 8u * slot, (static_cast<uint32_t>((g - g0) / kSfSlots) & 1u) ^ 1u, ctl, p.guard, 24);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_st8(lane_addr + kSfCol + 8u * slot, w);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sff0 + 8u * slot);
    }
    // ---------------------------------------------------------------- result
    // into shared memory as [token][feature]: the stages are free once the
    // last MMA is done
    const bool got = guard_wait(accf, 0, ctl, p.guard, 25);
    ok = __all_sync(0xffffffffu, got) && ok;
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);
    const int f = static_cast<int>(quad) * 32 + lane;
#pragma unroll
    for (int c = 0; c < NT; c += 16) {
      if (c < p.T) {
        float v[16];
        tmem_ld<16>(lane_addr + c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kTcM + f] = ok ? v[i] : 0.0f;
      }
    }
  }
  tc_fence_before();
  if (csize > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  {
    // the parts of the cluster in rank order, one rounding to bf16: four
    // features a thread, neighbouring threads on neighbouring features
    const int live = p.T * 32;
    const uint32_t base = smem_u32(smem);
    for (int i = static_cast<int>(rank) * kSplitThreads + threadIdx.x; i < live;
         i += static_cast<int>(csize) * kSplitThreads) {
      float4 s = ld_cluster_f32x4(mapa_shared(base + 16u * i, 0));
      for (uint32_t c = 1; c < csize; ++c) {
        const float4 v = ld_cluster_f32x4(mapa_shared(base + 16u * i, c));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      const int t = i / 32, f = mt * kTcM + 4 * (i % 32);
      if (f < p.nfeat)
        *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(t) * p.nfeat + f) =
            make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
  }
  if (csize > 1) cluster_sync();   // no CTA leaves while another reads its part
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, kCols);
  }
}

// ---------------------------------------------------------------------------
// CTA pairs
// ---------------------------------------------------------------------------
constexpr int kPairTok = 256;                        // most tokens per tile, half of them staged by either CTA
constexpr int kPairTwo = 224;                        // most tokens of a tile that has two accumulators
constexpr int kPairFeat = 256;                       // features per tile
constexpr int kPairKB = 2;                           // k blocks per stage
constexpr unsigned kPairBox = kTcM * kKB;            // 16 KB: 128 features, one k block
// half of the tile's tokens, one k block
__host__ __device__ constexpr unsigned pair_xbox(int ntok) { return static_cast<unsigned>(ntok / 2 * kKB); }
__host__ __device__ constexpr unsigned pair_stage(int ntok) { return kPairKB * (kPairBox + pair_xbox(ntok)); }
constexpr int kPairThreads = 14 * 32;
constexpr int kPairSfCol = 2 * kPairTwo, kPairSfStride = 16;   // scale words: 4 columns of W's, 8 of the tokens'
// feature tiles per tile-order group, for reuse in L2 (15360 x 8192 x 8192: 701,
// 676, 629, 628 us with 2, 4, 8, 16, 671 with one group; 8192 x 14336 x 4096: 327
// to 333 with each, 341 with one group)
constexpr int kGroupF = 8;

__device__ __forceinline__ void mma_q8_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
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
// the accumulator of a pair's tile: two in turn, or one
struct Acc {
  int n, i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Acc(int ntok) : n(ntok > kPairTwo ? 1 : 2) {}
  __device__ __forceinline__ uint32_t column() const { return static_cast<uint32_t>(i * kPairTwo); }
  __device__ __forceinline__ void next() {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};
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

template <bool TRANS>
__global__ void __launch_bounds__(kPairThreads, 1)
q8_pair_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const MmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int S = p.stages;
  const uint32_t xbox = pair_xbox(p.ntok), stage_bytes = pair_stage(p.ntok);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S * stage_bytes);
  // barriers (a pair uses the even CTA's full, scales full and accumulator
  // empty): full, empty, scales full and empty, accumulator full and empty, end
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S, sff0 = empty0 + 8u * S,
                 sfe0 = sff0 + 8u * kSfSlots, accf = sfe0 + 8u * kSfSlots, acce = accf + 16, fin = acce + 16;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 2 * S + 2 * kSfSlots + 5);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(sff0 + 8u * s, 8);     // four warps of either CTA
      mbar_init(sfe0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf + 8u * b, 1);
      mbar_init(acce + 8u * b, 16);    // eight warps of either CTA
    }
    mbar_init(fin, 1);
    ctl->abort = 0;
    fence_barrier_init();
    prefetch_map(&mW);
    prefetch_map(&mX);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised before either signals the other's
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  pdl_trigger();
  pdl_wait();       // the set-up above overlaps the end of the launch before
  const int pair = static_cast<int>(blockIdx.x / 2), npairs = static_cast<int>(gridDim.x / 2);
  const int ftiles = p.tiles / p.ntiles, stages = (p.kblocks + kPairKB - 1) / kPairKB, groups = (p.kblocks + 3) / 4;
  // tile t: groups of kGroupF feature tiles, all token tiles of a group in turn
  auto place = [&](int t, int *ft, int *tt) {
    const int per = kGroupF * p.ntiles, g = t / per, f0 = g * kGroupF, gf = min(kGroupF, ftiles - f0), r = t - g * per;
    *tt = r / gf;
    *ft = f0 + r - *tt * gf;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    bool ok = !loads_withheld(p.guard);
    bool issued = false;
    Ring st(S);
    for (int t = pair; t < p.tiles && ok; t += npairs) {
      int ft, tt;
      place(t, &ft, &tt);
      const int f0 = ft * kPairFeat + static_cast<int>(rank) * kTcM, t0 = tt * p.ntok + static_cast<int>(rank) * (p.ntok / 2);
      for (int s = 0; s < stages; ++s) {
        ok = guard_wait(empty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 41);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t fb = full0 + 8u * st.i, lb = mapa_shared(fb, 0);
        const uint32_t at = smem_u32(smem) + st.i * stage_bytes;
        if (elect_one()) {
          // the even CTA's barrier counts both CTAs' bytes
          if (rank == 0) mbar_expect_tx(fb, 2 * stage_bytes);
#pragma unroll
          for (int k = 0; k < kPairKB; ++k) {
            const int kx = (s * kPairKB + k) * kKB;
            if (TRANS) tma_load_2d_pair(at + k * kPairBox, &mW, f0, kx, lb);
            else tma_load_2d_pair(at + k * kPairBox, &mW, kx, f0, lb);
            tma_load_2d_pair(at + kPairKB * kPairBox + k * xbox, &mX, kx, t0, lb);
          }
        }
        __syncwarp();
        issued = true;
        st.next();
      }
    }
    if (!ok && issued) {
      // copies in flight, whose barrier may never complete after an abort: they
      // land within microseconds, wait 1 ms
      const unsigned long long t0 = globaltimer();
      while (globaltimer() - t0 < 1000000ull) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------------- MMA issuer
      // (a commit arrives on the barrier of this CTA and on the peer's)
      bool ok = true;
      Ring st(S), sf(kSfSlots);
      Acc acc(p.ntok);
      const uint32_t peer_off = mapa_shared(full0, peer) - full0;   // to the peer's copy of a barrier
      const uint32_t id0 = idesc_q8(kPairFeat, p.ntok, 0, TRANS);
      for (int t = pair; t < p.tiles && ok; t += npairs, acc.next()) {
        ok = guard_wait(acce + 8u * acc.i, acc.phase ^ 1u, ctl, p.guard, 42);
        const uint32_t d = tmem + acc.column();
        for (int s = 0; s < stages; ++s) {
          const bool second = (s & 1) != 0;   // which two of the group's four k blocks
          if (!second) ok = ok && guard_wait(sff0 + 8u * sf.i, sf.phase, ctl, p.guard, 43);
          ok = ok && guard_wait(full0 + 8u * st.i, st.phase, ctl, p.guard, 44);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t at = smem_u32(smem) + st.i * stage_bytes;
          const uint64_t a = sdesc<32>(at), b = sdesc<32>(at + kPairKB * kPairBox);
          const uint32_t sfa = tmem + kPairSfCol + kPairSfStride * sf.i;
          const uint32_t id = second ? id0 | (2u << 4) | (2u << 29) : id0;
          const bool last = s + 1 == stages;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kPairKB; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mma_q8_pair(d, a + (kPairBox >> 4) * k + (TRANS ? 256u : 2u) * j, b + (xbox >> 4) * k + 2u * j,
                            id | (static_cast<uint32_t>(k) << 4) | (static_cast<uint32_t>(k) << 29), sfa, sfa + 4,
                            s != 0 || k != 0 || j != 0 ? 1u : 0u);
            mma_commit_pair(empty0 + 8u * st.i);
            mma_commit_pair(empty0 + 8u * st.i + peer_off);
            if (second || last) {
              mma_commit_pair(sfe0 + 8u * sf.i);
              mma_commit_pair(sfe0 + 8u * sf.i + peer_off);
            }
            if (last) {
              mma_commit_pair(accf + 8u * acc.i);
              mma_commit_pair(accf + 8u * acc.i + peer_off);
            }
          }
          __syncwarp();
          if (second || last) sf.next();
          st.next();
        }
      }
      if (elect_one()) {
        mma_commit_pair(fin);
        wait_drain_ns(fin, 0, kWaitNs);
      }
      __syncwarp();
    }
  } else if (warp < 6) {
    // ---------------------------------------------------------------- scales
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const bool words = p.nsx % 4 == 0 && (reinterpret_cast<uintptr_t>(p.xscale) & 3) == 0;
    bool ok = true;
    Ring sf(kSfSlots);
    for (int t = pair; t < p.tiles && ok; t += npairs) {
      int ft, tt;
      place(t, &ft, &tt);
      const int wt = 2 * ft + static_cast<int>(rank);   // 128 features
      const bool live = wt * kTcM < p.nfeat;
      const uint8_t *row[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int tok = tt * p.ntok + 32 * j + lane;
        row[j] = tok < p.T ? p.xscale + static_cast<int64_t>(tok) * p.nsx : nullptr;
      }
      for (int g = 0; g < groups; ++g) {
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = row[j] ? token_word(row[j], g, p.kblocks, words) : 0x7f7f7f7fu;
        const uint32_t w = live ? weight_word<TRANS>(p, wt, g) : 0x7f7f7f7fu;
        ok = guard_wait(sfe0 + 8u * sf.i, sf.phase ^ 1u, ctl, p.guard, 45);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t to = lane_addr + kPairSfCol + kPairSfStride * sf.i;
        tmem_st4(to, w, w, w, w);
        tmem_st8(to + 4, x);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair_relaxed(mapa_shared(sff0 + 8u * sf.i, 0));
        sf.next();
      }
    }
  } else {
    // ---------------------------------------------------------------- result
    const int e = warp - 6;
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    const int half = p.ntok / 2;                   // tokens of this warp, from c0
    const int c0 = (e >> 2) * half;
    const uint32_t lane_addr = tmem + ((quad * 32u) << 16) + static_cast<uint32_t>(c0);
    bool ok = true;
    Acc acc(p.ntok);
    for (int t = pair; t < p.tiles && ok; t += npairs, acc.next()) {
      int ft, tt;
      place(t, &ft, &tt);
      ok = guard_wait(accf + 8u * acc.i, acc.phase, ctl, p.guard, 46);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t o[kPairTok / 4];                    // two tokens a register
#pragma unroll
      for (int c = 0; c < kPairTok / 2; c += 8)
        if (c < half) {
          float v[8];
          tmem_ld<8>(lane_addr + acc.column() + static_cast<uint32_t>(c), v);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[c / 2 + i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair_relaxed(mapa_shared(acce + 8u * acc.i, 0));
      const int f = ft * kPairFeat + static_cast<int>(rank) * kTcM + static_cast<int>(quad) * 32 + lane;
      const int t0 = tt * p.ntok + c0;
      if (f < p.nfeat) {
        uint16_t *y = reinterpret_cast<uint16_t *>(p.y) + static_cast<int64_t>(t0) * p.nfeat + f;
        const int64_t ld = p.nfeat;
        const int live = min(p.T - t0, half);
#pragma unroll
        for (int i = 0; i < kPairTok / 4; ++i, y += 2 * ld) {
          if (2 * i < live) y[0] = static_cast<uint16_t>(o[i]);
          if (2 * i + 1 < live) y[ld] = static_cast<uint16_t>(o[i] >> 16);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // the even CTA's MMAs, which read this CTA's shared memory and write its
  // tensor memory, are complete, and both CTAs' results are out
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
size_t split_smem(int nt, int stages) { return 1024 + static_cast<size_t>(stages) * (kWBytes + nt * kKB) + 512; }

template <int NT, bool TRANS>
dora_status launch_split(const CUtensorMap &mW, const CUtensorMap &mX, MmParams p, int cluster, cudaStream_t cs) {
  constexpr auto kern = &q8_split_kernel<NT, TRANS>;
  // two CTAs an SM: half of the shared memory each
  constexpr int stages = static_cast<int>((kSmemMax / 2 - 2048) / (kWBytes + NT * kKB));
  static_assert(2 * stages + 2 * kSfSlots + 1 <= 56, "barriers and control words");
  p.stages = stages;
  const size_t smem = split_smem(NT, stages);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles * cluster));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kern, mW, mX, p) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

dora_status mm_init(int device, MmParams *p) {
  static const void *const kernels[] = {
      (const void *)q8_split_kernel<16, false>, (const void *)q8_split_kernel<32, false>,
      (const void *)q8_split_kernel<64, false>, (const void *)q8_split_kernel<128, false>,
      (const void *)q8_split_kernel<16, true>,  (const void *)q8_split_kernel<32, true>,
      (const void *)q8_split_kernel<64, true>,  (const void *)q8_split_kernel<128, true>,
      (const void *)q8_pair_kernel<false>,      (const void *)q8_pair_kernel<true>};
  return tc_init(device, &p->guard, kernels, sizeof(kernels) / sizeof(kernels[0]));
}

// as many stages as fit: the loads' latency over them is what a narrow tile's
// stage takes (64 tokens: five of 40 KB; 256: three of 64 KB.  200 x 8192 x 8192,
// in tiles of 112: 19.1 us with four, 21.4 with three)
constexpr int pair_stages(int ntok) { return static_cast<int>((kSmemMax - 1024 - 512) / pair_stage(ntok)); }
constexpr size_t pair_smem(int ntok) { return 1024 + pair_stages(ntok) * pair_stage(ntok) + 512; }
static_assert(2 * pair_stages(64) + 2 * kSfSlots + 5 <= 56, "barriers and control words");

void pair_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int ntok, int pairs, cudaStream_t cs) {
  *cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg->gridDim = dim3(2 * static_cast<unsigned>(pairs));
  cfg->blockDim = dim3(kPairThreads);
  cfg->dynamicSmemBytes = pair_smem(ntok);
  cfg->stream = cs;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// pairs that are resident at once (a pair takes every npairs-th tile, so one
// that had to wait for another to end would double the time); 0 where the
// device has no clusters of two
int resident_pairs(int device, int sms) {
  static std::mutex mu;
  static int known[64] = {};   // pairs + 1
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (known[device] == 0) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    pair_config(&cfg, attr, kPairTok, sms / 2, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, q8_pair_kernel<false>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[device] = n + 1;
  }
  return known[device] - 1;
}

template <bool TRANS>
dora_status launch_pairs(const void *q, const void *wq, int64_t out, int64_t in, MmParams p, int pairs,
                         cudaStream_t cs) {
  CUtensorMap mW, mX;
  if (!map_q8(&mW, wq, out, in, 128, kPromote) || !map_q8(&mX, q, p.T, p.kdim, p.ntok / 2, kPromote))
    return DORA_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  pair_config(&cfg, attr, p.ntok, p.tiles < pairs ? p.tiles : pairs, cs);
  if (cudaLaunchKernelEx(&cfg, q8_pair_kernel<TRANS>, mW, mX, p) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

// q: the activation's bytes [T, kdim]; features and k are (out, in) or, for dy W, (in, out)
template <bool TRANS>
dora_status run_matmul(const void *q, const void *scale, const void *wq, const void *wscale, int64_t T, int64_t out,
                       int64_t in, void *y, dora_stream_t stream) {
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  MmParams p = {};
  st = mm_init(device, &p);
  if (st != DORA_OK) return st;
  p.T = static_cast<int>(T);
  p.nfeat = static_cast<int>(TRANS ? in : out);
  p.kdim = static_cast<int>(TRANS ? out : in);
  p.kblocks = static_cast<int>(dora::ceil_div(p.kdim, kKB));
  p.nsx = p.kblocks;
  p.nsw = static_cast<int>(dora::ceil_div(in, kQBlock));
  p.xscale = static_cast<const uint8_t *>(scale);
  p.wscale = static_cast<const uint8_t *>(wscale);
  p.y = static_cast<__nv_bfloat16 *>(y);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // up to 128 tokens W is read by all SMs at once, its k range split where there
  // are few tiles; the pairs, one tile of 256 features each, leave many of them
  // idle where a weight has few features (us split / on pairs: 70 x 4096 x 14336
  // 16.0 / 24.6, 128 x 4096 x 14336 18.5 / 24.7, 70 x 8192 x 8192 16.2 / 17.2).  128 is
  // the most that the split kernel takes, not where the two are even: that lies
  // lower for a wide weight (128 x 8192 x 8192 18.6 / 17.5, 70 x 14336 x 4096 15.1 / 14.2,
  // 128 x 14336 x 4096 17.2 / 14.8) and higher for a narrow one (128 x 256 x 14336 10.0 on
  // the split kernel, 129 on pairs 23.9)
  if (T > kSplitTok) {
    const int pairs = resident_pairs(device, info.sms);
    if (pairs == 0) return DORA_ERR_CUDA;
    const int64_t ftiles = dora::ceil_div(p.nfeat, kPairFeat);
    // tokens per tile: the least time over the waves of tiles, a stage of two k
    // blocks taken as n + 100, and 20 more with one accumulator (15360 x 8192 x 8192,
    // us a stage: 0.37, 0.45, 0.54, 0.59, 0.67, 0.79 with 64, 128, 176, 192, 224,
    // 256 tokens; with 125 and 10, which prefer wider tiles: 5000 x 14336 x 4096
    // 210 us against 192, 8192 x 4096 x 4096 99 against 94, others the same)
    int64_t best = 0;
    for (int n = 64; n <= kPairTok; n += 16) {
      const int64_t waves = dora::ceil_div(ftiles * dora::ceil_div(T, n), pairs);
      const int64_t cost = waves * (n + 100 + (n > kPairTwo ? 20 : 0));
      if (best == 0 || cost < best) {
        best = cost;
        p.ntok = n;
      }
    }
    p.stages = pair_stages(p.ntok);
    p.ntiles = static_cast<int>(dora::ceil_div(T, p.ntok));
    const int64_t tiles = ftiles * p.ntiles;
    if (tiles > kMaxDim) return DORA_ERR_SHAPE;
    p.tiles = static_cast<int>(tiles);
    return launch_pairs<TRANS>(q, wq, out, in, p, pairs, cs);
  }
  const int nt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  p.tiles = static_cast<int>(dora::ceil_div(p.nfeat, kTcM));
  // the k range over as many CTAs as keep all clusters resident at two CTAs an SM
  // (us with clusters of up to 1, 2, 4, 8: 1 x 8192 x 8192 20.0, 14.6, 13.2, 13.2;
  // 37 x 4096 x 14336 33.8, 22.1, 15.7, 14.3; 1 x 1024 x 8192 18.3, 11.3, 8.0, 7.9)
  int cluster = 1;
  while (cluster < kMaxCluster && p.tiles * cluster * 2 <= 2 * info.sms && cluster * 2 <= p.kblocks) cluster *= 2;
  CUtensorMap mW, mX;
  if (!map_q8(&mW, wq, out, in, 128, kPromote) || !map_q8(&mX, q, T, p.kdim, nt, kPromote)) return DORA_ERR_CUDA;
  switch (nt) {
    case 16: return launch_split<16, TRANS>(mW, mX, p, cluster, cs);
    case 32: return launch_split<32, TRANS>(mW, mX, p, cluster, cs);
    case 64: return launch_split<64, TRANS>(mW, mX, p, cluster, cs);
  }
  return launch_split<128, TRANS>(mW, mX, p, cluster, cs);
}

dora_status matmul_check(const void *xq, const void *xscale, const void *wq, const void *wscale, int64_t out,
                         int64_t in, const void *y) {
  if (!xq || !xscale || !wq || !wscale || !y) return DORA_ERR_NULL;
  // TMA: 16-byte aligned bases and row strides
  if (out % 16 != 0 || in % 16 != 0) return DORA_ERR_ALIGN;
  if (!dora::aligned(xq, 16) || !dora::aligned(wq, 16) || !dora::aligned(y, 16)) return DORA_ERR_ALIGN;
  return DORA_OK;
}

}  // namespace

// (both kernels join a tile's parts on chip)
extern "C" size_t dora_matmul_q8_workspace(int64_t, int64_t, int64_t) { return 0; }
extern "C" size_t dora_matmul_q8_t_workspace(int64_t, int64_t, int64_t) { return 0; }

extern "C" dora_status dora_matmul_q8(const void *xq, const void *xscale, const void *wq, const void *wscale, int64_t T,
                                      int64_t out, int64_t in, void *y, void *, size_t, dora_stream_t stream) {
  if (bad_size(T, 0) || bad_size(out, 0) || bad_size(in, 1)) return DORA_ERR_SHAPE;
  if (T == 0 || out == 0) return DORA_OK;
  const dora_status st = matmul_check(xq, xscale, wq, wscale, out, in, y);
  if (st != DORA_OK) return st;
  return run_matmul<false>(xq, xscale, wq, wscale, T, out, in, y, stream);
}

extern "C" dora_status dora_matmul_q8_t(const void *dyq, const void *dyscale, const void *wq, const void *wscale,
                                        int64_t T, int64_t out, int64_t in, void *dx, void *, size_t,
                                        dora_stream_t stream) {
  if (bad_size(T, 0) || bad_size(out, 1) || bad_size(in, 0)) return DORA_ERR_SHAPE;
  if (T == 0 || in == 0) return DORA_OK;
  const dora_status st = matmul_check(dyq, dyscale, wq, wscale, out, in, dx);
  if (st != DORA_OK) return st;
  return run_matmul<true>(dyq, dyscale, wq, wscale, T, out, in, dx, stream);
}
