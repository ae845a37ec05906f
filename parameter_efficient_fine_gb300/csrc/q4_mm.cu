// Products with a weight in 4 bits (see q4.cuh for the form) on the tensor cores
// of GB300 (sm_103a), in bf16.
//
//   dora_matmul_q4     y  = x W^T      x [T, in], W [out, in]
//   dora_matmul_q4_t   dx = dy W       dy [T, out], the same W
//
// With experts, W is a stack and the rows of x are sorted by expert: rows
// offsets[e] to offsets[e + 1] meet W[e].
//
// The features are the M side, the tokens the N side.  A block of W, 128 rows of
// it by 128 columns, arrives as it is stored (8 KB) and is turned into bf16 by
// conversion warps.  For x W^T its rows are features: they go to
// tensor memory, a lane each, from where the tensor core takes them as its A
// operand.  For dy W its rows are k: they go to shared memory as two panels of 64
// rows x 64 features, 128 bytes a row, swizzled, read M-major.  Neither makes a
// transposed copy.
//
// CTA pairs (tcgen05.mma.cta_group::2): tiles of 256 features by up to 256 tokens,
// each CTA converting its 128 features and staging half of the tokens.
//   warp 0       TMA: tokens into the stages
//   warp 1       tensor memory, MMA issue (even CTA)
//   warp 2       TMA: blocks of W into a ring of their own
//   then         conversion, four groups of four warps taking turns at the blocks (dy W:
//                three, which is what shared memory holds)
//   last 8       the result
// A tile's MMAs and copies are as wide as its own tokens are, in steps of 32: a tile of
// an expert is seldom full, and one 256 wide saves converting W twice (4096 tokens at 32
// experts of 2048 x 4096: 76 us, 96 with all tiles' MMAs 256 wide).
//
// What bounds it: with 256 tokens, the MMAs, 0.56 us a block of 128 k, and over longer
// calls the power limit (8192 x 4096 x 4096 143 to 147 us, 1.9 PFLOP/s; 15360 x 8192 x
// 8192 1127; 512 x 8192 x 8192 42); of dy W they read both operands from shared memory
// and take a little more (15360 x 8192 x 8192 1145 to 1170 us, 1.8 PFLOP/s; 512 44).  With
// up to 192 the conversion and its hand-overs, about 0.46 us a block whatever the tokens
// (128 x 38912 x 4096 34 us; 700 x 8192 x 8192 61; 4096 tokens evenly at 32 experts of
// 2048 x 4096 63 to 70, unevenly 74, dy W 85 and 85 to 95).  Its groups take whole blocks, with
// half the waits and addresses of half blocks (with those, and values by a table, 128 x
// 38912 x 4096 took 40, 700 70, dy W 512 53).
// Every wait on a shared-memory barrier is bounded; a wait that gives up records
// a code in the library's device error word and all roles leave.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "q4.cuh"
#include "q4_mm.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kKB = 128;                              // the side of a block of W
constexpr int kKS = 64;                               // k per stage
constexpr int kTileF = 256;                           // features per tile
constexpr int kTileT = 256;                           // most tokens per tile
constexpr unsigned kRawBytes = 128 * kKB / 2;         // 8 KB
constexpr unsigned kPanel = kKS * 128;                // 8 KB: 64 rows of 64 bf16
constexpr int kGroupWarps = 4, kOutWarps = 8;
template <bool TRANS> constexpr int kGroups = TRANS ? 3 : 4;   // of conversion warps
constexpr int kConv0 = 3;
template <bool TRANS> constexpr int kOut0 = kConv0 + kGroups<TRANS> * kGroupWarps;
template <bool TRANS> constexpr int kThreadsMm = 32 * (kOut0<TRANS> + kOutWarps);
constexpr int kAhead = 2;                             // blocks whose scales are on their way
constexpr uint32_t kACol = 256;                       // x W^T: first column of the converted W
// half of the tile's tokens, 64 k
__host__ __device__ constexpr unsigned tok_box(int ntok) { return static_cast<unsigned>(ntok / 2 * 128); }
template <bool TRANS> __host__ __device__ constexpr unsigned stage_size(int ntok) {
  return (TRANS ? 2 * kPanel : 0) + tok_box(ntok);
}
// stages and blocks of W in flight.  x W^T: a stage is 32 columns of tensor memory,
// of which the accumulator leaves 256
template <bool TRANS> constexpr int kStages = TRANS ? 6 : 8;
// dy W: six blocks of W where the stages leave room, which hides their copies' latency
// where few tokens leave little else to do (129 x 8192 x 8192 26.8 us, 30.8 with three)
template <bool TRANS> constexpr int raw_slots(int ntok) { return !TRANS ? 8 : ntok <= 192 ? 6 : 3; }
// a wait goes by the parity of a phase, so a group visits every use of the slots that
// it visits: it has a slot of the ring of blocks, and one or two of that of W
template <bool TRANS> constexpr bool turns_ok() {
  for (int n = 32; n <= kTileT; n += 32)
    if (raw_slots<TRANS>(n) != kGroups<TRANS> && raw_slots<TRANS>(n) != 2 * kGroups<TRANS>) return false;
  return kStages<TRANS> == 2 * kGroups<TRANS>;
}
static_assert(turns_ok<false>() && turns_ok<true>(), "slots of a group");

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t *v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// D (+)= A B over the pair, A of each CTA in its tensor memory
__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// arrive on an mbarrier of the pair after writes to this CTA's shared memory, which
// the tensor core of this SM reads; they are ordered before it by fence_async_proxy
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// once all MMAs of the pair issued so far are done, arrive on a barrier of either CTA,
// at the same place in both
__device__ __forceinline__ void mma_commit_both(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\t"
      "mov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
      : "memory");
}
// the accumulators: for x W^T the converted W leaves 256 columns, two of 128 tokens
// or one of more
struct Acc {
  int n, stride, i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ Acc(bool trans, int ntok) : n(trans || ntok <= 128 ? 2 : 1), stride(trans ? 256 : 128) {}
  __device__ __forceinline__ uint32_t column() const { return static_cast<uint32_t>(i * stride); }
  __device__ __forceinline__ void next() {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// M-major panels: 64 features a row of 128 bytes, k down the rows, the panel of the
// next 64 features kPanel further
__device__ __forceinline__ uint64_t sdesc_mmajor(uint32_t saddr) {
  return (sdesc<32>(saddr) & ~(static_cast<uint64_t>(0x3fff) << 16)) | (static_cast<uint64_t>(kPanel >> 4) << 16);
}

// A tile, or a part of its k where the tiles are few: blocks b0 to b0 + nb
struct Unit : Tile {
  int n;                            // tokens that its MMAs take: its own, in steps of 32
  int part, b0, nb;
};
__device__ __forceinline__ bool find_unit(const Q4Params &p, int u, Unit *o) {
  const int t = p.parts > 1 ? u / p.parts : u, blocks = (p.kdim + kKB - 1) / kKB;
  o->part = u - t * p.parts;
  o->b0 = blocks * o->part / p.parts;
  o->nb = blocks * (o->part + 1) / p.parts - o->b0;
  if (t >= p.tiles || !find_tile(p, t, o)) return false;
  o->n = (o->t1 - o->t0 + 31) & ~31;
  return true;
}

template <bool TRANS, int R>
__global__ void __launch_bounds__(kThreadsMm<TRANS>, 1)
q4_pair_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const Q4Params p) {
  constexpr int S = kStages<TRANS>, B = S / 2, NG = kGroups<TRANS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t xbox = tok_box(p.ntok), stage_bytes = stage_size<TRANS>(p.ntok);
  uint8_t *raw = smem + S * stage_bytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(raw + R * kRawBytes);
  // barriers (a pair uses the even CTA's full and accumulator empty): tokens here and
  // W converted, empty; raw full and empty; accumulator full and empty; end
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * B, rfull0 = empty0 + 8u * B,
                 rempty0 = rfull0 + 8u * R, accf = rempty0 + 8u * R, acce = accf + 16, fin = acce + 16;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 2 * B + 2 * R + 5);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < B; ++s) {
      mbar_init(full0 + 8u * s, 1 + 2 * kGroupWarps);   // the copies; a group of either CTA
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int s = 0; s < R; ++s) {
      mbar_init(rfull0 + 8u * s, 1);
      mbar_init(rempty0 + 8u * s, kGroupWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf + 8u * b, 1);
      mbar_init(acce + 8u * b, 2 * kOutWarps);
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
  Unit o;

  if (warp == 0) {
    // ---------------------------------------------------------------- tokens
    bool ok = !loads_withheld(p.guard), issued = false;
    Ring st(B);
    for (int t = pair; ok && find_unit(p, t, &o); t += npairs) {
      const int t0 = o.t0 + static_cast<int>(rank) * (o.n / 2), boxes = o.n / 2 > p.xrows ? 2 : 1;
      for (int s = o.b0; s < o.b0 + o.nb; ++s) {
        ok = guard_wait(empty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 62);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t fb = full0 + 8u * st.i, at = smem_u32(smem) + (2 * st.i + 1) * stage_bytes - xbox;
          // the even CTA's barrier counts both CTAs' bytes
          if (rank == 0) mbar_expect_tx(fb, static_cast<uint32_t>(4 * boxes * p.xrows) * 128u);
          for (int b = 0; b < boxes; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d_pair(at + h * stage_bytes + static_cast<uint32_t>(b * p.xrows) * 128u, &mX, s * kKB + h * kKS,
                               t0 + b * p.xrows, mapa_shared(fb, 0));
        }
        __syncwarp();
        issued = true;
        st.next();
      }
    }
    if (!ok && issued) {
      // copies in flight, whose barrier may never complete after an abort: they
      // land within microseconds, wait 1 ms
      const unsigned long long c0 = globaltimer();
      while (globaltimer() - c0 < 1000000ull) {
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- blocks of W
    bool ok = !loads_withheld(p.guard);
    int issued = 0;
    Ring rw(R);
    for (int t = pair; ok && find_unit(p, t, &o); t += npairs) {
      const int f0 = o.ft * kTileF + static_cast<int>(rank) * 128;
      for (int s = o.b0; s < o.b0 + o.nb; ++s) {
        ok = guard_wait(rempty0 + 8u * rw.i, rw.phase ^ 1u, ctl, p.guard, 61);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t fb = rfull0 + 8u * rw.i, at = smem_u32(raw) + rw.i * kRawBytes;
          mbar_expect_tx(fb, kRawBytes);
          // coordinates in bytes along a row of W
          if (TRANS) tma_load_3d(at, &mW, f0 / 2, s * kKB, o.e, fb);
          else tma_load_3d(at, &mW, s * (kKB / 2), f0, o.e, fb);
        }
        __syncwarp();
        ++issued;
        rw.next();
      }
    }
    if (!ok)
      for (int k = 0; k < R && k < issued; ++k) {   // copies in flight
        if (--rw.i < 0) {
          rw.i = R - 1;
          rw.phase ^= 1u;
        }
        wait_drain_ns(rfull0 + 8u * rw.i, rw.phase, kWaitNs);
      }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------------- MMA issuer
      // (a commit arrives on the barrier of this CTA and on the peer's)
      bool ok = true;
      Ring st(B);
      Acc acc(TRANS, p.ntok);
      for (int t = pair; ok && find_unit(p, t, &o); t += npairs, acc.next()) {
        ok = guard_wait(acce + 8u * acc.i, acc.phase ^ 1u, ctl, p.guard, 63);
        const uint32_t d = tmem + acc.column(), id = idesc_bf16_pair(o.n) | (TRANS ? 1u << 15 : 0u);
        for (int s = 0; s < o.nb; ++s) {
          ok = ok && guard_wait(full0 + 8u * st.i, st.phase, ctl, p.guard, 64);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = 2 * st.i + h;
              const uint32_t at = smem_u32(smem) + i * stage_bytes;
              const uint64_t b = sdesc<32>(at + stage_bytes - xbox);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t more = s != 0 || h != 0 || k != 0 ? 1u : 0u;
                // 16 k: 32 bytes along a K-major row, 16 rows of an M-major panel, 8 columns
                if (TRANS) mma_bf16_ss_pair(d, sdesc_mmajor(at) + 128u * k, b + 2u * k, id, more);
                else mma_bf16_ts_pair(d, tmem + kACol + 32u * i + 8u * k, b + 2u * k, id, more);
              }
            }
            mma_commit_both(empty0 + 8u * st.i);
            if (s + 1 == o.nb) {
              mma_commit_both(accf + 8u * acc.i);
            }
          }
          __syncwarp();
          st.next();
        }
      }
      if (elect_one()) {
        mma_commit_pair(fin);
        wait_drain_ns(fin, 0, kWaitNs);
      }
      __syncwarp();
    }
  } else if (warp < kOut0<TRANS>) {
    // ---------------------------------------------------------------- conversion
    // a thread has a row of the block: of x W^T a feature, of dy W a k
    const int g = (warp - kConv0) / kGroupWarps, i = (warp & 3) * 32 + lane;
    const int G = p.in / kQ4Group;
    const bool words = G % 4 == 0;                 // the scales of a block's row are a word
    const uint32_t to = TRANS ? smem_u32(smem) + (i >> 6) * stage_bytes + (i & 63) * 128u
                              : tmem + kACol + (static_cast<uint32_t>(warp & 3) * 32u << 16);
    const uint32_t from = smem_u32(raw) + static_cast<uint32_t>(i) * 64u, swz = static_cast<uint32_t>((i >> 1) & 3) * 16u;
    bool ok = true;
    int u = g;                                     // block, counted over all tiles
    const int blk = g;                             // its slot, in the ring of W `slot`
    int slot = g;
    uint32_t rphase = 0, ephase = 1;
    const uint32_t full = mapa_shared(full0 + 8u * blk, 0);
    for (int t = pair, u0 = 0; ok && find_unit(p, t, &o); t += npairs, u0 += o.nb) {
      const int f0 = o.ft * kTileF + static_cast<int>(rank) * 128;
      // scales of this thread's row of block q of the unit
      const int64_t row0 = static_cast<int64_t>(o.e) * p.out + i + (TRANS ? o.b0 * kKB : f0);
      auto scales = [&](int q) -> uint32_t {
        const int k = (o.b0 + q) * kKB, f = i + (TRANS ? k : f0), c = (TRANS ? f0 : k) / kQ4Group;
        if (q >= o.nb || f >= p.out || c >= G) return 0x7f7f7f7fu;
        const uint8_t *at = p.scale + (row0 + (TRANS ? q * kKB : 0)) * G + c;
        if (words) return load_now(reinterpret_cast<const uint32_t *>(at));
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= (c + j < G ? load_now(at + j) : 127u) << (8 * j);
        return w;
      };
      const int q0 = u - u0;                       // this group's first block of the unit
      uint32_t sc[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) sc[k] = scales(q0 + k * NG);
      for (int qa = q0; qa < o.nb && ok; qa += kAhead * NG) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int q = qa + k * NG;
          if (q >= o.nb || !ok) break;
          const uint32_t b = sc[k];
          sc[k] = scales(q + kAhead * NG);
          ok = guard_wait(rfull0 + 8u * slot, rphase, ctl, p.guard, 66);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t at = from + slot * kRawBytes;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            const uint4 w0 = lds128(at + ((h * 32u) ^ swz)), w1 = lds128(at + ((h * 32u + 16u) ^ swz));
            q4_bf16x32(w0, b >> (16 * h) & 255u, v);
            q4_bf16x32(w1, b >> (16 * h + 8) & 255u, v + 16);
            if (h == 0) {
              ok = guard_wait(empty0 + 8u * blk, ephase, ctl, p.guard, 67);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
            }
            if (TRANS) {
              const uint32_t dst = to + 2 * blk * stage_bytes + h * kPanel;
#pragma unroll
              for (int c = 0; c < 8; ++c) sts128(dst + static_cast<uint32_t>((c ^ (i & 7)) * 16), v + 4 * c);
            } else {
              tmem_st32(to + 32u * (2 * blk + h), v);
            }
          }
          if (!ok) break;
          // W's slot only now, behind stores that take what was loaded from it: an arrival
          // right after the loads does not wait for them, and the next copy overtook some
          __syncwarp();
          if (lane == 0) mbar_arrive(rempty0 + 8u * slot);
          if (TRANS) {
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(full);
          } else {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair_relaxed(full);
          }
          u += NG;
          ephase ^= 1u;
          if (R > NG && slot < NG) {
            slot += NG;
          } else {
            slot = g;
            rphase ^= 1u;
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- result
    const int e = warp - kOut0<TRANS>;
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    bool ok = true;
    Acc acc(TRANS, p.ntok);
    for (int t = pair; ok && find_unit(p, t, &o); t += npairs, acc.next()) {
      ok = guard_wait(accf + 8u * acc.i, acc.phase, ctl, p.guard, 68);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const int half = o.n / 2, c0 = (e >> 2) * half;   // tokens of this warp
      const uint32_t lane_addr = tmem + ((quad * 32u) << 16) + static_cast<uint32_t>(c0);
      const int f = o.ft * kTileF + static_cast<int>(rank) * 128 + static_cast<int>(quad) * 32 + lane;
      const int t0 = o.t0 + c0, live = min(o.t1 - t0, half);
      const int64_t ld = p.nfeat;
      if (p.parts > 1) {
        float *to = p.partial + (static_cast<int64_t>(o.part) * p.T + t0) * ld + f;
#pragma unroll 1
        for (int c = 0; c < half; c += 16, to += 16 * ld) {
          float w[16];
          tmem_ld<16>(lane_addr + acc.column() + static_cast<uint32_t>(c), w);
          if (f < p.nfeat)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c + i < live) to[i * ld] = w[i];
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair_relaxed(mapa_shared(acce + 8u * acc.i, 0));
        continue;
      }
      // in two goes, for which there are registers
      const int quarter = half / 2;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint32_t v[kTileT / 8];                    // two tokens a register
#pragma unroll
        for (int c = 0; c < kTileT / 4; c += 8)
          if (c < quarter) {
            float w[8];
            tmem_ld<8>(lane_addr + acc.column() + static_cast<uint32_t>(h * quarter + c), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[c / 2 + i] = pack_bf16x2(w[2 * i], w[2 * i + 1]);
          }
        if (h == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_pair_relaxed(mapa_shared(acce + 8u * acc.i, 0));
        }
        if (f < p.nfeat) {
          uint16_t *y = reinterpret_cast<uint16_t *>(p.y) + static_cast<int64_t>(t0 + h * quarter) * ld + f;
          const int n = min(live - h * quarter, quarter);
#pragma unroll
          for (int i = 0; i < kTileT / 8; ++i, y += 2 * ld) {
            if (2 * i < n) y[0] = static_cast<uint16_t>(v[i]);
            if (2 * i + 1 < n) y[ld] = static_cast<uint16_t>(v[i] >> 16);
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();   // the cluster's barrier takes whole warps
  // the even CTA's MMAs, which read this CTA's shared memory and write its
  // tensor memory, are complete, and both CTAs' results are out
  cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

// the sum of a tile's parts in their order, rounded once; rows that no expert has are
// left as they are
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
q4_join_kernel(const float4 *__restrict__ parts, int n, int T, int quads, const int *__restrict__ offsets, int experts,
               uint2 *__restrict__ y) {
  pdl_trigger();
  pdl_wait();
  const int a = offsets ? min(max(offsets[0], 0), T) : 0, b = offsets ? min(max(offsets[experts], a), T) : T;
  const int64_t all = static_cast<int64_t>(T) * quads, end = static_cast<int64_t>(b) * quads;
  for (int64_t i = static_cast<int64_t>(a) * quads + blockIdx.x * kJoinThreads + threadIdx.x; i < end;
       i += static_cast<int64_t>(gridDim.x) * kJoinThreads) {
    float4 s = parts[i];
    for (int k = 1; k < n; ++k) {
      const float4 v = parts[k * all + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    y[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Tokens per tile and parts of k: the least time, in us, of the waves of units over
// the pairs that a GB300 holds, a fixed number so that the workspace is the same
// everywhere.  A block of k takes the conversion's time, above 192 tokens the MMAs'
// (or, of dy W, the copies' with half of the slots); parts cost their way through memory
// and a launch.
// One weight: within 2% of the best of all widths and parts but for the smallest (129 x
// 8192 x 8192: 160 tokens in 2 parts 22.4 us, in 3 29.4, in 4 25.7; 129 x 1024 x 1024 8.2,
// 7.1).  Experts: the host does not know their loads, which are taken as squares of
// even numbers, up to three times the mean; so an expert has a (k + 1)th tile in 1 -
// sqrt(k n / most) of the cases, and a last wave behind others counts half.  Over four
// draws of such loads, us by 256 tokens and by 192: 4096 at 32 of 2048 x 4096 72-74,
// 78-80; 1001 at 8 of 1040 x 2080 16.1, 14.1; dy W 13-19, 17; 8192 at 64 of 1024 x 2048
// 47-49, 49-50; dy W 58-59, 62.  Loads of other shapes, by 256 tokens: 4096 at 32 evenly 63, as
// a router without preferences draws them 65, one expert with half of the tokens 79, falling
// as 1 / rank 75; dy W 85, 86, 104, 97.
struct Plan {
  int ntok, parts;
};
Plan plan(bool trans, int64_t T, int64_t nfeat, int64_t kdim, int64_t experts) {
  constexpr int kPairs = 76;
  const int64_t groups = experts < T ? experts : T, ftiles = dora::ceil_div(nfeat, kTileF), blocks = dora::ceil_div(kdim, kKB);
  Plan best = {kTileT, 1};
  double least = 0;
  for (int n = 32; n <= kTileT; n += 32) {
    double tiles = static_cast<double>(ftiles * dora::ceil_div(T, n));
    if (experts > 1) {
      const double most = 3.0 * static_cast<double>(T) / static_cast<double>(groups * n);
      double own = 0;
      if (most > 6) own = most / 3 + 0.5;          // what the sum tends to (6: 2.58)
      else
        for (int k = 0; k < most; ++k) own += 1 - std::sqrt(k / most);
      tiles = own * static_cast<double>(groups * ftiles);
    }
    const bool wide = n > 192;
    const double block = experts > 1 ? (trans ? (wide ? 0.59 : 0.57) : (wide ? 0.52 : 0.5))
                                     : (trans ? (wide ? 0.64 : 0.57) : (wide ? 0.56 : 0.5)) + 0.0001 * n;
    for (int parts = 1; parts <= 8; ++parts) {
      if (parts > 1 && (blocks < 4 * parts || tiles * (parts - 1) > 4 * kPairs)) break;   // enough without
      double waves = std::ceil(tiles * parts / kPairs);
      if (experts > 1 && waves > 1) waves = (waves + tiles * parts / kPairs) / 2;
      double cost = waves * (static_cast<double>(dora::ceil_div(blocks, parts)) * block + 1.5);
      if (parts > 1) cost += 2.5 + static_cast<double>(parts) * T * nfeat * 8 / 5e6;
      if (least == 0 || cost < least) {
        least = cost;
        best = {n, parts};
      }
    }
  }
  return best;
}
size_t parts_bytes(const Plan &pl, int64_t T, int64_t nfeat) {
  return pl.parts > 1 ? static_cast<size_t>(pl.parts) * T * nfeat * 4 : 0;
}

template <bool TRANS> constexpr size_t pair_smem(int ntok) {
  return 1024 + raw_slots<TRANS>(ntok) * kRawBytes + 512 + kStages<TRANS> * static_cast<size_t>(stage_size<TRANS>(ntok));
}
template <bool TRANS> constexpr bool fits() {
  for (int n = 32; n <= kTileT; n += 32)
    if (pair_smem<TRANS>(n) > kSmemMax || 8 * (kStages<TRANS> + 2 * raw_slots<TRANS>(n) + 5) + sizeof(SharedCtl) > 512) return false;
  return true;
}
static_assert(fits<false>() && fits<true>(), "rings, barriers and control words");

template <bool TRANS>
void pair_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int ntok, int64_t pairs, cudaStream_t cs) {
  *cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->gridDim = dim3(2 * static_cast<unsigned>(pairs));
  cfg->blockDim = dim3(kThreadsMm<TRANS>);
  cfg->dynamicSmemBytes = pair_smem<TRANS>(ntok);
  cfg->stream = cs;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// pairs that are resident at once; 0 where the device has no clusters of two
int resident_pairs(int device, int sms) {
  static std::mutex mu;
  static int known[64] = {};   // pairs + 1
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (known[device] == 0) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    pair_config<false>(&cfg, attr, kTileT, sms / 2, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, q4_pair_kernel<false, raw_slots<false>(kTileT)>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[device] = n + 1;
  }
  return known[device] - 1;
}

dora_status mm_init(int device, Q4Params *p) {
  static const void *const kernels[] = {(const void *)q4_pair_kernel<false, 8>, (const void *)q4_pair_kernel<true, 3>,
                                        (const void *)q4_pair_kernel<true, 6>};
  return tc_init(device, &p->guard, kernels, sizeof(kernels) / sizeof(kernels[0]));
}

template <bool TRANS>
dora_status run_matmul(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T, int64_t out,
                       int64_t in, int64_t experts, void *y, void *workspace, dora_stream_t stream) {
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  Q4Params p = {};
  st = mm_init(device, &p);
  if (st != DORA_OK) return st;
  p.T = static_cast<int>(T);
  p.out = static_cast<int>(out);
  p.in = static_cast<int>(in);
  p.nfeat = static_cast<int>(TRANS ? in : out);
  p.kdim = static_cast<int>(TRANS ? out : in);
  p.experts = static_cast<int>(experts);
  p.offsets = offsets;
  p.scale = static_cast<const uint8_t *>(wscale);
  p.y = static_cast<__nv_bfloat16 *>(y);
  const int pairs = resident_pairs(device, info.sms);
  if (pairs == 0) return DORA_ERR_CUDA;
  p.ftiles = static_cast<int>(dora::ceil_div(p.nfeat, kTileF));
  const Plan pl = plan(TRANS, T, p.nfeat, p.kdim, experts);
  p.ntok = pl.ntok;
  p.xrows = p.ntok / 2 <= 64 ? p.ntok / 2 : p.ntok / 4;
  p.parts = pl.parts;
  p.partial = static_cast<float *>(workspace);
  // an expert of n tokens has (n - 1) / ntok + 1
  const int64_t groups = experts < T ? experts : T;
  const int64_t tiles = p.ftiles * (offsets ? (T - groups) / p.ntok + groups : dora::ceil_div(T, p.ntok));
  if (tiles * p.parts > kMaxDim) return DORA_ERR_SHAPE;
  p.tiles = static_cast<int>(tiles);
  const int64_t units = tiles * p.parts;
  CUtensorMap mW, mX;
  if (!map_w(&mW, wq, experts, out, in) || !make_map(&mX, x, true, T, p.kdim, p.kdim, p.xrows, 128)) return DORA_ERR_CUDA;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  pair_config<TRANS>(&cfg, attr, p.ntok, units < pairs ? units : pairs, cs);
  constexpr int kMost = raw_slots<TRANS>(kTileT), kFew = raw_slots<TRANS>(32);
  if ((raw_slots<TRANS>(p.ntok) == kFew ? cudaLaunchKernelEx(&cfg, q4_pair_kernel<TRANS, kFew>, mW, mX, p)
                                        : cudaLaunchKernelEx(&cfg, q4_pair_kernel<TRANS, kMost>, mW, mX, p)) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  if (p.parts == 1) return DORA_OK;
  const int quads = p.nfeat / 4;
  const int64_t all = dora::ceil_div(T * quads, kJoinThreads), most = 8 * static_cast<int64_t>(info.sms);
  cudaLaunchConfig_t jc = {};
  jc.gridDim = dim3(static_cast<unsigned>(all < most ? all : most));
  jc.blockDim = dim3(kJoinThreads);
  jc.stream = cs;
  jc.attrs = attr + 1;   // a programmatic dependent launch
  jc.numAttrs = 1;
  if (cudaLaunchKernelEx(&jc, q4_join_kernel, static_cast<const float4 *>(workspace), p.parts, p.T, quads, offsets, p.experts,
                         static_cast<uint2 *>(y)) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

dora_status check(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T, int64_t out,
                  int64_t in, int64_t experts, const void *y) {
  if (bad_size(T, 0) || bad_size(out, 0) || bad_size(in, 0) || experts < 1 || experts > kMaxExperts) return DORA_ERR_SHAPE;
  if (!offsets && experts != 1) return DORA_ERR_NULL;
  if (in % kQ4Group != 0) return DORA_ERR_SHAPE;
  if (T == 0 || out == 0 || in == 0) return DORA_OK;
  if (!x || !wq || !wscale || !y) return DORA_ERR_NULL;
  // TMA: 16-byte aligned bases and row strides
  if (out % 16 != 0) return DORA_ERR_ALIGN;
  if (!dora::aligned(x, 16) || !dora::aligned(wq, 16) || !dora::aligned(y, 16) || !dora::aligned(wscale, 16) ||
      !dora::aligned(offsets, 4))
    return DORA_ERR_ALIGN;
  return DORA_OK;
}

}  // namespace

static bool bad_call(int64_t T, int64_t out, int64_t in, int64_t experts) {
  return bad_size(T, 1) || bad_size(out, 1) || bad_size(in, 1) || experts < 1 || experts > kMaxExperts;
}

extern "C" size_t dora_matmul_q4_workspace(int64_t T, int64_t out, int64_t in, int64_t experts) {
  if (bad_call(T, out, in, experts)) return 0;
  if (dora::q4_few(T, in, experts)) return dora::q4_few_workspace(T, in, experts);
  return parts_bytes(plan(false, T, out, in, experts), T, out);
}
extern "C" size_t dora_matmul_q4_t_workspace(int64_t T, int64_t out, int64_t in, int64_t experts) {
  return bad_call(T, out, in, experts) ? 0 : parts_bytes(plan(true, T, in, out, experts), T, in);
}
static bool short_of(size_t need, const void *workspace, size_t bytes) {
  return need > 0 && (!workspace || !dora::aligned(workspace, 256) || bytes < need);
}

extern "C" dora_status dora_matmul_q4(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T,
                                      int64_t out, int64_t in, int64_t experts, void *y, void *workspace,
                                      size_t workspace_bytes, dora_stream_t stream) {
  if (in < 1) return DORA_ERR_SHAPE;
  const dora_status st = check(x, offsets, wq, wscale, T, out, in, experts, y);
  if (st != DORA_OK || T == 0 || out == 0) return st;
  if (short_of(dora_matmul_q4_workspace(T, out, in, experts), workspace, workspace_bytes)) return DORA_ERR_WORKSPACE;
  if (dora::q4_few(T, in, experts))                 // few tokens a weight, W read as it is
    return dora::matmul_q4_few(x, offsets, wq, wscale, T, out, in, experts, y, workspace,
                               reinterpret_cast<cudaStream_t>(stream));
  return run_matmul<false>(x, offsets, wq, wscale, T, out, in, experts, y, workspace, stream);
}

extern "C" dora_status dora_matmul_q4_t(const void *dy, const int32_t *offsets, const void *wq, const void *wscale,
                                        int64_t T, int64_t out, int64_t in, int64_t experts, void *dx, void *workspace,
                                        size_t workspace_bytes, dora_stream_t stream) {
  if (out < 1) return DORA_ERR_SHAPE;
  const dora_status st = check(dy, offsets, wq, wscale, T, out, in, experts, dx);
  if (st != DORA_OK || T == 0 || in == 0) return st;
  if (short_of(dora_matmul_q4_t_workspace(T, out, in, experts), workspace, workspace_bytes)) return DORA_ERR_WORKSPACE;
  return run_matmul<true>(dy, offsets, wq, wscale, T, out, in, experts, dx, workspace, stream);
}
