// The gradient of A from the 8-bit x (see q8.cuh for the form) for GB300
// (sm_103a): dora_lora_grad_q8, dA = dxa^T x with dxa [T, r] in bf16 and x
// [T, in] in 8 bits.
//
// Every value of an 8-bit form is exact in bf16, so the product runs as
// kind::f16 bf16 MMAs with exact products: 128 features of x on the M side, up
// to 192 columns of dxa on the N side, the tokens as k.  dxa is read as it
// lies, token by token (N-major).  x passes through registers once: transposed
// loads from shared memory (ldmatrix) give a thread two features at two tokens
// a register, a few bit operations and one product per pair turn them into
// bf16 words of one feature each, and tcgen05.st puts them into tensor memory,
// where the MMA takes its M side from.  Shared memory moves each byte of x
// once in and once out; as a bf16 operand in shared memory (the form measured
// first) it moved six times that and was the limit.
//
// The tensor core's fp32 sum rounds toward zero, so its error grows with the
// length of a chain of MMAs.  A window of 512 tokens is one chain (32 MMAs of
// k = 16); the windows are added up in registers with ordinary rounding.
//
// Work: a tile of the result is 128 features x N columns of r; its stages of
// 128 tokens are units, and each CTA (one or two an SM) takes an equal run of
// units over all tiles, in windows of up to four.  (Runs of whole windows left up
// to a sixth of the CTAs idle at the end: 6% more time at r = 16.)  A CTA that
// has a whole tile writes dA; otherwise it writes its part to the workspace and
// grad_join_kernel adds the parts of a tile in order (bitwise reproducible).
//   warp 0      x by TMA: 128 tokens x 128 features a stage (16 KB), and the
//               stage's 128 scales as bf16 factors in shared memory
//   warp 1      tensor memory (two window accumulators, a ring of M operands),
//               MMA issue
//   warps 2-9   bytes -> bf16, two groups on alternate stages, a lane quadrant a
//               warp; window w - 1 out of tensor memory while window w runs,
//               half of the columns a warp
//   warp 10     dxa by TMA: 128 tokens x 64 columns a box (16 KB)
// What bounds it: the work is 2 T in r bf16 operations and T in bytes of x, and
// it reaches about half of either rate, as the conversion warps' chains of
// instructions and the hand-overs set the time of a stage.  15360 x 8192, us, and
// what reading x or the products (at 1886 TFLOP/s) would take: r = 16 29 (19, x),
// r = 128 43 (20, x), r = 384 90 (51, products), r = 768 166 (103).  With every
// operand in L2 the first two are 28 and 41: it is not the memory.  At r = 384
// (8192 x 8192) the tensor pipe is active in 45% of the cycles, the issue slots in 44%.
// A hand-over through an mbarrier was measured at 230 cycles, and four of them
// and a load from memory lie on the way of a stage, so each buffer is a ring of
// its own that is freed as early as it can be: x once it is in registers, dxa
// and the M operand when their MMAs are done.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q8.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kTok = 128;                        // tokens per stage
// Tokens per window.  Longer ones are read out and joined less often, but the
// sum's error grows with them (parts of dA's norm; an fp32 product's is 1.8e-7 at
// the first size, 1.1e-7 at the last).
// 256, 512, 1024, in us and 1e-7: 15360 x 8192, r = 384 98 1.4, 90 1.6, 88 2.9;
// r = 16 30.4 1.1, 29.2 1.5, 29.1 2.8; 8192 x 4096, r = 64 17.2 1.0, 16.6 1.4, 16.4
// 2.5
constexpr int kWin = 512;
constexpr int kWorkers = 8;                      // conversion warps, in two groups that take alternate stages
constexpr int kThreadsG = 96 + 32 * kWorkers;
// a box's 128-byte rows are fetched alone: their neighbours belong to CTAs that
// are at other tokens (15360 x 8192, us: r = 16 29.2 against 31.6 with 256 bytes
// at a time, r = 128 43.0 against 46.9)
constexpr CUtensorMapL2promotion kPromote = CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
constexpr unsigned kRawBytes = kTok * 128;       // 16 KB of x
constexpr unsigned kBox = kTok * 128;            // 128 tokens x 64 columns of dxa
constexpr int kMaxR = 1024;
constexpr int kMaxN = 192;                       // columns of a tile: two windows and the M operands fill tensor memory
constexpr int kMaxSMs = 256;                     // workspace bound: any device up to this size
// By the columns of a tile: CTAs per SM; stages of x and of dxa in shared
// memory; M operands (64 columns) in tensor memory beside two windows of the
// tile's columns.  x and the operands in even numbers, as two groups take
// turns, and no fewer of dxa than of operands (the kernel says why).  What limits
// a stage is the length of the roles' instruction chains, so where a CTA needs
// half of an SM's memory, two share it (r = 16 at 15360 x 8192, with runs of
// whole windows: 36.5 us against 42.4 with one CTA and twice the rings; at 64
// columns the registers that two CTAs leave do not hold the sums)
struct Rings {
  int per_sm, x, d, ops;
};
__host__ __device__ constexpr Rings rings_of(int columns) {
  return columns > 128 ? Rings{1, 4, 3, 2} : columns > 64 ? Rings{1, 4, 4, 4} : columns > 32 ? Rings{1, 8, 4, 4} : Rings{2, 4, 2, 2};
}
constexpr int kOpCols = kTok / 2;
// a place in a ring of N
template <int N> struct At {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int by = 1) {
    i += by;
    if (i >= N) {
      i -= N;
      phase ^= 1u;
    }
  }
};
constexpr unsigned kFactorBytes = kTok * 2 + 16; // a stage's factors, and whether one is too large for bf16

struct GradParams {
  int T, in, r;
  int mtiles, ntiles, stages;      // tiles are m fastest; stages (of kTok tokens) per tile
  int ncols;                       // columns of r per tile (N of the MMA)
  int boxes;                       // dxa boxes per stage
  int nsx;
  const uint8_t *scale;
  float *dA;
  float *part;                     // [2 per CTA][columns][128]
  Guard guard;
};

// first unit of CTA i of n
__host__ __device__ __forceinline__ int64_t first_unit(int64_t units, int i, int n) { return units * i / n; }

// a unit's place: stage k of tile (mt, nt).  Counted up, as a 64-bit division
// in every role's loop costs more than a stage of work
struct Place {
  int mt, nt, k;
  __device__ __forceinline__ Place(const GradParams &p, int64_t u) {
    const int tile = static_cast<int>(u / p.stages);
    k = static_cast<int>(u - static_cast<int64_t>(tile) * p.stages);
    nt = tile / p.mtiles;
    mt = tile - nt * p.mtiles;
  }
  // stages of the window that begins here: up to the tile's end and the run's
  __device__ __forceinline__ int window(const GradParams &p, int left) const {
    return min(min(kWin / kTok, p.stages - k), left);
  }
  // n stages on, which do not pass the tile's end
  __device__ __forceinline__ void next(const GradParams &p, int n) {
    k += n;
    if (k == p.stages) {
      k = 0;
      if (++mt == p.mtiles) {
        mt = 0;
        ++nt;
      }
    }
  }
};

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
// Four E4M3 bytes (two features at two tokens) times the tokens' scales as
// bf16 pairs: .x = bytes 0 and 2, .y = bytes 1 and 3.  The exponent and
// mantissa bits of an E4M3 value, four places up in a bf16, are that value
// times 2^-120 (subnormals too: their bits become a bf16 subnormal's), so one
// product with 2^120 scale, with the value's sign, finishes it, exactly.  `up` holds the two tokens'
// factors, which are bf16 as long as the scales are at most 2^7
struct Mags {
  uint32_t even, odd;
};
__device__ __forceinline__ Mags mags4(uint32_t w) { return {(w << 4) & 0x07f007f0u, (w >> 4) & 0x07f007f0u}; }
__device__ __forceinline__ uint2 decode4(uint32_t w, Mags m, uint32_t up) {
  return make_uint2(mul_bf16x2(m.even, ((w << 8) & 0x80008000u) ^ up), mul_bf16x2(m.odd, (w & 0x80008000u) ^ up));
}
// the largest magnitude so far in each half; 0x7f0 is a NaN byte's
__device__ __forceinline__ uint32_t max_mag(uint32_t top, Mags m) { return __vimax3_u16x2(top, m.even, m.odd); }
__device__ __forceinline__ bool has_nan(uint32_t top) { return (top & 0xffffu) == 0x07f0u || (top >> 16) == 0x07f0u; }
constexpr uint32_t kMaxFast = 134;               // the scale byte of 2^7
__device__ __forceinline__ uint32_t factor_of(uint32_t byte) { return (min(byte, kMaxFast) + 120u) << 7; }
// feature of a tile at M row m: a 16 x 16 transposed load gives rows 0-7 the
// even features and rows 8-15 the odd ones
__device__ __forceinline__ int feature_of(int m) { return (m & ~15) | ((m & 7) << 1) | ((m >> 3) & 1); }

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes x 16 columns of tensor memory: registers 0-3 the first 8 columns
// (lane / 4 at columns 2 (lane % 4) and + 1, then the same of lane / 4 + 8)
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// a warp's share of a stage through fp32, for larger scales and for NaN bytes.
// The scales of tokens t0 + 16 g .. + 3 come from memory; out of line, and with
// no arrays of the caller's, so that the common path keeps its registers
__device__ __noinline__ void convert_any(const uint8_t *scale, int nsx, int T, int t0, uint32_t from0, uint32_t from1,
                                         uint32_t to) {
  uint32_t o[2][8];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t raw[4];
    ldmatrix_x4_trans(g ? from1 : from0, raw);
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 16 * g + i;
      s[i] = scale_value(t < T ? __ldg(scale + static_cast<int64_t>(t) * nsx) : 127u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = i / 2, half = i % 2;
      const float2 a = dequant2(raw[i] & 0xffffu, s[2 * half]), b = dequant2(raw[i] >> 16, s[2 * half + 1]);
      o[h][4 * g + half] = pack_bf16x2(a.x, b.x);
      o[h][4 * g + 2 + half] = pack_bf16x2(a.y, b.y);
    }
  }
  tmem_st_16x256b_x2(to, o[0]);
  tmem_st_16x256b_x2(to + (16u << 16), o[1]);
}

// NC: columns of a tile per worker warp (half of the tile's, rounded up)
template <int NC>
__global__ void __launch_bounds__(kThreadsG, rings_of(2 * NC).per_sm)
lora_grad_kernel(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mD, const GradParams p) {
  constexpr int kN = 2 * NC;                             // columns of one window accumulator
  constexpr Rings kR = rings_of(kN);
  constexpr int kUsed = 2 * kN + kOpCols * kR.ops;       // two windows, the M operands
  constexpr int kCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512 / kR.per_sm, "tensor memory");
  // a wait tells a barrier's phase from the one before, not from the one before
  // that, so whoever waits for use c of a slot must know that use c - 1 is over:
  // a group's own earlier stage for x and the operands, the end of an earlier
  // MMA for dxa (which stage c's operand slot was waited for)
  static_assert(kR.x % 2 == 0 && kR.ops % 2 == 0 && kR.d >= kR.ops, "phases");
  // Who waits for a stage's dxa: the MMA warp, or, for wide tiles, one of the
  // warps that hand it the operand.  A wait takes the MMA warp 150 cycles or
  // more, in which it issues nothing, and the others' chains are shorter than a
  // wide tile's MMAs (15360 x 8192, us, MMA warp / other: r = 768 174 / 166, r = 384
  // 92.8 / 89.7, r = 192 54.1 / 51.8; r = 128 43.0 / 43.2, r = 64 39.1 / 40.1, r = 16
  // 29.2 / 30.1)
  constexpr bool kRelay = kN > 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t d_stage = p.boxes * kBox;
  const uint32_t x_at = smem_u32(smem), d_at = x_at + kR.x * kRawBytes;
  uint8_t *factors = smem + kR.x * kRawBytes + kR.d * d_stage;
  uint64_t *bars = reinterpret_cast<uint64_t *>(factors + kR.x * kFactorBytes);
  // barriers: x loaded and free, dxa loaded and free, M operand written and
  // consumed, window done[2] and read[2], the end
  const uint32_t xfull = smem_u32(bars), xfree = xfull + 8u * kR.x, dfull = xfree + 8u * kR.x, dfree = dfull + 8u * kR.d,
                 conv0 = dfree + 8u * kR.d, used0 = conv0 + 8u * kR.ops, done0 = used0 + 8u * kR.ops, read0 = done0 + 16,
                 fin = read0 + 16;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 2 * (kR.x + kR.d + kR.ops) + 5);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kR.x; ++s) {
      mbar_init(xfull + 8u * s, 2);               // the copy (and its bytes), the factors
      mbar_init(xfree + 8u * s, kWorkers / 2);
    }
    for (int s = 0; s < kR.d; ++s) {
      mbar_init(dfull + 8u * s, 1);
      mbar_init(dfree + 8u * s, 1);
    }
    for (int s = 0; s < kR.ops; ++s) {
      mbar_init(conv0 + 8u * s, kWorkers / 2);
      mbar_init(used0 + 8u * s, 1);
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
  pdl_trigger();    // grad_join_kernel's launch overlaps this kernel; it waits for its end
  pdl_wait();       // the set-up above overlaps the end of the launch before
  const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.stages;
  const int64_t u0 = first_unit(units, blockIdx.x, gridDim.x);
  int left = static_cast<int>(first_unit(units, blockIdx.x + 1, gridDim.x) - u0);   // of the run, in each role
  Place at(p, u0);

  // a producer that gives up leaves copies in flight, whose barriers may also
  // wait for others that have left: they land within microseconds, wait 1 ms
  auto settle_copies = [] {
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- x
    // the scales, four tokens a lane, are requested kAhead stages before they
    // are needed (one byte per token and tile: a sector each, often from memory)
    constexpr int kAhead = 3;
    uint32_t ring[kAhead][kTok / 32];
    Place from = at;        // of the stage whose scales are requested next
    int from_left = left;
    auto fetch = [&](uint32_t (&dst)[kTok / 32]) {
      const uint8_t *sp = p.scale + from.mt;
#pragma unroll
      for (int i = 0; i < kTok / 32; ++i) {
        const int t = from.k * kTok + 32 * i + lane;
        dst[i] = 127u;
        if (from_left > 0 && t < p.T)
          // volatile: not moved down to its use by the compiler
          asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(dst[i]) : "l"(sp + static_cast<int64_t>(t) * p.nsx));
      }
      --from_left;
      from.next(p, 1);
    };
#pragma unroll
    for (int a = 0; a < kAhead; ++a) fetch(ring[a]);
    bool ok = !loads_withheld(p.guard);
    bool issued = false;
    At<kR.x> x;
    while (ok && left > 0) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (!ok || left == 0) break;
        ok = guard_wait(xfree + 8u * x.i, x.phase ^ 1u, ctl, p.guard, 31);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t fb = xfull + 8u * x.i;
        if (elect_one()) {
          mbar_expect_tx(fb, kRawBytes);
          tma_load_2d(x_at + x.i * kRawBytes, &mX, at.mt * kTcM, at.k * kTok, fb);
        }
        issued = true;
        uint16_t *dst = reinterpret_cast<uint16_t *>(factors + x.i * kFactorBytes);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kTok / 32; ++i) {
          dst[32 * i + lane] = static_cast<uint16_t>(factor_of(ring[a][i]));
          top = max(top, ring[a][i]);
        }
        const bool large = __any_sync(0xffffffffu, top > kMaxFast);
        if (lane == 0) *reinterpret_cast<uint32_t *>(dst + kTok) = large ? 1u : 0u;
        __syncwarp();
        if (lane == 0) mbar_arrive(fb);
        fetch(ring[a]);
        x.next();
        --left;
        at.next(p, 1);
      }
    }
    if (!ok && issued) settle_copies();
  } else if (warp == 2 + kWorkers) {
    // ---------------------------------------------------------------- dxa
    bool ok = !loads_withheld(p.guard);
    bool issued = false;
    At<kR.d> d;
    for (; left > 0 && ok; --left, at.next(p, 1)) {
      ok = guard_wait(dfree + 8u * d.i, d.phase ^ 1u, ctl, p.guard, 39);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t fb = dfull + 8u * d.i, to = d_at + d.i * d_stage;
      if (elect_one()) {
        mbar_expect_tx(fb, d_stage);
#pragma unroll
        for (int b = 0; b < (kN + 63) / 64; ++b)
          if (b < p.boxes) tma_load_2d(to + b * kBox, &mD, at.nt * p.ncols + 64 * b, at.k * kTok, fb);
      }
      __syncwarp();
      issued = true;
      d.next();
    }
    if (!ok && issued) settle_copies();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // bf16, fp32 accumulator, the N side N-major
    const uint32_t idesc = idesc_bf16(p.ncols) | (1u << 16);
    bool ok = true;
    At<kR.d> ds;
    At<kR.ops> op;
    At<2> win;
    const uint64_t b0 = mn_desc(d_at, kBox);
    while (left > 0 && ok) {
      const int ns = at.window(p, left);
      const uint32_t d = tmem + static_cast<uint32_t>(win.i * kN);
      ok = guard_wait(read0 + 8u * win.i, win.phase ^ 1u, ctl, p.guard, 32);
      uint32_t acc = 0;
      for (int k = 0; k < ns; ++k) {
        if (!kRelay) ok = ok && guard_wait(dfull + 8u * ds.i, ds.phase, ctl, p.guard, 36);
        ok = ok && guard_wait(conv0 + 8u * op.i, op.phase, ctl, p.guard, 33);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = b0 + (ds.i * d_stage >> 4);
        const uint32_t a = tmem + 2 * kN + static_cast<uint32_t>(kOpCols * op.i);
        if (elect_one()) {
          // 16 tokens at a time: 8 columns of the M operand, 16 rows of 128 bytes
          mma_bf16_ta(d, a, b, idesc, acc);
#pragma unroll
          for (int j = 1; j < kTok / 16; ++j) mma_bf16_ta(d, a + 8u * j, b + 128u * j, idesc, 1u);
          mma_commit(used0 + 8u * op.i);
          mma_commit(dfree + 8u * ds.i);
          if (k + 1 == ns) mma_commit(done0 + 8u * win.i);
        }
        __syncwarp();
        acc = 1;
        ds.next();
        op.next();
      }
      left -= ns;
      at.next(p, ns);
      win.next();
    }
    if (elect_one()) {
      mma_commit(fin);
      wait_drain_ns(fin, 0, kWaitNs);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- workers
    const int wk = warp - 2;
    const uint32_t quad = static_cast<uint32_t>(warp & 3);
    const int grp = wk >> 2;                             // which stages, and which half of the columns
    const uint32_t lane_addr = tmem + ((quad * 32u) << 16) + static_cast<uint32_t>(grp * NC);
    constexpr int C = NC % 32 == 0 ? 32 : NC % 16 == 0 ? 16 : 8;
    float sum[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[j] = 0.0f;
    // this lane's row of a transposed load: lanes 0-7 and 8-15 give the rows of
    // tokens 4 i, 4 i + 1 and 4 i + 2, 4 i + 3 (i < 4) of 16 features, lanes
    // 16-31 the same of the next 16 features
    const int tok = 4 * ((lane & 7) >> 1) + (lane & 1) + 2 * ((lane >> 3) & 1);
    const int chunk = 2 * static_cast<int>(quad) + (lane >> 4);
    const uint32_t from_off = static_cast<uint32_t>(tok * 128 + ((chunk ^ (tok & 7)) << 4));
    bool ok = true;
    int flushed = 0;         // windows of this CTA that are in `sum` or written out
    At<2> win;               // the next of them
    auto flush = [&]() {
      const bool got = guard_wait(done0 + 8u * win.i, win.phase, ctl, p.guard, 34);
      if (!__all_sync(0xffffffffu, got)) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NC; c += C) {
        float v[C];
        tmem_ld<C>(lane_addr + static_cast<uint32_t>(win.i * kN + c), v);
#pragma unroll
        for (int j = 0; j < C; ++j) sum[c + j] += v[j];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(read0 + 8u * win.i);
      win.next();
      ++flushed;
      return true;
    };
    // the stage this warp is at: stage k of the ns of the CTA's window wi, which
    // begins at `at`
    int wi = 0, k = grp, ns = at.window(p, left);
    bool from_start = at.k == 0;   // the run's part of this tile begins at the tile's start
    // the end of that part: its remaining windows, up to window wi, and the sum
    // to dA or to the workspace
    auto finish = [&](bool at_end) {
      while (flushed <= wi)
        if (!flush()) return false;
      const int m = static_cast<int>(quad) * 32 + lane;
      if (from_start && at_end) {
        const int f = at.mt * kTcM + feature_of(m);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const int n = grp * NC + j, col = at.nt * p.ncols + n;
          if (n < p.ncols && col < p.r && f < p.in) p.dA[static_cast<int64_t>(col) * p.in + f] = sum[j];
        }
      } else {
        // slot 0: the run began inside the tile; slot 1: at its start
        float *dst = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (from_start ? 1 : 0)) * p.ncols * kTcM + m;
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (grp * NC + j < p.ncols) dst[(grp * NC + j) * kTcM] = sum[j];
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) sum[j] = 0.0f;
      from_start = true;
      return true;
    };
    // to the window that holds stage k (counted from the start of window wi)
    auto settle = [&]() {
      while (k >= ns && left > 0) {
        const bool at_end = at.k + ns == p.stages;
        if (at_end || ns == left) {
          if (!finish(at_end)) return false;
        }
        k -= ns;
        left -= ns;
        at.next(p, ns);
        ++wi;
        ns = at.window(p, left);
      }
      return true;
    };
    At<kR.x> x;
    At<kR.ops> op;
    At<kR.d> ds;
    x.next(grp);
    op.next(grp);
    ds.next(grp);
    for (ok = settle(); ok && left > 0; ok = settle()) {
      bool got = guard_wait(xfull + 8u * x.i, x.phase, ctl, p.guard, 35);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      const uint32_t from = x_at + x.i * kRawBytes + from_off;
      const uint8_t *fa = factors + x.i * kFactorBytes;
      const bool large = *reinterpret_cast<const uint32_t *>(fa + 2 * kTok) != 0;
      const uint32_t to = tmem + ((quad * 32u) << 16) + 2 * kN + static_cast<uint32_t>(kOpCols * op.i);
      // 32 tokens at a time, as 16 x 16 blocks, the next ones' loads before
      // these ones' arithmetic.  NaN bytes are looked for once, at the end
      struct Block {
        uint32_t raw[2][4];
        uint2 up[2];
      } blk[2];
      auto load_block = [&](int g2, Block &b) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          ldmatrix_x4_trans(from + 2048u * (2 * g2 + g), b.raw[g]);
          b.up[g] = *reinterpret_cast<const uint2 *>(fa + 2 * (16 * (2 * g2 + g) + 4 * (lane & 3)));
        }
      };
      uint32_t top = 0;
      load_block(0, blk[0]);
#pragma unroll
      for (int g2 = 0; g2 < kTok / 32; ++g2) {
        if (g2 + 1 < kTok / 32) load_block(g2 + 1, blk[(g2 + 1) % 2]);
        const Block &b = blk[g2 % 2];
        uint32_t o[2][8];              // o[h]: the 16 columns of feature block h
#pragma unroll
        for (int g = 0; g < 2; ++g) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int h = i / 2, half = i % 2;
            const Mags m = mags4(b.raw[g][i]);
            top = max_mag(top, m);
            const uint2 d = decode4(b.raw[g][i], m, half ? b.up[g].y : b.up[g].x);
            o[h][4 * g + half] = d.x;
            o[h][4 * g + 2 + half] = d.y;
          }
        }
        if (g2 == 0) {
          got = guard_wait(used0 + 8u * op.i, op.phase ^ 1u, ctl, p.guard, 38);
          ok = __all_sync(0xffffffffu, got);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st_16x256b_x2(to + 16u * g2, o[0]);
        tmem_st_16x256b_x2(to + 16u * g2 + (16u << 16), o[1]);
      }
      if (!ok) break;
      if (__any_sync(0xffffffffu, large || has_nan(top))) [[unlikely]] {
        tmem_wait_st();                // what was written is written again
#pragma unroll 1
        for (int g2 = 0; g2 < kTok / 32; ++g2)
          convert_any(p.scale + at.mt, p.nsx, p.T, (at.k + k) * kTok + 32 * g2 + 4 * (lane & 3), from + 4096u * g2,
                      from + 4096u * g2 + 2048u, to + 16u * g2);
      }
      if (lane == 0) mbar_arrive(xfree + 8u * x.i);
      if (kRelay && (wk & 3) == 0) {
        got = guard_wait(dfull + 8u * ds.i, ds.phase, ctl, p.guard, 36);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(conv0 + 8u * op.i);
      x.next(2);
      op.next(2);
      ds.next(2);
      // the windows before this one, after this warp's last stage of it: their
      // MMAs are done by then, and the one after it starts no earlier (a window
      // without a stage for this warp is the last of its tile or of the run,
      // which `finish` reads)
      while (ok && flushed < wi && k + 2 >= ns) ok = flush();
      if (!ok) break;
      k += 2;
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
// One block: one tile, kJoin of its columns; a thread: one feature, kJoin / 2
// columns, the parts of AT CTAs loaded at a time.  Many at a time where a tile
// has more than four parts, whose loads are all that it waits for, else two, as
// a load that is not needed costs its instructions (us with 2 and 16 at a time,
// the gradient's kernel included: 8192 x 4096, r = 64 18.3, 16.6; 16384 x 1024,
// r = 128 18.8, 13.5; 15360 x 8192, r = 384 89.4, 98.6; 2048 x 2048, r = 384 12.1,
// 13.3)
constexpr int kJoin = 8;
template <int AT> __global__ void __launch_bounds__(256) grad_join_kernel(const GradParams p, int ctas) {
  __shared__ int owner[2];
  const int tile = blockIdx.x;
  if (threadIdx.x < 2) {
    // the CTA of the tile's first and of its last unit: first_unit(i) <= unit <
    // first_unit(i + 1), that is i = ceil((unit + 1) ctas / units) - 1.  Two
    // threads divide (in every thread the divisions were half of this kernel)
    const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.stages;
    const int64_t next = static_cast<int64_t>(tile) * p.stages + (threadIdx.x == 0 ? 1 : p.stages);
    owner[threadIdx.x] = static_cast<int>((next * ctas - 1) / units);
  }
  __syncthreads();
  pdl_wait();
  const int i0 = owner[0], i1 = owner[1];
  const int mt = tile % p.mtiles, nt = tile / p.mtiles;
  const int m = threadIdx.x % kTcM, f = mt * kTcM + feature_of(m);
  if (i0 == i1 || f >= p.in) return;
  const int n0 = blockIdx.y * kJoin + threadIdx.x / kTcM;
  const int live = (p.ncols - n0 + 1) / 2;                  // of this thread's columns n0, n0 + 2, ...
  const int64_t slot = static_cast<int64_t>(p.ncols) * kTcM;
  // the first CTA's part is its second (its run of the tile began at the tile's
  // start), the others' their first
  const float *src = p.part + static_cast<int64_t>(i0) * 2 * slot + n0 * kTcM + m;
  float s[kJoin / 2] = {};
  for (int i = i0; i <= i1; i += AT, src += 2 * AT * slot) {
    float v[AT][kJoin / 2];
#pragma unroll
    for (int b = 0; b < AT; ++b) {
      const float *from = src + (2 * b + (b == 0 && i == i0 ? 1 : 0)) * slot;
#pragma unroll
      for (int j = 0; j < kJoin / 2; ++j) v[b][j] = i + b <= i1 && j < live ? __ldcs(from + 2 * j * kTcM) : 0.0f;
    }
#pragma unroll
    for (int b = 0; b < AT; ++b)
#pragma unroll
      for (int j = 0; j < kJoin / 2; ++j) s[j] += v[b][j];
  }
  const int col = nt * p.ncols + n0;
  float *dst = p.dA + static_cast<int64_t>(col) * p.in + f;
#pragma unroll
  for (int j = 0; j < kJoin / 2; ++j, dst += 2 * static_cast<int64_t>(p.in))
    if (j < live && col + 2 * j < p.r) *dst = s[j];
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// columns of r per tile: as few tiles as hold it at kMaxN each, of equal width
int tile_columns(int64_t r) {
  const int64_t tiles = dora::ceil_div(r, kMaxN);
  return static_cast<int>(dora::round_up(dora::ceil_div(r, tiles), 16));
}

// CTAs: at least four stages each, or a tile's where it has fewer, as parts
// have to be joined (us with 1, 2, 4, 8 stages: 16384 x 256, r = 256 11.9, 12.0,
// 10.9, 11.2; 16384 x 128, r = 16 10.4, 8.5, 8.5, 9.0; 256 x 512, r = 16 8.5, 6.8, 6.8,
// 6.8; 100 x 4096, r = 192, a stage a tile, 6.8 with one and 16.7 with four)
int64_t grad_ctas(int64_t T, int64_t in, int64_t r, int sms) {
  const int cols = tile_columns(r);
  const int64_t stages = dora::ceil_div(T, kTok);
  const int64_t units = dora::ceil_div(in, kTcM) * dora::ceil_div(r, cols) * stages;
  const int64_t runs = dora::ceil_div(units, stages < kWin / kTok ? stages : kWin / kTok);
  const int64_t room = static_cast<int64_t>(sms < kMaxSMs ? sms : kMaxSMs) * rings_of(cols).per_sm;
  return runs < room ? runs : room;
}

template <int NC>
dora_status launch_grad(const CUtensorMap &mX, const CUtensorMap &mD, GradParams p, int ctas, cudaStream_t cs) {
  constexpr Rings kR = rings_of(2 * NC);
  const size_t smem = 1024 + kR.x * (kRawBytes + kFactorBytes) + static_cast<size_t>(kR.d) * p.boxes * kBox + 512;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreadsG);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, lora_grad_kernel<NC>, mX, mD, p) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  // no tile is cut when every CTA's run is a whole number of tiles
  const int64_t tiles = static_cast<int64_t>(p.mtiles) * p.ntiles;
  if (tiles % ctas != 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(dora::ceil_div(p.ncols, kJoin)));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    const auto join = ctas > 4 * tiles ? &grad_join_kernel<16> : &grad_join_kernel<2>;
    if (cudaLaunchKernelEx(&cfg, join, p, ctas) != cudaSuccess) return DORA_ERR_CUDA;
    dora::count_launches(1);
  }
  return dora::launch_status();
}

}  // namespace

extern "C" size_t dora_lora_grad_q8_workspace(int64_t T, int64_t in, int64_t r) {
  if (bad_size(T, 0) || bad_size(in, 0) || r < 1 || r > kMaxR) return 0;
  if (T == 0 || in == 0) return 256;
  // two parts per CTA
  return static_cast<size_t>(2 * grad_ctas(T, in, r, kMaxSMs)) * tile_columns(r) * kTcM * sizeof(float);
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
      (const void *)lora_grad_kernel<8>, (const void *)lora_grad_kernel<16>, (const void *)lora_grad_kernel<32>,
      (const void *)lora_grad_kernel<64>, (const void *)lora_grad_kernel<96>};
  st = tc_init(device, &p.guard, kernels, sizeof(kernels) / sizeof(kernels[0]));
  if (st != DORA_OK) return st;
  p.T = static_cast<int>(T);
  p.in = static_cast<int>(in);
  p.r = static_cast<int>(r);
  p.ncols = tile_columns(r);
  p.boxes = static_cast<int>(dora::ceil_div(p.ncols, 64));
  p.mtiles = static_cast<int>(dora::ceil_div(in, kTcM));
  p.ntiles = static_cast<int>(dora::ceil_div(r, p.ncols));
  p.stages = static_cast<int>(dora::ceil_div(T, kTok));
  p.nsx = static_cast<int>(dora::ceil_div(in, kQBlock));
  p.scale = static_cast<const uint8_t *>(xscale);
  p.dA = dA;
  p.part = static_cast<float *>(workspace);
  CUtensorMap mX, mD;
  if (!map_q8(&mX, xq, T, in, kTok, kPromote) || !make_map(&mD, dxa, true, T, r, r, kTok, 128)) return DORA_ERR_CUDA;
  const int ctas = static_cast<int>(grad_ctas(T, in, r, info.sms));
  const int half = p.ncols / 2;
  if (half <= 8) return launch_grad<8>(mX, mD, p, ctas, cs);
  if (half <= 16) return launch_grad<16>(mX, mD, p, ctas, cs);
  if (half <= 32) return launch_grad<32>(mX, mD, p, ctas, cs);
  if (half <= 64) return launch_grad<64>(mX, mD, p, ctas, cs);
  return launch_grad<96>(mX, mD, p, ctas, cs);
}
