// x W^T of few tokens with a weight in 4 bits (see q4.cuh for the form) on the
// tensor cores of GB300 (sm_103a), without turning W into anything.
//
// tcgen05.mma kind::mxf8f6f4 takes E2M1 beside E4M3 and multiplies every 32 k of a
// row of either operand by a power of two, which is W's form.  x, a bf16, becomes
// two E4M3 pieces with a scale per 32 columns: h = E4M3(x / s), s the power of two
// that brings the group's largest magnitude to at most 448, and E4M3((x / s - h) 16)
// with the scale s / 16.  8 bits less the 4 of h leave 4, so x / s is their sum exactly
// where it is a multiple of 2^-13: always from 2^-6 on, 2^-14 of the largest magnitude.
// Of 32 normal values one is below that with low bits set in 0.2% of the cases, beside
// one 24 times louder in 1.7%.  What the two pieces leave of such a group is at most 2^-14
// and becomes two more, 2^22 finer.  A group that those do not hold either (an
// infinity, values more than 2^36 apart) is added at the end in fp32 (add_rest).  So x
// counts as it is, whatever its neighbours and however many tokens there are.
//
// The features are the M side, the tokens' pieces the N side (NT first pieces, NT
// second ones; in blocks that have such a group, third and fourth ones by MMAs of their
// own into the same sums).  A tile of 128 features and up to NT tokens is a cluster of
// CTAs that share its k range and meet in distributed shared memory, summed in rank
// order.
//   workers      up to 8 tokens: x of a block of 128 k into pieces, in place, each
//                warp the blocks of its own in turn.  More tokens are split by a launch
//                of its own before (q4_split_kernel), while this one's first blocks of W
//                are already on their way (8 x 8192 x 8192 14.4 us, 9 13.9).  Third and
//                fourth pieces of either, from x in memory: for one block in a hundred of
//                one token's, for two in five of 32 tokens'.  Then the result out of
//                tensor memory
//   next warp    tensor memory, scale words into it, MMA issue (four 32-wide steps per
//                block)
//   next warps   copies of W; copies of x or its pieces; W's scale words (BOX)
// The tensor core takes 4-bit values 16 to every 16 bytes of shared memory, in 8 of
// them.  TMA lays W out like that where its rows are whole blocks of 128 (BOX); else
// a block arrives as it is stored, in the half of its place, and a worker spreads it
// (1 x 8192 x 8192 11.6 us, 8224 columns 15.3).  From boxes of 256 k, whose rows are
// twice as long, all of W spread by workers took 2.4 us more than boxes of 128 do.
// W's scales go through registers, 16 bytes of a row at a time (1.8 us less than a copy
// of 4 bytes a row and block straight to their place).
//
// What bounds it: reading W, in boxes of 64-byte rows, which TMA takes one by one: 4.4 us
// for a launch and the first loads, then 4.9 TB/s (1 x 8192 x 8192 11.6 us, 16384 x 8192
// 18.7, 32768 x 8192 33.1; 14336 x 4096 10.9, 4096 x 14336 11.5; at the copy bandwidth the
// first takes 5.3).  Of more tokens also the workers: 16 x 8192 x 8192 15.1, 32 16.9, where
// values of one binade, which two pieces always hold, take 13.6 and 14.5.  8 tokens at as many
// experts of 2048 x 4096 11.9, 512 at 32 45 (22).  x whose groups no pieces hold is slow: where
// all are such, 1 x 8192 x 8192 75 us, 8 290, 32 1150.
// Every wait on a shared-memory barrier is bounded; a wait that gives up records
// a code in the library's device error word and all roles leave.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "q4.cuh"
#include "q4_mm.cuh"
#include "q8.cuh"
#include "q8_tc.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kKB = 128;                    // k per stage
constexpr unsigned kWBytes = kTcM * kKB;    // 16 KB of shared memory, 8 of W
constexpr int kMaxClusterLog = 3;           // 8 CTAs, the portable limit
// blocks asked into L2 while the launch before ends (1 x 8192 x 8192: 0 0.3 us more, 16 1.3)
constexpr int kAheadL2 = 6;
constexpr unsigned kSfBytes = kTcM * 4;     // scale words of 128 rows

// what a kernel of up to NT tokens a tile is made of
template <int NT, bool BOX> struct Few {
  static constexpr bool kSplit = NT > 8;                        // x comes in pieces
  static constexpr int N = 2 * NT;                              // rows of first and second pieces
  static constexpr int kPerSm = 2;                              // CTAs, limited by shared memory
  static constexpr int kStages = NT == 32 ? 3 : 4;              // blocks of W
  static constexpr int kXStages = NT == 8 ? 8 : kStages;        // blocks of x
  static constexpr int kWorkers = kStages < 4 ? 4 : kStages;
  static constexpr int kMma = kWorkers, kCopyW = kMma + 1, kCopyX = kMma + 2, kScale = kMma + 3, kThreads = 32 * (kMma + 3 + (BOX ? 1 : 0));
  static constexpr unsigned kXSf = 2 * kSfBytes;                // scale words of a block: first and second pieces, third and fourth
  static constexpr unsigned kXBytes = 2 * N * kKB;              // first and second pieces, third and fourth
  // tensor memory: the result, then 4 columns of W's scale words and 8 of x's for each stage
  static constexpr int kSfCol = 64, kSfStride = 12, kCols = 128;
  static constexpr int kLeftWords = 8;                          // a bit a block, of 256 in turn
  static constexpr int kBars = 3 * kStages + 3 * kXStages + 1;
  static constexpr size_t kSmem = 1024 + kStages * (kWBytes + kSfBytes) + kXStages * (kXBytes + kXSf) + 8 * kBars +
                                  sizeof(SharedCtl) + 4 * (kXStages + kLeftWords);
  // a wait goes by the parity of a phase, so a worker's slots are its own: it visits
  // every use of them in turn
  static_assert(kXStages % kStages == 0 && kStages <= kWorkers, "slots of a worker");
  static_assert(N <= kSfCol && kSfCol + kSfStride * kStages <= kCols && kPerSm * kCols <= 512, "tensor memory");
  static_assert(kPerSm * (kSmem + 1024) <= kSmemMax + 1024, "shared memory, with 1 KB of the system's a CTA");
  static_assert(NT * kTcM * 4 <= kStages * kWBytes + kXStages * kXBytes, "the parts lie in the blocks");
};

// 4 bytes into shared memory
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// an arrival on `bar` once this thread's copies so far have landed
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void prefetch_line(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ uint4 load_now16(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// The scale words of 128 rows, 512 bytes, into 4 columns of tensor memory, the same in
// each lane quadrant: row 32 j + l at byte 16 l + 4 j comes to lane l, column j
__device__ __forceinline__ uint32_t sf_at(int row) { return static_cast<uint32_t>((row % 32) * 16 + row / 32 * 4); }
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
  // 8 rows of 16 bytes, the next 8 128 bytes on; no swizzle
  const uint64_t d = ((saddr & 0x3FFFFu) >> 4) | (8ull << 16) | (8ull << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}
// whether two pieces hold a value of a group over its scale: whether it is a multiple of
// 2^-13, the step of fp32 from 1024 to 2048 (a NaN is none)
__device__ __forceinline__ bool held(float v) { return __fsub_rn(__fadd_rn(v, 1536.0f), 1536.0f) == v; }
// Two pieces of four values of a group of 32 that 8 neighbouring lanes hold, and the
// first one's scale byte; the second's is 4 less.  Returns which of the warp's four
// groups the pieces do not hold, 1 in the byte of each
__device__ __forceinline__ uint32_t split4(uint2 raw, uint32_t *h, uint32_t *l, uint32_t *byte) {
  float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u), __uint_as_float(raw.y << 16),
                __uint_as_float(raw.y & 0xffff0000u)};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, finite_bits(v[i]));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
  *byte = scale_byte(m);
  const float inv = scale_inverse(*byte);
  float f[4];
  bool all = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = inf_to_nan(v[i]) * inv;
    all = all && held(v[i]);
  }
  *h = quant4(v, 1.0f);
  dequant4(*h, 1.0f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = v[i] - f[i];
  *l = quant4(f, 16.0f);
  uint32_t left = __ballot_sync(0xffffffffu, !all);
  left |= left >> 4;
  left |= left >> 2;
  return (left | left >> 1) & 0x01010101u;
}

// A group, a value a lane: what split4's pieces leave of it in two more, with scale bytes
// 22 and 26 less than the first's.  False where they do not hold it
__device__ __forceinline__ bool split_rest(float v, uint32_t *h, uint32_t *l, uint32_t *byte) {
  *byte = scale_byte(__reduce_max_sync(0xffffffffu, finite_bits(v)));
  // (a NaN is one in the first piece already, an infinity is held by none)
  float r = v == v ? inf_to_nan(v) * scale_inverse(*byte) : 0.0f;
  auto less = [](float x, uint32_t piece) { return x - dequant2(piece, 1.0f).x; };
  r = less(r, quant2(r, 0.0f, 1.0f)) * 16.0f;
  r = less(r, quant2(r, 0.0f, 1.0f)) * 262144.0f;
  *h = quant2(r, 0.0f, 1.0f) & 255u;
  r = less(r, *h) * 16.0f;
  *l = quant2(r, 0.0f, 1.0f) & 255u;
  return __all_sync(0xffffffffu, less(r, *l) == 0.0f) && *byte >= 26u;
}
// this lane's column of a group of x
__device__ __forceinline__ float load_bf16(const __nv_bfloat16 *p) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(p))) << 16);
}

// x [T, in] into pieces: first ones [T, in], second ones [T, in], then [blocks, 2, T] words, a byte
// per 32 columns: scales of the first; 1 where the two do not hold the group
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads)
q4_split_kernel(const __nv_bfloat16 *__restrict__ x, int T, int in, uint8_t *__restrict__ pieces) {
  pdl_trigger();
  const int c = 4 * static_cast<int>(blockIdx.x * kSplitThreads + threadIdx.x);
  const int64_t all = static_cast<int64_t>(T) * in;
  uint32_t *words = reinterpret_cast<uint32_t *>(pieces + 2 * all);
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    // a warp holds a block of 128 columns; any scale past the row
    const int64_t at = static_cast<int64_t>(t) * in + c;
    uint32_t h, l, b;
    const uint32_t left = split4(c < in ? __ldg(reinterpret_cast<const uint2 *>(x + at)) : make_uint2(0, 0), &h, &l, &b);
    if (c < in) {
      *reinterpret_cast<uint32_t *>(pieces + at) = h;
      *reinterpret_cast<uint32_t *>(pieces + all + at) = l;
    }
    b |= __shfl_down_sync(0xffffffffu, b, 8) << 8;      // lanes 0 and 16 hold two bytes,
    b |= __shfl_down_sync(0xffffffffu, b, 16) << 16;    // lane 0 four
    if ((threadIdx.x & 31) == 0 && c < in) {
      uint32_t *at = words + 2 * static_cast<int64_t>(c / kKB) * T + t;
      at[0] = b;
      at[T] = left;
    }
  }
}

// The groups of x that no pieces hold, in blocks that `bits` names, added to the tile's result
// [token][feature] in fp32 and in the order of k, from W and x as they are; a thread has
// feature f of the tile.  It is slow, as every group of such a block is looked at, and seldom called.
__device__ __forceinline__ void add_rest(const Q4Params &p, const uint8_t *wq, const __nv_bfloat16 *x, const Tile &o, int f0,
                                         int f, int kb0, int nb, const uint32_t *bits, float *part) {
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & 31, G = p.in / kQ4Group;
  const bool has = f0 + f < p.out;
  const int64_t row = static_cast<int64_t>(o.e) * p.out + f0 + f;
#pragma unroll 1
  for (int b = 0; b < nb; ++b) {
    if ((bits[b / 32 % 8] >> (b % 32) & 1u) == 0) continue;
#pragma unroll 1
    for (int g = 4 * (kb0 + b); g < min(4 * (kb0 + b) + 4, G); ++g) {
      const uint4 q = has ? __ldcg(reinterpret_cast<const uint4 *>(wq + row * (p.in / 2) + g * (kQ4Group / 2))) : make_uint4(0, 0, 0, 0);
      const float s = q4_scale(has ? __ldcg(p.scale + row * G + g) : 0u);
      const uint32_t words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll 1
      for (int t0 = o.t0; t0 < o.t1; t0 += kAtOnce) {
        float v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          v[i] = t0 + i < o.t1 ? load_bf16(x + static_cast<int64_t>(t0 + i) * p.in + g * kQ4Group + lane) : 0.0f;
#pragma unroll 1
        for (int i = 0; i < min(kAtOnce, o.t1 - t0); ++i) {
          const float xv = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
          uint32_t h, l, byte;
          if (split_rest(xv, &h, &l, &byte) || __all_sync(0xffffffffu, held(inf_to_nan(xv) * scale_inverse(byte)))) continue;
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < kQ4Group; j += 2) {
            const float2 c = q4_value2(words[j / 8] >> (4 * (j % 8)) & 0xffu);
            sum = fmaf(__shfl_sync(0xffffffffu, xv, j), c.x * s, sum);
            sum = fmaf(__shfl_sync(0xffffffffu, xv, j + 1), c.y * s, sum);
          }
          part[(t0 + i - o.t0) * kTcM + f] += sum;
        }
      }
    }
  }
}

template <int NT, bool BOX>
__global__ void __launch_bounds__(Few<NT, BOX>::kThreads, Few<NT, BOX>::kPerSm)
q4_few_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const Q4Params p,
              const uint8_t *wq, const __nv_bfloat16 *x, const uint32_t *xwords) {
  using F = Few<NT, BOX>;
  constexpr int S = F::kStages, XS = F::kXStages, N = F::N;
  constexpr bool PRE = F::kSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *xs0 = smem + S * kWBytes;                         // x's pieces, [XS]
  uint8_t *wsf0 = xs0 + XS * F::kXBytes, *xsf0 = wsf0 + S * kSfBytes;   // scale words, as sf_at says
  uint64_t *bars = reinterpret_cast<uint64_t *>(xsf0 + XS * F::kXSf);
  // barriers: of a block of W here, spread (!BOX), empty; of a block of x here, split, empty; the result
  const uint32_t wfull0 = smem_u32(bars), wready0 = wfull0 + 8u * S, wempty0 = wready0 + 8u * S, xfull0 = wempty0 + 8u * S,
                 xready0 = xfull0 + 8u * XS, xempty0 = xready0 + 8u * XS, accf = xempty0 + 8u * XS;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + F::kBars);
  // which blocks of x have third and fourth pieces [XS]; which have groups that no pieces hold
  volatile uint32_t *wide = reinterpret_cast<uint32_t *>(ctl + 1);
  uint32_t *left_out = reinterpret_cast<uint32_t *>(ctl + 1) + XS;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(wfull0 + 8u * s, BOX ? 2 : 1);               // the box; the scale words
      mbar_init(wready0 + 8u * s, 1);
      mbar_init(wempty0 + 8u * s, 1);
    }
    for (int s = 0; s < XS; ++s) {
      mbar_init(xfull0 + 8u * s, PRE ? 33 : 1);
      mbar_init(xready0 + 8u * s, 1);
      mbar_init(xempty0 + 8u * s, 1);
    }
    mbar_init(accf, 1);
    ctl->abort = 0;
    for (int i = 0; i < F::kLeftWords; ++i) left_out[i] = 0;
    fence_barrier_init();
    prefetch_map(&mW);
    prefetch_map(&mX);
  }
  // scale words that nothing writes: of rows without a token or a feature
  for (int i = threadIdx.x; i < static_cast<int>((S * kSfBytes + XS * F::kXSf) / 4); i += F::kThreads)
    reinterpret_cast<uint32_t *>(wsf0)[i] = 0x7f7f7f7fu;
  if (warp == F::kMma) {
    __syncwarp();
    tmem_alloc(smem_u32(&ctl->tmem_base), F::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const uint32_t rank = cluster_ctarank(), clog = 31u - __clz(csize);      // a power of two
  const int tile = static_cast<int>(blockIdx.x >> clog);
  const uint32_t blocks = static_cast<uint32_t>((p.kdim + kKB - 1) / kKB);
  // blocks kb0 to kb0 + nb of k, at least one: a cluster has no more CTAs than there are
  const int kb0 = static_cast<int>((blocks * rank) >> clog), nb = static_cast<int>((blocks * (rank + 1)) >> clog) - kb0;
  // Without pieces the launch before this one may still run: nothing is read or
  // written before it has ended, but the first blocks of W are on their way into L2
  // (by lines: TMA takes rows of a box one by one, and that is what bounds this
  // kernel).  With pieces it is q4_split_kernel, which itself started after all
  // launches before it had ended: only what it writes is waited for
  pdl_trigger();
  if (!PRE) {
    if (!p.offsets)
      for (int f = threadIdx.x; f < kTcM && tile * kTcM + f < p.out; f += F::kThreads) {
        const uint8_t *row = wq + static_cast<int64_t>(tile * kTcM + f) * (p.in / 2) + kb0 * (kKB / 2);
        for (int c = 0; c < min(nb, kAheadL2) * (kKB / 2); c += 128) prefetch_line(row + c);
        prefetch_line(p.scale + static_cast<int64_t>(tile * kTcM + f) * (p.in / kQ4Group) + 4 * kb0);
      }
    pdl_wait();
  }
  Tile o = {0, tile, 0, p.T};       // one weight: all tokens are one tile
  const bool work = !p.offsets || find_tile(p, tile, &o);                  // all of a cluster alike
  const int ntok = o.t1 - o.t0, f0 = o.ft * kTcM, G = p.in / kQ4Group;
  // W's scales of row f, block kb0 + b
  auto scale_at = [&](int f, int b) { return (static_cast<int64_t>(o.e) * p.out + f0 + f) * G + 4 * (kb0 + b); };
  bool ok = true;

  if (!work) {
    // no tile for this cluster
  } else if (warp == F::kCopyW) {
    // ---------------------------------------------------------------- W and its scales
    ok = !loads_withheld(p.guard);
    bool issued = false;
    Ring st(S);
    for (int b = 0; b < nb && ok; ++b, st.next()) {
      ok = guard_wait(wempty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 71);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t full = wfull0 + 8u * st.i, at = smem_u32(smem) + st.i * kWBytes;
      if (elect_one()) {
        // a box counts the bytes that it reads
        mbar_expect_tx(full, kWBytes / 2);
        if (BOX) tma_load_3d(at, &mW, (kb0 + b) * kKB, f0, o.e, full);
        else tma_load_3d(at, &mW, (kb0 + b) * (kKB / 2), f0, o.e, full);
      }
      __syncwarp();
      issued = true;
    }
    if (!ok && issued) {
      // boxes in flight, whose barrier nobody may wait for after an abort: they land
      // within microseconds, wait 1 ms
      const unsigned long long c0 = globaltimer();
      while (globaltimer() - c0 < 1000000ull) {
      }
    }
  } else if (BOX && warp == F::kScale) {
    // ---------------------------------------------------------------- W's scales
    // lane l has rows l, l + 32, ...: 16 bytes of each, four blocks, are on their way
    // while the four before go block by block to where sf_at says
    const bool wide = G % 16 == 0 && kb0 % 4 == 0;
    uint4 next[4];
    auto fetch = [&](int b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool has = f0 + 32 * j + lane < p.out;
        const uint8_t *at = p.scale + scale_at(32 * j + lane, b);
        if (wide) {
          next[j] = has && b < nb ? load_now16(at) : make_uint4(0, 0, 0, 0);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = has && b + i < nb ? load_now(reinterpret_cast<const uint32_t *>(at) + i) : 0u;
          next[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    };
    fetch(0);
    Ring st(S);
    for (int b0 = 0; b0 < nb && ok; b0 += 4) {
      uint4 now[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) now[j] = next[j];
      fetch(b0 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (b0 + i >= nb) break;
        ok = guard_wait(wempty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 79);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        auto word = [&](const uint4 &v) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
        *reinterpret_cast<uint4 *>(wsf0 + st.i * kSfBytes + 16 * lane) =
            make_uint4(word(now[0]), word(now[1]), word(now[2]), word(now[3]));
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(wfull0 + 8u * st.i);
        st.next();
      }
    }
  } else if (warp == F::kCopyX) {
    // ---------------------------------------------------------------- x or its pieces
    ok = !loads_withheld(p.guard);
    bool issued = false;
    if (PRE) pdl_wait();
    Ring st(XS);
    for (int b = 0; b < nb && ok; ++b, st.next()) {
      ok = guard_wait(xempty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 72);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t xs = smem_u32(xs0) + st.i * F::kXBytes, full = xfull0 + 8u * st.i;
      const int k = (kb0 + b) * kKB;
      if (elect_one()) {
        mbar_expect_tx(full, N * kKB);
        // x as it is: the 256 bytes of token t where its two pieces go, rows t and NT + t
        tma_load_2d(xs, &mX, k, o.t0, full);
        tma_load_2d(xs + NT * kKB, &mX, PRE ? k : k + 64, PRE ? p.T + o.t0 : o.t0, full);
      }
      __syncwarp();
      issued = true;
      if (PRE) {
        const uint32_t to = smem_u32(xsf0) + st.i * F::kXSf;
        const uint32_t *from = xwords + 2 * static_cast<int64_t>(kb0 + b) * p.T + o.t0;
        for (int t = lane; t < ntok; t += 32) copy4(to + sf_at(t), from + t);
        copies_arrive(full);
      }
    }
    copies_wait();
    if (!ok && issued) {
      const unsigned long long c0 = globaltimer();
      while (globaltimer() - c0 < 1000000ull) {
      }
    }
  } else if (warp == F::kMma) {
    // ---------------------------------------------------------------- MMA issuer
    Ring st(S), xt(XS);
    for (int b = 0; b < nb; ++b, st.next(), xt.next()) {
      ok = guard_wait(xready0 + 8u * xt.i, xt.phase, ctl, p.guard, 73);
      ok = ok && guard_wait((BOX ? wfull0 : wready0) + 8u * st.i, st.phase, ctl, p.guard, 74);
      if (!__all_sync(0xffffffffu, ok)) break;
      // x's scale words came by copies that the tensor core's reads are not ordered after
      if (PRE) fence_async_proxy();
      tc_fence_after();
      const uint64_t da = sdesc<32>(smem_u32(smem) + st.i * kWBytes), db = sdesc<32>(smem_u32(xs0) + xt.i * F::kXBytes);
      const uint32_t sf = tmem + F::kSfCol + F::kSfStride * st.i;
      const bool more = wide[xt.i] != 0;
      if (elect_one()) {
        // (a copy runs before the MMAs that this thread issues after it)
        copy_scales(sf, smem_u32(wsf0) + st.i * kSfBytes);
        copy_scales(sf + 4, smem_u32(xsf0) + xt.i * F::kXSf);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_q8(tmem, da + 2u * k, db + 2u * k, idesc_q8(kTcM, N, k, false) | 5u << 7 /* A: E2M1 */, sf, sf + 4,
                 b != 0 || k != 0 ? 1u : 0u);
        if (more) {
          copy_scales(sf + 8, smem_u32(xsf0) + xt.i * F::kXSf + kSfBytes);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_q8(tmem, da + 2u * k, db + (N * kKB >> 4) + 2u * k, idesc_q8(kTcM, N, k, false) | 5u << 7, sf, sf + 8, 1u);
        }
        mma_commit(wempty0 + 8u * st.i);
        mma_commit(xempty0 + 8u * xt.i);
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(accf);
      wait_drain_ns(accf, 0, kWaitNs);   // every MMA issued is done before this CTA's memory is given back
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- workers
    // blocks warp, warp + S, ...
    if (warp < S) {
      Ring st(S), xt(XS);
      for (int i = 0; i < warp; ++i) {
        st.next();
        xt.next();
      }
      // !BOX: the two aligned words that hold the scale bytes of rows 32 j + lane
      uint32_t sw[4][2];
      auto fetch = [&](int b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int f = 32 * j + lane;
          const int64_t at = scale_at(f, b), from = at & ~int64_t(3);
          const bool has = b < nb && f0 + f < p.out;
          sw[j][0] = has ? load_now(reinterpret_cast<const uint32_t *>(p.scale + from)) : 0u;
          // the scales end on 16 bytes
          sw[j][1] = has && at != from && from + 4 < static_cast<int64_t>(p.experts) * p.out * G
                         ? load_now(reinterpret_cast<const uint32_t *>(p.scale + from + 4)) : 0u;
        }
      };
      if (!BOX) fetch(warp);
      constexpr int kAtOnce = 4;                     // tokens, or groups left over, worked on together
      // PRE: a byte of a token's word says whether the two pieces leave something of a group
      auto mark = [&](int b) { return b < nb && lane < ntok ? __ldcg(xwords + (2 * static_cast<int64_t>(kb0 + b) + 1) * p.T + o.t0 + lane) : 0u; };
      uint32_t marks = 0;
      if (PRE) {
        pdl_wait();
        marks = mark(warp);
      }
      for (int b = warp; b < nb; b += S) {
        uint8_t *xs = xs0 + xt.i * F::kXBytes, *sf = xsf0 + xt.i * F::kXSf;
        uint32_t over[4] = {}, rest[4] = {};         // of each group, tokens of which the two pieces leave something; the four too
        // third and fourth pieces, zeros but for these groups.  x comes from memory once more.  PRE:
        // while the first two are on their way, once the MMAs of the block before here are done
        auto more_pieces = [&]() {
          const __nv_bfloat16 *from = x + static_cast<int64_t>(o.t0) * p.in + (kb0 + b) * kKB + lane;
          uint8_t *sf2 = sf + kSfBytes;
          bool first = true;
#pragma unroll 1
          while ((over[0] | over[1] | over[2] | over[3]) != 0) {
            int at[kAtOnce];                         // group and token
            float v[kAtOnce];
            uint32_t h[kAtOnce], l[kAtOnce], byte[kAtOnce];
            bool all[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              const int g = over[0] != 0 ? 0 : over[1] != 0 ? 1 : over[2] != 0 ? 2 : 3;
              const uint32_t m = over[0] != 0 ? over[0] : over[1] != 0 ? over[1] : over[2] != 0 ? over[2] : over[3];
              at[j] = m != 0 ? 32 * g + __ffs(m) - 1 : -1;
              v[j] = m != 0 ? load_bf16(from + static_cast<int64_t>(at[j] & 31) * p.in + g * kQ4Group) : 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i == g) over[i] &= over[i] - 1;
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) all[j] = split_rest(v[j], &h[j], &l[j], &byte[j]);
            if (first) {
              if (PRE) {
                // (a wait that may be left out: this warp saw the use before here arrive, so
                // the phase is that one's or it is over)
                ok = guard_wait(xempty0 + 8u * xt.i, xt.phase ^ 1u, ctl, p.guard, 78);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
              }
              for (int i = lane; i < N * kKB / 16; i += 32) reinterpret_cast<uint4 *>(xs + N * kKB)[i] = make_uint4(0, 0, 0, 0);
              __syncwarp();
              first = false;
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              if (at[j] < 0) break;
              const int g = at[j] >> 5, t = at[j] & 31, to = ((2 * g + (lane >> 4)) ^ (t & 7)) * 16 + (lane & 15);
              if (all[j]) {
                xs[(N + t) * kKB + to] = static_cast<uint8_t>(h[j]);
                xs[(N + NT + t) * kKB + to] = static_cast<uint8_t>(l[j]);
                if (lane == 0) {
                  sf2[sf_at(t) + g] = static_cast<uint8_t>(byte[j] - 22u);
                  sf2[sf_at(NT + t) + g] = static_cast<uint8_t>(byte[j] - 26u);
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (i == g) rest[i] |= 1u << t;
              }
            }
          }
        };
        bool more = false;
        if constexpr (PRE) {
#pragma unroll
          for (int g = 0; g < 4; ++g) over[g] = __ballot_sync(0xffffffffu, (marks >> (8 * g) & 255u) != 0);
          marks = mark(b + S);
          more = (over[0] | over[1] | over[2] | over[3]) != 0;
          if (more) {
            more_pieces();
            if (!ok) break;
          }
        }
        ok = guard_wait(xfull0 + 8u * xt.i, xt.phase, ctl, p.guard, 75);
        if (!__all_sync(0xffffffffu, ok)) break;
        if constexpr (PRE) {
          // the second pieces' scales
          if (lane < ntok)
            *reinterpret_cast<uint32_t *>(sf + sf_at(NT + lane)) = *reinterpret_cast<const uint32_t *>(sf + sf_at(lane)) - 0x04040404u;
        } else {
          // a place without a token holds anything: its column of the result is not read
          uint32_t groups = 0;
          // four at a time, whose steps hide one another's latencies
#pragma unroll 1
          for (int t0 = 0; t0 < ntok; t0 += kAtOnce) {
            uint2 v[kAtOnce];
            uint32_t h[kAtOnce], l[kAtOnce], sb[kAtOnce];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
              v[j] = *reinterpret_cast<const uint2 *>(xs + (t0 + j + (lane >= 16 ? NT : 0)) * 128 + (lane & 15) * 8);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              const uint32_t left = split4(v[j], &h[j], &l[j], &sb[j]);
              if (t0 + j < ntok) groups |= left << (t0 + j);
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              const int t = t0 + j, to = ((lane >> 2) ^ (t & 7)) * 16 + (lane & 3) * 4;
              *reinterpret_cast<uint32_t *>(xs + t * 128 + to) = h[j];
              *reinterpret_cast<uint32_t *>(xs + (NT + t) * 128 + to) = l[j];      // NT % 8 == 0: the same swizzle
              if ((lane & 7) == 0) {
                sf[sf_at(t) + (lane >> 3)] = static_cast<uint8_t>(sb[j]);
                sf[sf_at(NT + t) + (lane >> 3)] = static_cast<uint8_t>(sb[j] - 4u);
              }
            }
          }
          more = groups != 0;
          if (more) {
#pragma unroll
            for (int g = 0; g < 4; ++g) over[g] = groups >> (8 * g) & 255u;
            more_pieces();
          }
        }
        if (more && (rest[0] | rest[1] | rest[2] | rest[3]) != 0) {
          // groups that no pieces hold: zeros (add_rest)
          __syncwarp();
#pragma unroll 1
          for (int g = 0; g < 4; ++g)
#pragma unroll 1
            for (uint32_t m = g == 0 ? rest[0] : g == 1 ? rest[1] : g == 2 ? rest[2] : rest[3]; m != 0; m &= m - 1) {
              const int t = __ffs(m) - 1, to = ((2 * g + (lane >> 4)) ^ (t & 7)) * 16 + (lane & 15);
              xs[t * kKB + to] = 0;
              xs[(NT + t) * kKB + to] = 0;
            }
          if (lane == 0) atomicOr(left_out + b / 32 % F::kLeftWords, 1u << (b % 32));
        }
        if (lane == 0) wide[xt.i] = more ? 1u : 0u;
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(xready0 + 8u * xt.i);
        if constexpr (!BOX) {
          ok = guard_wait(wfull0 + 8u * st.i, st.phase, ctl, p.guard, 76);
          if (!__all_sync(0xffffffffu, ok)) break;
          // 64 bytes of each of 128 rows, 64-byte swizzle; lane l has rows l, l + 32, ...
          uint8_t *at = smem + st.i * kWBytes;
          uint4 w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int f = 32 * (j / 4) + lane;
            w[j] = *reinterpret_cast<const uint4 *>(at + f * 64 + (((j % 4) ^ ((f >> 1) & 3)) * 16));
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            // 32 values: 8 bytes to each of chunks 2 c and 2 c + 1 of the row
            const int f = 32 * (j / 4) + lane, c = j % 4;
            *reinterpret_cast<uint2 *>(at + f * 128 + (((2 * c) ^ (f & 7)) * 16)) = make_uint2(w[j].x, w[j].y);
            *reinterpret_cast<uint2 *>(at + f * 128 + (((2 * c + 1) ^ (f & 7)) * 16)) = make_uint2(w[j].z, w[j].w);
          }
          // past the last group of a row lies the next row's first
          const int left = G - 4 * (kb0 + b);
          const uint32_t none = left < 4 ? 0xffffffffu << (8 * left) : 0u;
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = (__funnelshift_r(sw[j][0], sw[j][1], 8 * static_cast<uint32_t>(scale_at(32 * j + lane, b) & 3)) & ~none) |
                   (0x7f7f7f7fu & none);
          *reinterpret_cast<uint4 *>(wsf0 + st.i * kSfBytes + 16 * lane) = make_uint4(v[0], v[1], v[2], v[3]);
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) mbar_arrive(wready0 + 8u * st.i);
          fetch(b + S);
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
          st.next();
          xt.next();
        }
      }
    }
    // ---------------------------------------------------------------- result
    asm volatile("bar.sync 1, %0;" ::"n"(32 * F::kWorkers) : "memory");   // all workers' words of left_out
    if (warp < 4) {
      // into shared memory as [token][feature]: the blocks are free once the last MMA
      // is done
      const bool got = guard_wait(accf, 0, ctl, p.guard, 77);
      ok = __all_sync(0xffffffffu, got) && ok;
      tc_fence_after();
      const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp) * 32u << 16);
      float *part = reinterpret_cast<float *>(smem);
#pragma unroll
      for (int c = 0; c < NT; c += 8) {
        if (c < ntok) {
          float a[8], d[8];
          tmem_ld<8>(lane_addr + c, a);
          tmem_ld<8>(lane_addr + NT + c, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) part[(c + i) * kTcM + 32 * warp + lane] = ok ? a[i] + d[i] : 0.0f;
        }
      }
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < F::kLeftWords; ++i) any |= left_out[i];
      if (any != 0 && ok) add_rest(p, wq, x, o, f0, 32 * warp + lane, kb0, nb, left_out, part);
    }
  }
  // the pieces are written, whoever reads them: no launch after this one comes
  // before the split has ended
  if (PRE) pdl_wait();
  tc_fence_before();
  __syncwarp();   // the cluster's barrier takes whole warps
  if (csize > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (work) {
    // the parts of the cluster in rank order, one rounding to bf16: four
    // features a thread, neighbouring threads on neighbouring features
    const int quads = ntok * 32;
    const uint32_t base = smem_u32(smem);
    for (int i = static_cast<int>(rank) * F::kThreads + threadIdx.x; i < quads; i += static_cast<int>(csize) * F::kThreads) {
      const int t = o.t0 + i / 32, f = f0 + 4 * (i % 32);
      if (f >= p.nfeat) continue;   // nothing is read that no store waits for
      float4 s = ld_cluster_f32x4(mapa_shared(base + 16u * i, 0));
      for (uint32_t c = 1; c < csize; ++c) {
        const float4 v = ld_cluster_f32x4(mapa_shared(base + 16u * i, c));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      *reinterpret_cast<uint2 *>(p.y + static_cast<int64_t>(t) * p.nfeat + f) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
  }
  __syncwarp();
  if (csize > 1) cluster_sync();   // no CTA leaves while another reads its part
  else __syncthreads();
  if (warp == F::kMma) {
    __syncwarp();
    tmem_dealloc(tmem, F::kCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
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

template <int NT, bool BOX>
void few_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int64_t tiles, int cluster, cudaStream_t cs) {
  using F = Few<NT, BOX>;
  *cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg->gridDim = dim3(static_cast<unsigned>(tiles * cluster));
  cfg->blockDim = dim3(F::kThreads);
  cfg->dynamicSmemBytes = F::kSmem;
  cfg->stream = cs;
  cfg->attrs = attr;
  cfg->numAttrs = 2;
}

// clusters of 2^`log` CTAs that are resident at once, at least: the query counts one CTA an
// SM of these kernels where two run, and twice that leaves out what remains of each group of SMs
template <int NT, bool BOX> int resident_clusters(int device, int log) {
  using F = Few<NT, BOX>;
  static std::mutex mu;
  static int known[64][4] = {};   // clusters + 1
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  int &k = known[device][log];
  if (k == 0) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    few_config<NT, BOX>(&cfg, attr, 1, 1 << log, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, q4_few_kernel<NT, BOX>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    int one = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&one, q4_few_kernel<NT, BOX>, F::kThreads, F::kSmem) != cudaSuccess || one < 1) one = 1;
    k = n * F::kPerSm / one + 1;
  }
  return k - 1;
}

template <int NT, bool BOX>
dora_status launch(const void *x, const void *wq, Q4Params p, void *workspace, int device, int sms, cudaStream_t cs) {
  using F = Few<NT, BOX>;
  const int64_t groups = p.offsets ? (p.experts < p.T ? p.experts : p.T) : 1;
  // an expert of n tokens has (n - 1) / NT + 1
  const int64_t tiles = p.ftiles * (p.offsets ? (p.T - groups) / NT + groups : 1);
  // the k range over as many CTAs as keep all clusters resident.  Up to 27 CTAs on 16 SMs
  // were, as clusters of 8 too, where the query counts fewer: that matters for 29 to 32 tiles
  // (1 x 4096 x 4096 6.4 us, by the query alone 7.3; 4096 x 8192 8.3, 10.8; 4096 x 14336 11.4,
  // 16.3, 32 tokens 17.5, 20.9), for other sizes both choose alike (20 and 28 tiles, 48 and 64)
  int log = 0;
  const int64_t blocks = dora::ceil_div(p.in, kKB);
  while (log < kMaxClusterLog && (2 << log) <= blocks &&
         (tiles <= resident_clusters<NT, BOX>(device, log + 1) ||
          tiles << (log + 1) <= sms * 27 / 16))
    ++log;
  if (tiles << log > kMaxDim) return DORA_ERR_SHAPE;
  p.ntok = NT;
  p.tiles = static_cast<int>(tiles);
  CUtensorMap mW, mX;
  const int64_t all = static_cast<int64_t>(p.T) * p.in;
  uint8_t *pieces = static_cast<uint8_t *>(workspace);
  if (!(BOX ? map_w4(&mW, wq, p.experts, p.out, p.in) : map_w(&mW, wq, p.experts, p.out, p.in))) return DORA_ERR_CUDA;
  if (F::kSplit) {
    if (!map_q8(&mX, pieces, 2 * static_cast<int64_t>(p.T), p.in, NT, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)) return DORA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(dora::ceil_div(p.in, 4 * kSplitThreads)), p.T < 65535 ? p.T : 65535);
    q4_split_kernel<<<grid, kSplitThreads, 0, cs>>>(static_cast<const __nv_bfloat16 *>(x), p.T, p.in, pieces);
    if (dora::launch_status() != DORA_OK) return DORA_ERR_CUDA;
    dora::count_launches(1);
  } else if (!map_x(&mX, x, p.T, p.in, NT)) {
    return DORA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  few_config<NT, BOX>(&cfg, attr, tiles, 1 << log, cs);
  if (cudaLaunchKernelEx(&cfg, q4_few_kernel<NT, BOX>, mW, mX, p, static_cast<const uint8_t *>(wq),
                         static_cast<const __nv_bfloat16 *>(x),
                         reinterpret_cast<const uint32_t *>(pieces + 2 * all)) !=
      cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

template <int NT>
dora_status launch(const void *x, const void *wq, const Q4Params &p, void *workspace, int device, int sms, cudaStream_t cs) {
  // boxes of 4-bit values take whole blocks of 128 and 32-byte rows
  return p.in % kKB == 0 && dora::aligned(wq, 32) ? launch<NT, true>(x, wq, p, workspace, device, sms, cs)
                                                  : launch<NT, false>(x, wq, p, workspace, device, sms, cs);
}

}  // namespace

namespace dora {

size_t q4_few_workspace(int64_t T, int64_t in, int64_t experts) {
  return q4_tile(T, experts) <= 8 ? 0 : static_cast<size_t>(2 * T * in + 8 * T * ceil_div(in, kKB));
}

dora_status matmul_q4_few(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T,
                          int64_t out, int64_t in, int64_t experts, void *y, void *workspace, cudaStream_t cs) {
  DeviceInfo info;
  int device = 0;
  dora_status st = current_device(&info, &device);
  if (st != DORA_OK) return st;
  static const void *const kernels[] = {
      (const void *)q4_few_kernel<8, false>,  (const void *)q4_few_kernel<8, true>,   (const void *)q4_few_kernel<16, false>,
      (const void *)q4_few_kernel<16, true>,  (const void *)q4_few_kernel<32, false>, (const void *)q4_few_kernel<32, true>};
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
  p.ftiles = static_cast<int>(ceil_div(out, kTcM));
  const int64_t n = q4_tile(T, experts);
  if (n <= 8) return launch<8>(x, wq, p, workspace, device, info.sms, cs);
  if (n <= 16) return launch<16>(x, wq, p, workspace, device, info.sms, cs);
  return launch<32>(x, wq, p, workspace, device, info.sms, cs);
}

}  // namespace dora
