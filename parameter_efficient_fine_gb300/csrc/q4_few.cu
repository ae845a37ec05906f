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
//   first warps  scale words into tensor memory, each warp its lane quadrant; then
//                the result out of it.  Up to 8 tokens they also make the pieces of
//                x, in place, three groups of four warps taking turns; more tokens
//                are split by a launch of its own before (q4_split_kernel), while
//                this one's first blocks of W are already on their way
//   next warp    tensor memory, MMA issue (four 32-wide steps per 128 k)
//   last two     copies of W, its scales and x.  W: 16 values, 8 bytes, to every 16
//                bytes of shared memory, the layout that the tensor core takes 4-bit
//                values in.  TMA does that (BOX) where rows are whole blocks of 128;
//                other rows come by asynchronous copies of 8 bytes
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
constexpr int kQuads = 4, kCopyWarps = 2;   // warps of a group, of copies
constexpr int kMaxCluster = 8;              // the portable limit

// what a kernel of up to NT tokens a tile is made of
template <int NT> struct Few {
  static constexpr bool kSplit = NT > 8;                        // x comes in pieces
  static constexpr int N = 2 * NT;                              // rows of pieces
  static constexpr int kGroups = kSplit ? 1 : 3;                // turns
  static constexpr int kStages = NT == 8 ? 6 : NT == 16 ? 5 : NT == 64 ? 3 : 4;
  static constexpr int kPerSm = NT == 128 ? 1 : 2;              // CTAs, limited by shared memory
  static constexpr int kMma = kGroups * kQuads, kCopy = kMma + 1, kThreads = 32 * (kCopy + kCopyWarps);
  static constexpr unsigned kXBytes = N * kKB, kStage = kWBytes + kXBytes;
  // tensor memory: the result, then 4 columns of W's scale words and one per 32 rows of x's for each stage
  static constexpr int kXCols = (N + 31) / 32, kSfCol = N < 64 ? 64 : N, kSfStride = kXCols > 4 ? 16 : 8;
  static constexpr int kCols = NT == 128 ? 512 : NT == 64 ? 256 : 128;
  static constexpr int kWords = kSplit ? NT : N;                // scale words of x in shared memory, a stage
  static constexpr size_t kSmem = 1024 + kStages * (kStage + 4 * (kTcM + kWords)) + 8 * (4 * kStages + 1) + sizeof(SharedCtl);
  // each group visits every use of its slots
  static_assert(kStages % kGroups == 0 && kSfCol + kSfStride * kStages <= kCols && kPerSm * kCols <= 512, "stages, tensor memory");
  static_assert(kPerSm * (kSmem + 1024) <= kSmemMax + 1024, "shared memory, with 1 KB of the system's a CTA");
  static_assert(NT * kTcM * 4 <= kStages * kStage, "the parts lie in the stages");
};

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

// Two pieces of four values of a group of 32 that 8 neighbouring lanes hold, and the
// first one's scale byte; the second's is 4 less
__device__ __forceinline__ void split4(uint2 raw, uint32_t *h, uint32_t *l, uint32_t *byte) {
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
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = inf_to_nan(v[i]) * inv;
  *h = quant4(v, 1.0f);
  dequant4(*h, 1.0f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = v[i] - f[i];
  *l = quant4(f, 16.0f);
}

// x [T, in] into pieces: first ones [T, in], second ones [T, in], then the scale words of
// the first ones [T, blocks], a byte per 32 columns; the second ones' bytes are 4 less
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads)
q4_split_kernel(const __nv_bfloat16 *__restrict__ x, int T, int in, uint8_t *__restrict__ pieces) {
  pdl_trigger();
  const int blocks = (in + kKB - 1) / kKB, c = 4 * static_cast<int>(blockIdx.x * kSplitThreads + threadIdx.x);
  const int64_t all = static_cast<int64_t>(T) * in;
  uint8_t *words = pieces + 2 * all;
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    // a warp holds 128 columns: all of a block's scale bytes, any past the row
    const int64_t at = static_cast<int64_t>(t) * in + c;
    uint32_t h, l, b;
    split4(c < in ? __ldg(reinterpret_cast<const uint2 *>(x + at)) : make_uint2(0, 0), &h, &l, &b);
    if (c < in) {
      *reinterpret_cast<uint32_t *>(pieces + at) = h;
      *reinterpret_cast<uint32_t *>(pieces + all + at) = l;
    }
    if ((threadIdx.x & 7) == 0 && c < blocks * kKB) words[static_cast<int64_t>(t) * blocks * 4 + c / 32] = static_cast<uint8_t>(b);
  }
}

template <int NT, bool BOX>
__global__ void __launch_bounds__(Few<NT>::kThreads, Few<NT>::kPerSm)
q4_few_kernel(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const Q4Params p,
              const __nv_bfloat16 *x, const uint8_t *wq, const uint32_t *xwords) {
  using F = Few<NT>;
  constexpr int S = F::kStages, N = F::N;
  constexpr bool PRE = F::kSplit;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t *wscale = reinterpret_cast<uint32_t *>(smem + S * F::kStage);  // W's scale words, [S][128]
  uint32_t *words = wscale + S * kTcM;                                    // x's, [S][kWords]
  uint64_t *bars = reinterpret_cast<uint64_t *>(words + S * F::kWords);
  // barriers of a stage: W (and pieces), scales (and x), scale words in tensor memory, empty; the result
  const uint32_t wfull0 = smem_u32(bars), sfull0 = wfull0 + 8u * S, xfull0 = sfull0 + 8u * S, empty0 = xfull0 + 8u * S,
                 accf = empty0 + 8u * S;
  SharedCtl *ctl = reinterpret_cast<SharedCtl *>(bars + 4 * S + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // boxes; every thread's copies of W
      mbar_init(wfull0 + 8u * s, (BOX || PRE ? 1 : 0) + (BOX ? 0 : 32 * kCopyWarps));
      // every thread's copies, every warp's plain stores; boxes of x
      mbar_init(sfull0 + 8u * s, 33 * kCopyWarps + (BOX && !PRE ? 1 : 0));
      mbar_init(xfull0 + 8u * s, kQuads);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(accf, 1);
    ctl->abort = 0;
    fence_barrier_init();
    if (BOX) prefetch_map(&mW);
    if (BOX || PRE) prefetch_map(&mX);
  }
  for (int i = threadIdx.x; i < S * F::kWords; i += F::kThreads) words[i] = 0x7f7f7f7fu;
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
  const uint32_t rank = cluster_ctarank();
  // Without pieces the launch before this one may still run: nothing is read or
  // written before it has ended.  With pieces it is q4_split_kernel, which itself
  // started after all launches before it had ended: only what it writes is waited for
  pdl_trigger();
  if (!PRE) pdl_wait();

  Tile o = {};
  const bool work = find_tile(p, static_cast<int>(blockIdx.x / csize), &o);   // all of a cluster alike
  const uint32_t blocks = static_cast<uint32_t>((p.kdim + kKB - 1) / kKB);
  // at least one block: a cluster has no more CTAs than there are
  const int kb0 = static_cast<int>(blocks * rank / csize), kb1 = static_cast<int>(blocks * (rank + 1) / csize);
  const int ntok = o.t1 - o.t0, f0 = o.ft * kTcM;
  bool ok = true;

  if (!work) {
    // no tile for this cluster
  } else if (warp >= F::kCopy) {
    // ---------------------------------------------------------------- copies
    const int i = threadIdx.x - 32 * F::kCopy;
    const bool boxes = warp == F::kCopy;               // this warp issues them
    const int G = p.in / kQ4Group;
    const bool words4 = G % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scale) & 3) == 0;
    // what the boxes of a stage count on wfull: those of W count the bytes that they read
    constexpr uint32_t tx = (BOX ? kWBytes / 2 : 0) + (PRE ? F::kXBytes : 0);
    ok = !loads_withheld(p.guard);
    int ahead = 0;                                     // blocks of W asked for before the pieces
    if (BOX && PRE && ok) {
      ahead = min(S, kb1 - kb0);
      if (boxes && elect_one())
        for (int s = 0; s < ahead; ++s) {
          mbar_expect_tx(wfull0 + 8u * s, tx);
          tma_load_3d(smem_u32(smem) + s * F::kStage, &mW, (kb0 + s) * kKB, f0, o.e, wfull0 + 8u * s);
        }
      __syncwarp();
    }
    if (PRE) pdl_wait();
    Ring st(S);
    for (int kb = kb0; kb < kb1 && ok; ++kb) {
      ok = guard_wait(empty0 + 8u * st.i, st.phase ^ 1u, ctl, p.guard, 71);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t at = smem_u32(smem) + st.i * F::kStage, xs = at + kWBytes;
      const uint32_t wb = wfull0 + 8u * st.i, sb = sfull0 + 8u * st.i;
      if ((BOX || PRE) && boxes && elect_one()) {
        if (kb - kb0 >= ahead) {
          mbar_expect_tx(wb, tx);
          if (BOX) tma_load_3d(at, &mW, kb * kKB, f0, o.e, wb);
        }
        if (PRE) {
          tma_load_2d(xs, &mX, kb * kKB, o.t0, wb);
          tma_load_2d(xs + NT * kKB, &mX, kb * kKB, p.T + o.t0, wb);
        } else {
          // x as it is: the 256 bytes of token t where its two pieces go, rows t and NT + t
          mbar_expect_tx(sb, F::kXBytes);
          tma_load_2d(xs, &mX, kb * kKB, o.t0, sb);
          tma_load_2d(xs + NT * kKB, &mX, kb * kKB + 64, o.t0, sb);
        }
      }
      __syncwarp();
      if (!BOX && !PRE) {
#pragma unroll
        for (int j = 0; j < NT / 4; ++j) {
          const int t = 4 * j + i / 16, d = i % 16, k = kb * kKB + 8 * d;
          const bool has = t < ntok && k < p.in;
          copy16(xs + static_cast<uint32_t>(t + (d >= 8 ? NT : 0)) * 128u + static_cast<uint32_t>(d & 7) * 16u,
                 has ? x + static_cast<int64_t>(o.t0 + t) * p.in + k : x, has ? 16u : 0u);
        }
      }
      if (PRE) {
        const uint32_t to = smem_u32(words + st.i * F::kWords);
        for (int t = i; t < ntok; t += 32 * kCopyWarps)
          copy4(to + 4u * t, xwords + static_cast<int64_t>(o.t0 + t) * blocks + kb, 4u);
      }
      const uint32_t sc = smem_u32(wscale + st.i * kTcM);
#pragma unroll
      for (int j = 0; j < kTcM / (32 * kCopyWarps); ++j) {
        const int f = 32 * kCopyWarps * j + i;
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
      // full when the copies of all these threads have landed and their plain stores
      // are out.  The threads that wait for it order both before the tensor core's
      // reads: a proxy fence here would wait for the copies
      copies_arrive(sb);
      __syncwarp();
      if (lane == 0) mbar_arrive(sb);
      if (!BOX) {
        const int r = i / 8, c = i % 8;                       // first row, piece of 16 values
        const int64_t ld = p.in / 2;
        const uint8_t *src = wq + (static_cast<int64_t>(o.e) * p.out + f0 + r) * ld + kb * (kKB / 2) + 8 * c;
        const uint32_t dst = at + r * 128u + static_cast<uint32_t>((c ^ r) * 16);
        const int live = kb * kKB + 16 * c < p.in ? p.out - f0 - r : 0;      // rows from r that exist
#pragma unroll
        for (int j = 0; j < kTcM / 8; ++j) copy8(dst + j * 1024u, 8 * j < live ? src + 8 * j * ld : wq, 8 * j < live ? 8u : 0u);
        copies_arrive(wb);
      }
      st.next();
    }
    copies_wait();
    if ((BOX || PRE) && !ok && boxes) {
      // boxes in flight, whose barrier may never complete after an abort: they land
      // within microseconds, wait 1 ms
      const unsigned long long c0 = globaltimer();
      while (globaltimer() - c0 < 1000000ull) {
      }
    }
  } else if (warp == F::kMma) {
    // ---------------------------------------------------------------- MMA issuer
    Ring st(S);
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = guard_wait(xfull0 + 8u * st.i, st.phase, ctl, p.guard, 72);
      ok = ok && guard_wait(wfull0 + 8u * st.i, st.phase, ctl, p.guard, 73);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (!BOX) fence_async_proxy();
      tc_fence_after();
      const uint32_t at = smem_u32(smem) + st.i * F::kStage;
      const uint64_t a = sdesc<32>(at), b = sdesc<32>(at + kWBytes);
      const uint32_t sf = tmem + F::kSfCol + F::kSfStride * st.i;
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
    // ---------------------------------------------------------------- scales (and x)
    const int group = warp / kQuads, own = warp % kQuads;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(own) * 32u << 16);
    Ring st(S);
    for (int i = 0; i < group; ++i) st.next();
    for (int kb = kb0 + group; kb < kb1; kb += F::kGroups) {
      ok = guard_wait(sfull0 + 8u * st.i, st.phase, ctl, p.guard, 74);
      if constexpr (!PRE) {
        // a place without a token keeps what it holds: its column of the result is not read
        uint8_t *xs = smem + st.i * F::kStage + kWBytes;
        uint8_t *ws = reinterpret_cast<uint8_t *>(words + st.i * N);
#pragma unroll
        for (int j = 0; j < NT / kQuads; ++j) {
          const int t = own + kQuads * j, at = ((lane >> 2) ^ (t & 7)) * 16 + (lane & 3) * 4;
          if (t >= ntok) break;
          const uint2 raw = *reinterpret_cast<const uint2 *>(xs + (t + (lane >= 16 ? NT : 0)) * 128 + (lane & 15) * 8);
          __syncwarp();
          uint32_t h, l, b;
          split4(raw, &h, &l, &b);
          *reinterpret_cast<uint32_t *>(xs + t * 128 + at) = h;
          *reinterpret_cast<uint32_t *>(xs + (NT + t) * 128 + at) = l;      // NT % 8 == 0: the same swizzle
          if ((lane & 7) == 0) {
            ws[4 * t + (lane >> 3)] = static_cast<uint8_t>(b);
            ws[4 * (NT + t) + (lane >> 3)] = static_cast<uint8_t>(b - 4u);
          }
        }
        fence_async_proxy();
        // all scale words are there; the four warps go on or leave together
        ok = all_of<32 * kQuads>(1 + group, ok);
      } else {
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      uint32_t all[F::kSfStride] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) all[j] = wscale[st.i * kTcM + 32 * j + lane];
#pragma unroll
      for (int j = 0; j < F::kXCols; ++j) {
        const int n = 32 * j + lane;
        if (PRE) all[4 + j] = n < NT ? words[st.i * NT + n] : words[st.i * NT + n - NT] - 0x04040404u;
        else if (n < N) all[4 + j] = words[st.i * N + n];
      }
      tc_fence_after();
      const uint32_t to = lane_addr + F::kSfCol + F::kSfStride * st.i;
      const uint32_t lo[8] = {all[0], all[1], all[2], all[3], all[4], all[5], all[6], all[7]};
      tmem_st8(to, lo);
      if constexpr (F::kSfStride > 8) tmem_st4(to + 8, all[8], all[9], all[10], all[11]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(xfull0 + 8u * st.i);
#pragma unroll
      for (int i = 0; i < F::kGroups; ++i) st.next();
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
      if (c < ntok && (c / 8) % F::kGroups == group) {
        float a[8], b[8];
        tmem_ld<8>(lane_addr + c, a);
        tmem_ld<8>(lane_addr + NT + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) part[(c + i) * kTcM + f] = ok ? a[i] + b[i] : 0.0f;
      }
    }
  }
  // the pieces are written, whoever reads them: no launch after this one comes
  // before the split has ended
  if (PRE) pdl_wait();
  tc_fence_before();
  if (csize > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (work) {
    // the parts of the cluster in rank order, one rounding to bf16: four
    // features a thread, neighbouring threads on neighbouring features
    const int quads = ntok * 32;
    const uint32_t base = smem_u32(smem);
    for (int i = static_cast<int>(rank) * F::kThreads + threadIdx.x; i < quads; i += static_cast<int>(csize) * F::kThreads) {
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
  if (warp == F::kMma) {
    __syncwarp();
    tmem_dealloc(tmem, F::kCols);
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
dora_status launch(const void *x, const void *wq, const Q4Params &p, int cluster, void *workspace, cudaStream_t cs) {
  using F = Few<NT>;
  CUtensorMap mW = {}, mX = {};
  const int64_t all = static_cast<int64_t>(p.T) * p.in;
  uint8_t *pieces = static_cast<uint8_t *>(workspace);
  if (BOX && !map_w4(&mW, wq, p.experts, p.out, p.in)) return DORA_ERR_CUDA;
  if (F::kSplit) {
    if (!map_q8(&mX, pieces, 2 * static_cast<int64_t>(p.T), p.in, NT, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)) return DORA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(dora::ceil_div(p.in, 4 * kSplitThreads)), p.T < 65535 ? p.T : 65535);
    q4_split_kernel<<<grid, kSplitThreads, 0, cs>>>(static_cast<const __nv_bfloat16 *>(x), p.T, p.in, pieces);
    if (dora::launch_status() != DORA_OK) return DORA_ERR_CUDA;
    dora::count_launches(1);
  } else if (BOX && !map_x(&mX, x, p.T, p.in, NT)) {
    return DORA_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles * cluster));
  cfg.blockDim = dim3(F::kThreads);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, q4_few_kernel<NT, BOX>, mW, mX, p, static_cast<const __nv_bfloat16 *>(x),
                         static_cast<const uint8_t *>(wq), reinterpret_cast<const uint32_t *>(pieces + 2 * all)) != cudaSuccess) {
    cudaGetLastError();
    return DORA_ERR_CUDA;
  }
  dora::count_launches(1);
  return DORA_OK;
}

template <int NT>
dora_status launch_few(const void *x, const void *wq, Q4Params p, void *workspace, int sms, cudaStream_t cs) {
  const int64_t groups = p.offsets ? (p.experts < p.T ? p.experts : p.T) : 1;
  const int64_t tiles = p.ftiles * (p.offsets ? p.T / NT + groups : dora::ceil_div(p.T, NT));
  // the k range over as many CTAs as keep all clusters resident
  int cluster = 1;
  const int64_t blocks = dora::ceil_div(p.in, kKB);
  while (cluster < kMaxCluster && tiles * cluster * 2 <= Few<NT>::kPerSm * sms && cluster * 2 <= blocks) cluster *= 2;
  if (tiles * cluster > kMaxDim) return DORA_ERR_SHAPE;
  p.ntok = NT;
  p.tiles = static_cast<int>(tiles);
  // boxes of 4-bit values take whole blocks of 128 and 32-byte rows
  return p.in % kKB == 0 && dora::aligned(wq, 32) ? launch<NT, true>(x, wq, p, cluster, workspace, cs)
                                                  : launch<NT, false>(x, wq, p, cluster, workspace, cs);
}

}  // namespace

namespace dora {

size_t q4_few_workspace(int64_t T, int64_t in, int64_t per) {
  return per <= 8 ? 0 : static_cast<size_t>(2 * T * in + T * 4 * ceil_div(in, kKB));
}

dora_status matmul_q4_few(const void *x, const int32_t *offsets, const void *wq, const void *wscale, int64_t T,
                          int64_t out, int64_t in, int64_t experts, void *y, void *workspace, cudaStream_t cs) {
  DeviceInfo info;
  int device = 0;
  dora_status st = current_device(&info, &device);
  if (st != DORA_OK) return st;
  static const void *const kernels[] = {
      (const void *)q4_few_kernel<8, false>,  (const void *)q4_few_kernel<8, true>,   (const void *)q4_few_kernel<16, false>,
      (const void *)q4_few_kernel<16, true>,  (const void *)q4_few_kernel<32, false>, (const void *)q4_few_kernel<32, true>,
      (const void *)q4_few_kernel<64, false>, (const void *)q4_few_kernel<64, true>,  (const void *)q4_few_kernel<128, false>,
      (const void *)q4_few_kernel<128, true>};
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
  const int64_t per = offsets ? q4_per(T, experts) : T;
  if (per <= 8) return launch_few<8>(x, wq, p, workspace, info.sms, cs);
  if (per <= 16) return launch_few<16>(x, wq, p, workspace, info.sms, cs);
  if (per <= 32) return launch_few<32>(x, wq, p, workspace, info.sms, cs);
  if (per <= 64) return launch_few<64>(x, wq, p, workspace, info.sms, cs);
  return launch_few<128>(x, wq, p, workspace, info.sms, cs);
}

}  // namespace dora
