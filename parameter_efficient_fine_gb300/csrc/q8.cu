// Activations and weights in 8 bits (see q8.cuh for the form), and the compose
// that keeps its backward's input in it, for GB300 (sm_103a).
//
//   dora_q8_store, dora_q8_load   a matrix into the 8-bit form and back
//   dora_compose_fwd_q8           y as dora_compose_fwd; v = base + s lora in 8 bits
//   dora_compose_bwd_q8           d_base, d_lora, d_mag from dy and that v
//
// The compose's backward needs base and lora only as v = base + s lora
// (d_mag = sum_t dy v / n), so the forward, which has both in registers, keeps
// v alone: one byte an element instead of four, and the backward reads it
// instead of both.  v is formed with two fp32 roundings (s lora, then the sum).
//
// Each is one streaming pass bound by HBM bandwidth, in the thread layout of
// compose.cu: a thread holds one 16-byte piece of a row, so a block of 128
// columns is 16 neighbouring threads in bf16 and a whole warp in fp32, and its
// maximum is a butterfly of shuffles over them; the quantised piece is stored
// from the same registers.  At 15360 x 8192, in us and as a fraction of the
// 6800 GB/s of a plain copy (bytes that have to move / time):
//            store       load        forward     backward (with the d_mag sum)
//   bf16    64  0.87    66  0.85    136  0.95    142  0.91
//   f32    101  0.92   109  0.85    248  0.97    269  0.90
// A call on a few rows costs its launch, 5 to 7 us (the backward's two, 10).
// Rows that are ragged or not 16-byte aligned take the same kernels with four
// columns a thread, 32 apart (Piece).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q8.cuh"
#include "stream.cuh"

#include <type_traits>

namespace {

// What a thread holds of a row.  Vector rows: 16 bytes of it, VEC neighbouring
// columns from c0, and the matching 8-bit piece.  Ragged rows (any length and
// alignment): four columns 32 apart, so that a warp's accesses are contiguous
// and a warp is one block of 128 columns.  `live` is how many of the columns
// lie inside the row (all or none in a vector row).
template <typename Act, bool RAGGED> struct Piece;

template <typename Act> struct Piece<Act, false> {
  static constexpr int VEC = 16 / sizeof(Act);
  using IO = Io<Act, VEC>;
  using Raw = typename IO::Raw;
  using Q = typename std::conditional<VEC == 8, uint2, uint32_t>::type;
  static __device__ __forceinline__ int64_t first() { return ((int64_t)blockIdx.x * kBX + threadIdx.x) * VEC; }
  static __device__ __forceinline__ int live(int64_t c0, int64_t cols) { return c0 < cols ? VEC : 0; }
  static __device__ __forceinline__ int at(int v) { return v; }                          // column c0 + at(v)
  static __device__ __forceinline__ int in_block(int v) { return threadIdx.x * VEC + v; }  // among the block's
  static __device__ __forceinline__ Raw load(const Act *p, int64_t e, int n) { return n ? IO::load(p, e) : Raw{}; }
  static __device__ __forceinline__ void store(Act *p, int64_t e, int n, const float (&v)[VEC]) {
    if (n) IO::store(p, e, IO::pack(v));
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[VEC]) { IO::unpack(r, v); }
  static __device__ __forceinline__ Q load_q(const uint8_t *q, int64_t e, int n) {
    return n ? __ldcs(reinterpret_cast<const Q *>(q + e)) : Q{};
  }
  static __device__ __forceinline__ void store_q(uint8_t *q, int64_t e, int n, const float (&v)[VEC], float inv) {
    if (!n) return;
    if constexpr (VEC == 8) __stcs(reinterpret_cast<Q *>(q + e), make_uint2(quant4(v, inv), quant4(v + 4, inv)));
    else __stcs(reinterpret_cast<Q *>(q + e), quant4(v, inv));
  }
  static __device__ __forceinline__ void dequant(Q r, float s, float (&v)[VEC]) {
    uint32_t w[2];
    if constexpr (VEC == 8) {
      w[0] = r.x;
      w[1] = r.y;
    } else {
      w[0] = r;
    }
#pragma unroll
    for (int k = 0; k < VEC; k += 4) dequant4(w[k / 4], s, v + k);
  }
};

template <typename Act> struct Piece<Act, true> {
  static constexpr int VEC = 4;
  using IO = Io<Act, 1>;
  struct Raw {
    typename IO::Raw v[VEC];
  };
  struct Q {
    uint8_t b[VEC];
  };
  static __device__ __forceinline__ int64_t first() { return (int64_t)blockIdx.x * kQBlock + threadIdx.x; }
  static __device__ __forceinline__ int live(int64_t c0, int64_t cols) {
    const int64_t n = (cols - c0 + 31) / 32;
    return n < 0 ? 0 : n > VEC ? VEC : static_cast<int>(n);
  }
  static __device__ __forceinline__ int at(int v) { return 32 * v; }
  static __device__ __forceinline__ int in_block(int v) { return threadIdx.x + 32 * v; }
  static __device__ __forceinline__ Raw load(const Act *p, int64_t e, int n) {
    Raw r = {};
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (k < n) r.v[k] = IO::load(p, e + 32 * k);
    return r;
  }
  static __device__ __forceinline__ void store(Act *p, int64_t e, int n, const float (&v)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float one[1] = {v[k]};
      if (k < n) IO::store(p, e + 32 * k, IO::pack(one));
    }
  }
  static __device__ __forceinline__ void unpack(Raw r, float (&v)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float one[1];
      IO::unpack(r.v[k], one);
      v[k] = one[0];
    }
  }
  static __device__ __forceinline__ Q load_q(const uint8_t *q, int64_t e, int n) {
    Q r = {};
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (k < n) r.b[k] = __ldcs(q + e + 32 * k);
    return r;
  }
  static __device__ __forceinline__ void store_q(uint8_t *q, int64_t e, int n, const float (&v)[VEC], float inv) {
    const uint32_t w = quant4(v, inv);
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (k < n) __stcs(q + e + 32 * k, static_cast<uint8_t>(w >> (8 * k)));
  }
  static __device__ __forceinline__ void dequant(Q r, float s, float (&v)[VEC]) {
    dequant4(r.b[0] | static_cast<uint32_t>(r.b[1]) << 8 | static_cast<uint32_t>(r.b[2]) << 16 |
                 static_cast<uint32_t>(r.b[3]) << 24, s, v);
  }
};

// largest `m` over the 128 / VEC neighbouring threads that hold a 128-column
// block.  All threads of the warp call it
template <int VEC>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
  for (int o = 64 / VEC; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// scale byte of the 128-column block that this thread's VEC values are part
// of; one past the row's end passes zeros.  The maximum passes over NaNs but
// not over infinities: a warp that meets one takes the maximum again without
// them and turns them into NaNs
template <int VEC>
__device__ __forceinline__ uint32_t block_scale(float (&v)[VEC]) {
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < VEC; ++k) top = fmaxf(top, fabsf(v[k]));
  uint32_t m = block_max<VEC>(__float_as_uint(top));
  if (__any_sync(0xffffffffu, m == kInfBits)) [[unlikely]] {
    m = 0;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      m = max(m, finite_bits(v[k]));
      v[k] = inf_to_nan(v[k]);
    }
    m = block_max<VEC>(m);
  }
  return scale_byte(m);
}

// ---------------------------------------------------------------------------
// store, and the compose forward that stores v
// ---------------------------------------------------------------------------
// COMPOSE: y = base + ((g-1) base + g s lora) and the 8-bit form of base + s
// lora; otherwise the 8-bit form of base alone
template <typename Act, bool RAGGED, bool COMPOSE>
__global__ void __launch_bounds__(kThreads)
q8_fwd_kernel(const Act *__restrict__ base, const Act *__restrict__ lora, const float *__restrict__ g, float s,
              int64_t T, int64_t out, Act *__restrict__ y, uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
  using P = Piece<Act, RAGGED>;
  constexpr int VEC = P::VEC;
  // token rows in flight per thread (15360 x 8192 bf16: store 66, 62, 63, 68 us
  // and compose 150, 137, 141, 146 us with 2, 3, 4 and 8; f32: compose 243, 267,
  // 264 us with 1, 2 and 3; 15360 x 8191 bf16: store 94, 128, 128 us and compose
  // 225, 219, 214 us with 1, 2 and 3)
  constexpr int U = RAGGED || (COMPOSE && VEC == 4) ? 1 : 3;
  const int64_t c0 = P::first();
  const int live = P::live(c0, out);   // a thread past the row's end takes part in the maxima, with zeros
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;

  float gm1[VEC], gs[VEC];
  if (COMPOSE) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float gv = v < live ? __ldg(g + c0 + P::at(v)) : 0.0f;
      gm1[v] = gv - 1.0f;
      gs[v] = gv * s;
    }
  }
  for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
    typename P::Raw rb[U], rl[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      const int n = tu < T ? live : 0;
      rb[u] = P::load(base, tu * out + c0, n);
      if (COMPOSE) rl[u] = P::load(lora, tu * out + c0, n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      const int n = tu < T ? live : 0;
      float b[VEC], v[VEC];
      P::unpack(rb[u], b);
      if (COMPOSE) {
        float l[VEC];
        P::unpack(rl[u], l);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          v[k] = __fadd_rn(b[k], __fmul_rn(s, l[k]));
          b[k] = b[k] + fmaf(gm1[k], b[k], gs[k] * l[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = b[k];
      }
      const uint32_t sc = block_scale<VEC>(v);
      if (COMPOSE) P::store(y, tu * out + c0, n, b);
      P::store_q(q, tu * out + c0, n, v, scale_inverse(sc));
      if (n > 0 && c0 % kQBlock == 0) scale[tu * nsc + c0 / kQBlock] = static_cast<uint8_t>(sc);
    }
  }
}

// a 128 x 128 block with one scale per thread block (a frozen weight, once),
// held in registers between its maximum and its bytes: one read of x
template <typename Act, bool RAGGED>
__global__ void __launch_bounds__(kThreads)
q8_store_tile_kernel(const Act *__restrict__ x, int64_t rows, int64_t cols, uint8_t *__restrict__ q,
                     uint8_t *__restrict__ scale) {
  using P = Piece<Act, RAGGED>;
  constexpr int kAcross = kQBlock / P::VEC, kDown = kThreads / kAcross, kPasses = kQBlock / kDown;
  __shared__ uint32_t wmax[kThreads / 32];
  const int64_t nsc = (cols + kQBlock - 1) / kQBlock;
  const int tid = threadIdx.x, at = tid % kAcross;
  const int64_t c0 = (int64_t)(blockIdx.x % nsc) * kQBlock + (RAGGED ? at : at * P::VEC);
  const int64_t r0 = (int64_t)(blockIdx.x / nsc) * kQBlock + tid / kAcross;
  const int live = P::live(c0, cols);
  // past the last row the last row again, and past the row's end its first
  // piece, which change no maximum.  Loads without conditions all go out at
  // once (8192 x 8192 f32: 69 us, 4870 GB/s; 147 us with a condition on each)
  const int64_t from = live > 0 ? c0 : c0 - at * (RAGGED ? 1 : P::VEC);
  const int load_live = RAGGED && live > 0 ? live : RAGGED ? 1 : P::VEC;
  typename P::Raw raw[kPasses];
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int64_t r = r0 + k * kDown;
    raw[k] = P::load(x, (r < rows ? r : rows - 1) * cols + from, load_live);
  }
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    float v[P::VEC];
    P::unpack(raw[k], v);
#pragma unroll
    for (int i = 0; i < P::VEC; ++i) m = max(m, finite_bits(v[i]));
  }
  m = block_max<4>(m);               // of the warp
  if (tid % 32 == 0) wmax[tid / 32] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) m = max(m, wmax[k]);
  const uint32_t sc = scale_byte(m);
  const float inv = scale_inverse(sc);
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int64_t r = r0 + k * kDown;
    float v[P::VEC];
    P::unpack(raw[k], v);
#pragma unroll
    for (int i = 0; i < P::VEC; ++i) v[i] = inf_to_nan(v[i]);
    P::store_q(q, r * cols + c0, r < rows ? live : 0, v, inv);
  }
  if (tid == 0) scale[blockIdx.x] = static_cast<uint8_t>(sc);
}

// ---------------------------------------------------------------------------
// load
// ---------------------------------------------------------------------------
// eight blocks an SM: what limits it is how much it has in flight (15360 x 8192
// f32 127 us with the seven that its registers would leave, 110 with eight;
// 15360 x 8191 bf16 117 and 99; 15360 x 8192 bf16 66 with either, 5730 GB/s)
template <typename Act, bool RAGGED>
__global__ void __launch_bounds__(kThreads, 8)
q8_load_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t T, int64_t out, int block_rows,
               Act *__restrict__ x) {
  using P = Piece<Act, RAGGED>;
  // bf16, 15360 x 8192: 72, 66, 73, 85 us with 1, 2, 4 and 8; 15360 x 8191: 117, 137, 161 us with 1, 2 and 3 (at seven)
  constexpr int U = RAGGED ? 1 : 2;
  const int64_t c0 = P::first();
  const int live = P::live(c0, out);
  if (live == 0) return;
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;
  const uint8_t *sp = scale + c0 / kQBlock;
  for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
    typename P::Q r[U];
    uint32_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      r[u] = typename P::Q{};
      sc[u] = 0;
      if (tu < T) {
        r[u] = P::load_q(q, tu * out + c0, live);
        sc[u] = __ldg(sp + (block_rows == 1 ? tu : tu / block_rows) * nsc);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      if (tu < T) {
        float v[P::VEC];
        P::dequant(r[u], scale_value(sc[u]), v);
        P::store(x, tu * out + c0, live, v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// compose backward from the 8-bit v
// ---------------------------------------------------------------------------
template <typename Act, bool RAGGED>
__global__ void __launch_bounds__(kThreads)
q8_compose_bwd_kernel(const Act *__restrict__ dy, const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale,
                      const float *__restrict__ g, float s, int64_t T, int64_t out, Act *__restrict__ d_base,
                      Act *__restrict__ d_lora, float *__restrict__ part) {
  using P = Piece<Act, RAGGED>;
  constexpr int VEC = P::VEC;
  // 15360 x 8192 bf16: 147 us with 2, more with 1, 3 and 4; 15360 x 8191: 236, 240, 209, 280 us with 1, 2, 3 and 4
  constexpr int U = RAGGED ? 3 : 2;
  __shared__ float red[kBY][kBX * VEC];

  const int64_t c0 = P::first();
  const int live = P::live(c0, out);
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;

  float acc[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) acc[v] = 0.0f;

  if (live > 0) {
    float gg[VEC], gs[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      gg[v] = v < live ? __ldg(g + c0 + P::at(v)) : 0.0f;
      gs[v] = gg[v] * s;
    }
    for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
      typename P::Raw rd[U];
      typename P::Q rq[U];
      uint32_t sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tu = t + u * lanes, e = tu * out + c0;
        const int n = tu < T ? live : 0;
        rd[u] = P::load(dy, e, n);
        rq[u] = P::load_q(q, e, n);
        sc[u] = n ? __ldg(scale + tu * nsc + c0 / kQBlock) : 0u;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tu = t + u * lanes, e = tu * out + c0;
        const int n = tu < T ? live : 0;
        float d[VEC], v[VEC], ob[VEC], ol[VEC];
        P::unpack(rd[u], d);
        P::dequant(rq[u], scale_value(sc[u]), v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          ob[k] = gg[k] * d[k];
          ol[k] = gs[k] * d[k];
          acc[k] = fmaf(d[k], v[k], acc[k]);     // zeros past the last row
        }
        P::store(d_base, e, n, ob);
        P::store(d_lora, e, n, ol);
      }
    }
  }

  // fixed-order sum of the 8 token lanes of this block
#pragma unroll
  for (int v = 0; v < VEC; ++v) red[threadIdx.y][P::in_block(v)] = acc[v];
  __syncthreads();
  if (threadIdx.y == 0) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (v >= live) break;
      float sum = red[0][P::in_block(v)];
#pragma unroll
      for (int k = 1; k < kBY; ++k) sum += red[k][P::in_block(v)];
      part[(int64_t)blockIdx.y * out + c0 + P::at(v)] = sum;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// 16-byte pieces of the rows of `act` and the matching pieces of their 8-bit form
template <typename Act>
bool q8_vector_ok(int64_t cols, std::initializer_list<const void *> ptrs, const void *q) {
  return vector_ok<Act>(cols, ptrs) && dora::aligned(q, 16 / sizeof(Act));
}

// grid of a kernel of Piece<Act, RAGGED> rows: its blocks hold 32 pieces a row
template <typename Act, bool RAGGED, auto *KERNEL>
Grid plan_rows(int64_t T, int64_t out, int device, int sms) {
  return plan_grid(T, RAGGED ? dora::ceil_div(out, kQBlock) * kBX : out / Piece<Act, RAGGED>::VEC,
                   (int64_t)sms * resident_blocks<KERNEL>(device));
}

template <typename Act, bool RAGGED, bool COMPOSE>
dora_status launch_q8_fwd(const void *base, const void *lora, const float *g, float s, int64_t T, int64_t out, void *y,
                          void *q, void *scale, cudaStream_t stream, int device, int sms) {
  constexpr auto kern = &q8_fwd_kernel<Act, RAGGED, COMPOSE>;
  const Grid gr = plan_rows<Act, RAGGED, kern>(T, out, device, sms);
  kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(
      static_cast<const Act *>(base), static_cast<const Act *>(lora), g, s, T, out, static_cast<Act *>(y),
      static_cast<uint8_t *>(q), static_cast<uint8_t *>(scale));
  dora::count_launches(1);
  return dora::launch_status();
}
template <typename Act, bool COMPOSE>
dora_status run_q8_fwd(const void *base, const void *lora, const float *g, float s, int64_t T, int64_t out, void *y,
                       void *q, void *scale, cudaStream_t stream, int device, int sms) {
  const bool vec = COMPOSE ? q8_vector_ok<Act>(out, {base, lora, y}, q) : q8_vector_ok<Act>(out, {base}, q);
  return vec ? launch_q8_fwd<Act, false, COMPOSE>(base, lora, g, s, T, out, y, q, scale, stream, device, sms)
             : launch_q8_fwd<Act, true, COMPOSE>(base, lora, g, s, T, out, y, q, scale, stream, device, sms);
}

template <typename Act>
dora_status run_q8_store_tile(const void *x, int64_t rows, int64_t cols, int64_t tiles, void *q, void *scale,
                              cudaStream_t stream) {
  const auto kern = q8_vector_ok<Act>(cols, {x}, q) ? &q8_store_tile_kernel<Act, false> : &q8_store_tile_kernel<Act, true>;
  kern<<<(unsigned)tiles, kThreads, 0, stream>>>(static_cast<const Act *>(x), rows, cols, static_cast<uint8_t *>(q),
                                                 static_cast<uint8_t *>(scale));
  dora::count_launches(1);
  return dora::launch_status();
}

template <typename Act, bool RAGGED>
dora_status launch_q8_load(const void *q, const void *scale, int64_t T, int64_t out, int block_rows, void *x,
                           cudaStream_t stream, int device, int sms) {
  constexpr auto kern = &q8_load_kernel<Act, RAGGED>;
  const Grid gr = plan_rows<Act, RAGGED, kern>(T, out, device, sms);
  kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(
      static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(scale), T, out, block_rows, static_cast<Act *>(x));
  dora::count_launches(1);
  return dora::launch_status();
}
template <typename Act>
dora_status run_q8_load(const void *q, const void *scale, int64_t T, int64_t out, int block_rows, void *x,
                        cudaStream_t stream, int device, int sms) {
  return q8_vector_ok<Act>(out, {x}, q)
             ? launch_q8_load<Act, false>(q, scale, T, out, block_rows, x, stream, device, sms)
             : launch_q8_load<Act, true>(q, scale, T, out, block_rows, x, stream, device, sms);
}

template <typename Act, bool RAGGED>
dora_status launch_q8_bwd(const void *dy, const void *q, const void *scale, const float *g, const float *norm, float s,
                          int64_t T, int64_t out, void *d_base, void *d_lora, float *d_mag, float *part,
                          size_t part_bytes, cudaStream_t stream, int device, int sms) {
  constexpr auto kern = &q8_compose_bwd_kernel<Act, RAGGED>;
  int64_t rows = 0;
  if (T > 0) {
    const Grid gr = plan_rows<Act, RAGGED, kern>(T, out, device, sms);
    rows = gr.gy;
    if ((size_t)rows * (size_t)out * sizeof(float) > part_bytes) return DORA_ERR_WORKSPACE;
    kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(
        static_cast<const Act *>(dy), static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(scale), g, s, T,
        out, static_cast<Act *>(d_base), static_cast<Act *>(d_lora), part);
    dora::count_launches(1);
    if (cudaGetLastError() != cudaSuccess) return DORA_ERR_CUDA;
  }
  dmag_reduce_kernel<<<(unsigned)dora::ceil_div(out, 256), 256, 0, stream>>>(part, rows, out, norm, d_mag);
  dora::count_launches(1);
  return dora::launch_status();
}

constexpr int64_t kMaxDim = (1ll << 31) - 1;
bool bad_size(int64_t rows, int64_t cols) { return rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim; }
size_t elem_size(dora_dtype act) { return act == DORA_F32 ? 4 : 2; }

}  // namespace

extern "C" dora_status dora_q8_store(dora_dtype act, const void *x, int64_t rows, int64_t cols, int block_rows, void *q,
                                     void *scale, dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_size(rows, cols) || (block_rows != 1 && block_rows != kQBlock)) return DORA_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DORA_OK;
  if (!x || !q || !scale) return DORA_ERR_NULL;
  if (!dora::aligned(x, elem_size(act))) return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (block_rows == 1)
    return act == DORA_BF16 ? run_q8_fwd<__nv_bfloat16, false>(x, nullptr, nullptr, 0.0f, rows, cols, nullptr, q,
                                                               scale, cs, device, info.sms)
                            : run_q8_fwd<float, false>(x, nullptr, nullptr, 0.0f, rows, cols, nullptr, q, scale, cs,
                                                       device, info.sms);
  const int64_t tiles = dora::ceil_div(rows, kQBlock) * dora::ceil_div(cols, kQBlock);
  if (tiles > kMaxDim) return DORA_ERR_SHAPE;
  return act == DORA_BF16 ? run_q8_store_tile<__nv_bfloat16>(x, rows, cols, tiles, q, scale, cs)
                          : run_q8_store_tile<float>(x, rows, cols, tiles, q, scale, cs);
}

extern "C" dora_status dora_q8_load(dora_dtype act, const void *q, const void *scale, int64_t rows, int64_t cols,
                                    int block_rows, void *x, dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_size(rows, cols) || (block_rows != 1 && block_rows != kQBlock)) return DORA_ERR_SHAPE;
  if (rows == 0 || cols == 0) return DORA_OK;
  if (!q || !scale || !x) return DORA_ERR_NULL;
  if (!dora::aligned(x, elem_size(act))) return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return act == DORA_BF16 ? run_q8_load<__nv_bfloat16>(q, scale, rows, cols, block_rows, x, cs, device, info.sms)
                          : run_q8_load<float>(q, scale, rows, cols, block_rows, x, cs, device, info.sms);
}

extern "C" dora_status dora_compose_fwd_q8(dora_dtype act, const void *base, const void *lora, const float *g, float s,
                                           int64_t T, int64_t out, void *y, void *q, void *scale,
                                           dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_size(T, out)) return DORA_ERR_SHAPE;
  if (T == 0 || out == 0) return DORA_OK;
  if (!base || !lora || !g || !y || !q || !scale) return DORA_ERR_NULL;
  const size_t esz = elem_size(act);
  if (!dora::aligned(base, esz) || !dora::aligned(lora, esz) || !dora::aligned(y, esz) || !dora::aligned(g, 4))
    return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return act == DORA_BF16
             ? run_q8_fwd<__nv_bfloat16, true>(base, lora, g, s, T, out, y, q, scale, cs, device, info.sms)
             : run_q8_fwd<float, true>(base, lora, g, s, T, out, y, q, scale, cs, device, info.sms);
}

extern "C" size_t dora_compose_bwd_q8_workspace(int64_t T, int64_t out) {
  if (bad_size(T, out) || out == 0) return 0;
  if (T == 0) return 256;
  return (size_t)bwd_rows_bound(T, out) * (size_t)out * sizeof(float);
}

extern "C" dora_status dora_compose_bwd_q8(dora_dtype act, const void *grad_out, const void *q, const void *scale,
                                           const float *g, const float *norm, float s, int64_t T, int64_t out,
                                           void *d_base, void *d_lora, float *d_mag, void *workspace,
                                           size_t workspace_bytes, dora_stream_t stream) {
  if (!valid_dtype(act)) return DORA_ERR_DTYPE;
  if (bad_size(T, out)) return DORA_ERR_SHAPE;
  if (out == 0) return DORA_OK;
  if (!g || !norm || !d_mag) return DORA_ERR_NULL;
  if (T > 0 && (!grad_out || !q || !scale || !d_base || !d_lora)) return DORA_ERR_NULL;
  if (!workspace) return DORA_ERR_WORKSPACE;
  if (!dora::aligned(workspace, 256) || workspace_bytes < dora_compose_bwd_q8_workspace(T, out))
    return DORA_ERR_WORKSPACE;
  const size_t esz = elem_size(act);
  if (T > 0 && (!dora::aligned(grad_out, esz) || !dora::aligned(d_base, esz) || !dora::aligned(d_lora, esz)))
    return DORA_ERR_ALIGN;
  if (!dora::aligned(g, 4) || !dora::aligned(norm, 4) || !dora::aligned(d_mag, 4)) return DORA_ERR_ALIGN;
  dora::DeviceInfo info;
  int device = 0;
  dora_status st = dora::current_device(&info, &device);
  if (st != DORA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  float *part = static_cast<float *>(workspace);
  auto run = act == DORA_BF16
                 ? (q8_vector_ok<__nv_bfloat16>(out, {grad_out, d_base, d_lora}, q) ? &launch_q8_bwd<__nv_bfloat16, false>
                                                                                    : &launch_q8_bwd<__nv_bfloat16, true>)
                 : (q8_vector_ok<float>(out, {grad_out, d_base, d_lora}, q) ? &launch_q8_bwd<float, false>
                                                                            : &launch_q8_bwd<float, true>);
  return run(grad_out, q, scale, g, norm, s, T, out, d_base, d_lora, d_mag, part, workspace_bytes, cs, device, info.sms);
}
