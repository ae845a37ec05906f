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
// from the same registers.  Rows that are ragged or not 16-byte aligned take
// a kernel whose warps own one block of 128 columns each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "q8.cuh"
#include "stream.cuh"

namespace {

// the 8-bit piece of VEC elements
template <int VEC> struct QPiece;
template <> struct QPiece<8> {
  using Raw = uint2;
  static __device__ __forceinline__ Raw quant(const float (&v)[8], float inv) {
    return make_uint2(quant4(v, inv), quant4(v + 4, inv));
  }
  static __device__ __forceinline__ void dequant(Raw r, float s, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.x >> 16, r.y, r.y >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = dequant2(w[k] & 0xffffu, s);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
};
template <> struct QPiece<4> {
  using Raw = uint32_t;
  static __device__ __forceinline__ Raw quant(const float (&v)[4], float inv) { return quant4(v, inv); }
  static __device__ __forceinline__ void dequant(Raw r, float s, float (&v)[4]) {
    const float2 a = dequant2(r & 0xffffu, s), b = dequant2(r >> 16, s);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  }
};
template <> struct QPiece<1> {
  using Raw = uint8_t;
  static __device__ __forceinline__ void dequant(Raw r, float s, float (&v)[1]) { v[0] = dequant2(r, s).x; }
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
template <typename Act, int VEC, bool COMPOSE>
__global__ void __launch_bounds__(kThreads)
q8_fwd_kernel(const Act *__restrict__ base, const Act *__restrict__ lora, const float *__restrict__ g, float s,
              int64_t T, int64_t out, Act *__restrict__ y, uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
  using IO = Io<Act, VEC>;
  using QP = QPiece<VEC>;
  // token rows in flight per thread (15360 x 8192 bf16: store 66, 62, 63, 68 us
  // and compose 150, 137, 141, 146 us with 2, 3, 4 and 8)
  constexpr int U = 3;
  constexpr int kPer = kQBlock / VEC;   // threads per scale
  const int64_t ncg = out / VEC;
  const int64_t cg = (int64_t)blockIdx.x * kBX + threadIdx.x;
  const bool active = cg < ncg;      // an idle thread of a ragged row's last warp takes part in the maxima
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t c0 = active ? cg * VEC : 0;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;

  float gm1[VEC], gs[VEC];
  if (COMPOSE) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float gv = __ldg(g + c0 + v);
      gm1[v] = gv - 1.0f;
      gs[v] = gv * s;
    }
  }
  for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
    typename IO::Raw rb[U], rl[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      rb[u] = typename IO::Raw{};
      if (COMPOSE) rl[u] = typename IO::Raw{};
      if (active && tu < T) {
        rb[u] = IO::load(base, tu * out + c0);
        if (COMPOSE) rl[u] = IO::load(lora, tu * out + c0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      float b[VEC], v[VEC];
      IO::unpack(rb[u], b);
      if (COMPOSE) {
        float l[VEC];
        IO::unpack(rl[u], l);
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
      if (active && tu < T) {
        if (COMPOSE) IO::store(y, tu * out + c0, IO::pack(b));
        __stcs(reinterpret_cast<typename QP::Raw *>(q + tu * out + c0), QP::quant(v, scale_inverse(sc)));
        if (cg % kPer == 0) scale[tu * nsc + cg / kPer] = static_cast<uint8_t>(sc);
      }
    }
  }
}

// the same for any row length and alignment: a warp takes block blockIdx.x *
// warps + warp of rows blockIdx.y, blockIdx.y + gridDim.y, ..., four columns a
// lane, 32 apart
template <typename Act, bool COMPOSE>
__global__ void __launch_bounds__(kThreads)
q8_fwd_ragged_kernel(const Act *__restrict__ base, const Act *__restrict__ lora, const float *__restrict__ g, float s,
                     int64_t T, int64_t out, Act *__restrict__ y, uint8_t *__restrict__ q,
                     uint8_t *__restrict__ scale) {
  using IO = Io<Act, 1>;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;
  const int64_t blk = (int64_t)blockIdx.x * kBY + threadIdx.y;
  if (blk >= nsc) return;            // a whole warp
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    float v[4], yv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = blk * kQBlock + 32 * k + threadIdx.x;
      v[k] = yv[k] = 0.0f;
      if (c < out) {
        float b[1], l[1];
        IO::unpack(IO::load(base, t * out + c), b);
        v[k] = b[0];
        if (COMPOSE) {
          IO::unpack(IO::load(lora, t * out + c), l);
          const float gv = __ldg(g + c);
          v[k] = __fadd_rn(b[0], __fmul_rn(s, l[0]));
          yv[k] = b[0] + fmaf(gv - 1.0f, b[0], gv * s * l[0]);
        }
      }
    }
    uint32_t m = max(max(finite_bits(v[0]), finite_bits(v[1])), max(finite_bits(v[2]), finite_bits(v[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t sc = scale_byte(m);
    const float inv = scale_inverse(sc);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = blk * kQBlock + 32 * k + threadIdx.x;
      if (c < out) {
        q[t * out + c] = static_cast<uint8_t>(quant2(inf_to_nan(v[k]), 0.0f, inv));
        const float yk[1] = {yv[k]};
        if (COMPOSE) IO::store(y, t * out + c, IO::pack(yk));
      }
    }
    if (threadIdx.x == 0) scale[t * nsc + blk] = static_cast<uint8_t>(sc);
  }
}

// a 128 x 128 block with one scale per thread block (a frozen weight, once)
template <typename Act>
__global__ void __launch_bounds__(kThreads)
q8_store_tile_kernel(const Act *__restrict__ x, int64_t rows, int64_t cols, uint8_t *__restrict__ q,
                     uint8_t *__restrict__ scale) {
  using IO = Io<Act, 1>;
  __shared__ uint32_t wmax[kBY];
  const int64_t nsc = (cols + kQBlock - 1) / kQBlock;
  const int64_t r0 = (int64_t)(blockIdx.x / nsc) * kQBlock, c0 = (int64_t)(blockIdx.x % nsc) * kQBlock;
  uint32_t m = 0;
  for (int64_t r = r0 + threadIdx.y; r < min(r0 + kQBlock, rows); r += kBY)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = c0 + 32 * k + threadIdx.x;
      float v[1] = {0.0f};
      if (c < cols) IO::unpack(IO::load(x, r * cols + c), v);
      m = max(m, finite_bits(v[0]));
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (threadIdx.x == 0) wmax[threadIdx.y] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kBY; ++k) m = max(m, wmax[k]);
  const uint32_t sc = scale_byte(m);
  const float inv = scale_inverse(sc);
  for (int64_t r = r0 + threadIdx.y; r < min(r0 + kQBlock, rows); r += kBY)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = c0 + 32 * k + threadIdx.x;
      if (c < cols) {
        float v[1];
        IO::unpack(IO::load(x, r * cols + c), v);
        q[r * cols + c] = static_cast<uint8_t>(quant2(inf_to_nan(v[0]), 0.0f, inv));
      }
    }
  if (threadIdx.x == 0 && threadIdx.y == 0) scale[blockIdx.x] = static_cast<uint8_t>(sc);
}

// ---------------------------------------------------------------------------
// load
// ---------------------------------------------------------------------------
template <typename Act, int VEC>
__global__ void __launch_bounds__(kThreads)
q8_load_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, int64_t T, int64_t out, int block_rows,
               Act *__restrict__ x) {
  using IO = Io<Act, VEC>;
  using QP = QPiece<VEC>;
  constexpr int U = 2;   // 15360 x 8192 bf16: 65, 65, 73, 85 us with 1, 2, 4 and 8
  const int64_t cg = (int64_t)blockIdx.x * kBX + threadIdx.x;
  if (cg >= out / VEC) return;
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t c0 = cg * VEC;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;
  const uint8_t *sp = scale + c0 / kQBlock;
  for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
    typename QP::Raw r[U];
    uint32_t sc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      r[u] = typename QP::Raw{};
      sc[u] = 0;
      if (tu < T) {
        r[u] = __ldcs(reinterpret_cast<const typename QP::Raw *>(q + tu * out + c0));
        sc[u] = __ldg(sp + (block_rows == 1 ? tu : tu / block_rows) * nsc);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tu = t + u * lanes;
      if (tu < T) {
        float v[VEC];
        QP::dequant(r[u], scale_value(sc[u]), v);
        IO::store(x, tu * out + c0, IO::pack(v));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// compose backward from the 8-bit v
// ---------------------------------------------------------------------------
template <typename Act, int VEC>
__global__ void __launch_bounds__(kThreads)
q8_compose_bwd_kernel(const Act *__restrict__ dy, const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale,
                      const float *__restrict__ g, float s, int64_t T, int64_t out, Act *__restrict__ d_base,
                      Act *__restrict__ d_lora, float *__restrict__ part) {
  using IO = Io<Act, VEC>;
  using QP = QPiece<VEC>;
  constexpr int U = 2;
  __shared__ float red[kBY][kBX * VEC];

  const int64_t ncg = out / VEC;
  const int64_t cg = (int64_t)blockIdx.x * kBX + threadIdx.x;
  const bool active = cg < ncg;
  const int64_t lanes = (int64_t)gridDim.y * kBY;
  const int64_t c0 = cg * VEC;
  const int64_t nsc = (out + kQBlock - 1) / kQBlock;

  float acc[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) acc[v] = 0.0f;

  if (active) {
    float gg[VEC], gs[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      gg[v] = __ldg(g + c0 + v);
      gs[v] = gg[v] * s;
    }
    for (int64_t t = (int64_t)blockIdx.y * kBY + threadIdx.y; t < T; t += U * lanes) {
      typename IO::Raw rd[U];
      typename QP::Raw rq[U];
      uint32_t sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tu = t + u * lanes;
        rd[u] = typename IO::Raw{};
        rq[u] = typename QP::Raw{};
        sc[u] = 0;
        if (tu < T) {
          rd[u] = IO::load(dy, tu * out + c0);
          rq[u] = __ldcs(reinterpret_cast<const typename QP::Raw *>(q + tu * out + c0));
          sc[u] = __ldg(scale + tu * nsc + c0 / kQBlock);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tu = t + u * lanes;
        if (tu < T) {
          float d[VEC], v[VEC], ob[VEC], ol[VEC];
          IO::unpack(rd[u], d);
          QP::dequant(rq[u], scale_value(sc[u]), v);
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            ob[k] = gg[k] * d[k];
            ol[k] = gs[k] * d[k];
            acc[k] = fmaf(d[k], v[k], acc[k]);
          }
          const int64_t e = tu * out + c0;
          IO::store(d_base, e, IO::pack(ob));
          IO::store(d_lora, e, IO::pack(ol));
        }
      }
    }
  }

  // fixed-order sum of the 8 token lanes of this block
#pragma unroll
  for (int v = 0; v < VEC; ++v) red[threadIdx.y][threadIdx.x * VEC + v] = acc[v];
  __syncthreads();
  if (threadIdx.y == 0 && active) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float sum = red[0][threadIdx.x * VEC + v];
#pragma unroll
      for (int k = 1; k < kBY; ++k) sum += red[k][threadIdx.x * VEC + v];
      part[(int64_t)blockIdx.y * out + c0 + v] = sum;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// resident blocks per SM of one kernel (each kernel has its own cache)
template <auto *KERNEL>
int resident_blocks(int device) {
  static std::mutex mu;
  static int cache[64] = {};
  if (device < 0 || device >= 64) return 1;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[device] == 0) {
    int b = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, KERNEL, kThreads, 0) != cudaSuccess || b <= 0) b = 1;
    cache[device] = b;
  }
  return cache[device];
}

// 16-byte pieces of the rows of `act` and the matching pieces of their 8-bit form
template <typename Act>
bool q8_vector_ok(int64_t cols, std::initializer_list<const void *> ptrs, const void *q) {
  return vector_ok<Act>(cols, ptrs) && dora::aligned(q, 16 / sizeof(Act));
}

template <typename Act, bool COMPOSE>
dora_status launch_q8_fwd(const void *base, const void *lora, const float *g, float s, int64_t T, int64_t out, void *y,
                          void *q, void *scale, cudaStream_t stream, int device, int sms) {
  constexpr int VEC = 16 / sizeof(Act);
  const Act *b = static_cast<const Act *>(base), *l = static_cast<const Act *>(lora);
  Act *yo = static_cast<Act *>(y);
  uint8_t *qo = static_cast<uint8_t *>(q), *so = static_cast<uint8_t *>(scale);
  const bool vec = COMPOSE ? q8_vector_ok<Act>(out, {base, lora, y}, q) : q8_vector_ok<Act>(out, {base}, q);
  if (vec) {
    constexpr auto kern = &q8_fwd_kernel<Act, VEC, COMPOSE>;
    const Grid gr = plan_grid(T, out / VEC, (int64_t)sms * resident_blocks<kern>(device));
    kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(b, l, g, s, T, out, yo, qo, so);
  } else {
    const int64_t gx = dora::ceil_div(dora::ceil_div(out, kQBlock), kBY);
    const unsigned gy = (unsigned)(T < 65535 ? T : 65535);
    q8_fwd_ragged_kernel<Act, COMPOSE>
        <<<dim3((unsigned)gx, gy), dim3(kBX, kBY), 0, stream>>>(b, l, g, s, T, out, yo, qo, so);
  }
  dora::count_launches(1);
  return dora::launch_status();
}

template <typename Act>
dora_status launch_q8_load(const void *q, const void *scale, int64_t T, int64_t out, int block_rows, void *x,
                           cudaStream_t stream, int device, int sms) {
  constexpr int VEC = 16 / sizeof(Act);
  const uint8_t *qi = static_cast<const uint8_t *>(q), *si = static_cast<const uint8_t *>(scale);
  Act *xo = static_cast<Act *>(x);
  if (q8_vector_ok<Act>(out, {x}, q)) {
    constexpr auto kern = &q8_load_kernel<Act, VEC>;
    const Grid gr = plan_grid(T, out / VEC, (int64_t)sms * resident_blocks<kern>(device));
    kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(qi, si, T, out, block_rows, xo);
  } else {
    constexpr auto kern = &q8_load_kernel<Act, 1>;
    const Grid gr = plan_grid(T, out, (int64_t)sms * resident_blocks<kern>(device));
    kern<<<dim3((unsigned)gr.gx, (unsigned)gr.gy), dim3(kBX, kBY), 0, stream>>>(qi, si, T, out, block_rows, xo);
  }
  dora::count_launches(1);
  return dora::launch_status();
}

template <typename Act, int VEC>
dora_status launch_q8_bwd(const void *dy, const void *q, const void *scale, const float *g, const float *norm, float s,
                          int64_t T, int64_t out, void *d_base, void *d_lora, float *d_mag, float *part,
                          size_t part_bytes, cudaStream_t stream, int device, int sms) {
  constexpr auto kern = &q8_compose_bwd_kernel<Act, VEC>;
  int64_t rows = 0;
  if (T > 0) {
    const Grid gr = plan_grid(T, out / VEC, (int64_t)sms * resident_blocks<kern>(device));
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
    return act == DORA_BF16 ? launch_q8_fwd<__nv_bfloat16, false>(x, nullptr, nullptr, 0.0f, rows, cols, nullptr, q,
                                                                  scale, cs, device, info.sms)
                            : launch_q8_fwd<float, false>(x, nullptr, nullptr, 0.0f, rows, cols, nullptr, q, scale, cs,
                                                          device, info.sms);
  const int64_t tiles = dora::ceil_div(rows, kQBlock) * dora::ceil_div(cols, kQBlock);
  if (tiles > kMaxDim) return DORA_ERR_SHAPE;
  uint8_t *qo = static_cast<uint8_t *>(q), *so = static_cast<uint8_t *>(scale);
  if (act == DORA_BF16)
    q8_store_tile_kernel<__nv_bfloat16><<<(unsigned)tiles, dim3(kBX, kBY), 0, cs>>>(
        static_cast<const __nv_bfloat16 *>(x), rows, cols, qo, so);
  else
    q8_store_tile_kernel<float>
        <<<(unsigned)tiles, dim3(kBX, kBY), 0, cs>>>(static_cast<const float *>(x), rows, cols, qo, so);
  dora::count_launches(1);
  return dora::launch_status();
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
  return act == DORA_BF16 ? launch_q8_load<__nv_bfloat16>(q, scale, rows, cols, block_rows, x, cs, device, info.sms)
                          : launch_q8_load<float>(q, scale, rows, cols, block_rows, x, cs, device, info.sms);
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
             ? launch_q8_fwd<__nv_bfloat16, true>(base, lora, g, s, T, out, y, q, scale, cs, device, info.sms)
             : launch_q8_fwd<float, true>(base, lora, g, s, T, out, y, q, scale, cs, device, info.sms);
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
  if (act == DORA_BF16) {
    if (q8_vector_ok<__nv_bfloat16>(out, {grad_out, d_base, d_lora}, q))
      return launch_q8_bwd<__nv_bfloat16, 8>(grad_out, q, scale, g, norm, s, T, out, d_base, d_lora, d_mag, part,
                                             workspace_bytes, cs, device, info.sms);
    return launch_q8_bwd<__nv_bfloat16, 1>(grad_out, q, scale, g, norm, s, T, out, d_base, d_lora, d_mag, part,
                                           workspace_bytes, cs, device, info.sms);
  }
  if (q8_vector_ok<float>(out, {grad_out, d_base, d_lora}, q))
    return launch_q8_bwd<float, 4>(grad_out, q, scale, g, norm, s, T, out, d_base, d_lora, d_mag, part,
                                   workspace_bytes, cs, device, info.sms);
  return launch_q8_bwd<float, 1>(grad_out, q, scale, g, norm, s, T, out, d_base, d_lora, d_mag, part, workspace_bytes,
                                 cs, device, info.sms);
}
