// Gradient of the expert FFN on CUDA cores: the fp32 layer, and the bf16
// path used to cross-check the tensor-core kernels.
//
// Expert e maps its rows r by (Qwen2-MoE module article, mlqm.cn, section 2.2)
//   a = W1 x + b1,  h = act(a),  y = W2 h + b2
// and from dy (the gradient of y) follow, with G = 1 (GELU) or 2 (SwiGLU, W1
// and W3 stacked):
//   dh = W2^T dy                      [rows, F]
//   da = dh act'(a)                   [rows, G F]
//   dx = W1^T da                      [rows, H]
//   dW1 = sum_r da_r x_r^T, db1 = sum_r da_r,  dW2 = sum_r dy_r h_r^T, db2 = sum_r dy_r
// a is computed again from x (the forward pass keeps h, from which GELU's
// slope cannot be had: GELU is not one-to-one).  da is kept in fp32.
#include "common.cuh"
#include "ffn_backward.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kB = 64, kBK = 16, kThreads = 256;   // 64 x 64 tiles, 4 x 4 values a thread

// Row tile `tile` of kB rows: its expert and rows; false past the last one.
__device__ __forceinline__ bool row_tile(const int32_t* __restrict__ offs, int E, int tile, int* e, int* r0, int* r1) {
  int before = 0;
  for (int i = 0; i < E; ++i) {
    const int a = offs[i], b = offs[i + 1], n = (b - a + kB - 1) / kB;
    if (tile < before + n) {
      *e = i;
      *r0 = a + (tile - before) * kB;
      *r1 = b;
      return true;
    }
    before += n;
  }
  return false;
}

// dst[k][i] = src[i * si + k * sk] for the tile's kB indices i < ni and kBK
// reduction indices k < nk, else 0.  One of the two strides is 1; consecutive
// threads run along it.
template <typename T>
__device__ __forceinline__ void load_tile(float (*dst)[kB + 4], const T* __restrict__ src, int64_t si, int64_t sk,
                                          int ni, int nk) {
#pragma unroll
  for (int c = 0; c < kB * kBK / kThreads; ++c) {
    const int at = c * kThreads + threadIdx.x;
    const int i = sk == 1 ? at / kBK : at % kB;
    const int k = sk == 1 ? at % kBK : at / kB;
    dst[k][i] = i < ni && k < nk ? to_f32(src[i * si + k * sk]) : 0.f;
  }
}

__device__ __forceinline__ void multiply(float (&acc)[4][4], const float (*A)[kB + 4], const float (*B)[kB + 4],
                                         int ty, int tx) {
#pragma unroll
  for (int k = 0; k < kBK; ++k) {
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = A[k][ty * 4 + i];
      b[i] = B[k][tx * 4 + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// da for one 64-row x 64-column tile: the products a (one, or gate and up)
// and dh, all of length H, then the activation's slope.
template <typename T, bool kSwi>
__global__ void __launch_bounds__(kThreads)
hidden_gradient_simt_kernel(const T* __restrict__ x, const T* __restrict__ dy, const int32_t* __restrict__ offs,
                            int E, const T* __restrict__ W1, const float* __restrict__ b1, const T* __restrict__ W2,
                            int H, int F, float* __restrict__ da) {
  __shared__ float sx[kBK][kB + 4], sdy[kBK][kB + 4], sg[kBK][kB + 4], su[kSwi ? kBK : 1][kB + 4], s2[kBK][kB + 4];
  constexpr int G = kSwi ? 2 : 1;
  pdl_enter();
  int e, r0, r1;
  if (!row_tile(offs, E, blockIdx.y, &e, &r0, &r1)) return;
  const int f0 = blockIdx.x * kB, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nr = min(kB, r1 - r0), nf = min(kB, F - f0);
  const T* w1 = W1 + ((int64_t)e * G * F + f0) * H;
  const T* w2 = W2 + (int64_t)e * H * F + f0;
  float ag[4][4] = {}, au[4][4] = {}, ah[4][4] = {};
  for (int k0 = 0; k0 < H; k0 += kBK) {
    const int nk = min(kBK, H - k0);
    load_tile(sx, x + (int64_t)r0 * H + k0, (int64_t)H, (int64_t)1, nr, nk);
    load_tile(sdy, dy + (int64_t)r0 * H + k0, (int64_t)H, (int64_t)1, nr, nk);
    load_tile(sg, w1 + k0, (int64_t)H, (int64_t)1, nf, nk);
    if (kSwi) load_tile(su, w1 + (int64_t)F * H + k0, (int64_t)H, (int64_t)1, nf, nk);
    load_tile(s2, w2 + (int64_t)k0 * F, (int64_t)1, (int64_t)F, nf, nk);
    __syncthreads();
    multiply(ag, sx, sg, ty, tx);
    if (kSwi) multiply(au, sx, su, ty, tx);
    multiply(ah, sdy, s2, ty, tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= nr) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = f0 + tx * 4 + j;
      if (f >= F) continue;
      float* d = da + (int64_t)(r0 + r) * G * F + f;
      const float a = ag[i][j] + (b1 ? b1[(int64_t)e * G * F + f] : 0.f);
      if (kSwi) {
        const float u = au[i][j] + (b1 ? b1[(int64_t)e * G * F + F + f] : 0.f);
        swiglu_gradient(a, u, ah[i][j], d, d + F);
      } else {
        *d = ah[i][j] * gelu_slope(a);
      }
    }
  }
}

// dx tile: da [rows, N] times W1[e] [N, H].
template <typename T>
__global__ void __launch_bounds__(kThreads)
input_gradient_simt_kernel(const float* __restrict__ da, const int32_t* __restrict__ offs, int E,
                           const T* __restrict__ W1, int N, int H, T* __restrict__ dx) {
  __shared__ float sa[kBK][kB + 4], sw[kBK][kB + 4];
  pdl_enter();
  int e, r0, r1;
  if (!row_tile(offs, E, blockIdx.y, &e, &r0, &r1)) return;
  const int h0 = blockIdx.x * kB, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nr = min(kB, r1 - r0), nh = min(kB, H - h0);
  float acc[4][4] = {};
  for (int k0 = 0; k0 < N; k0 += kBK) {
    const int nk = min(kBK, N - k0);
    load_tile(sa, da + (int64_t)r0 * N + k0, (int64_t)N, (int64_t)1, nr, nk);
    load_tile(sw, W1 + ((int64_t)e * N + k0) * H + h0, (int64_t)1, (int64_t)H, nh, nk);
    __syncthreads();
    multiply(acc, sa, sw, ty, tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ty * 4 + i < nr && tx * 4 + j < nh)
        dx[(int64_t)(r0 + ty * 4 + i) * H + h0 + tx * 4 + j] = from_f32<T>(acc[i][j]);
}

// One tile of dW[e] [M, N] = sum over expert e's rows of a_r b_r^T; zeros for
// an expert with no row.
template <typename TA, typename T>
__global__ void __launch_bounds__(kThreads)
weight_gradient_simt_kernel(const TA* __restrict__ A, const T* __restrict__ B, const int32_t* __restrict__ offs,
                            int M, int N, T* __restrict__ dW) {
  __shared__ float sa[kBK][kB + 4], sb[kBK][kB + 4];
  pdl_enter();
  const int e = blockIdx.z, r0 = offs[e], r1 = offs[e + 1];
  const int n0 = blockIdx.x * kB, m0 = blockIdx.y * kB, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nm = min(kB, M - m0), nn = min(kB, N - n0);
  float acc[4][4] = {};
  for (int r = r0; r < r1; r += kBK) {
    const int nk = min(kBK, r1 - r);
    load_tile(sa, A + (int64_t)r * M + m0, (int64_t)1, (int64_t)M, nm, nk);
    load_tile(sb, B + (int64_t)r * N + n0, (int64_t)1, (int64_t)N, nn, nk);
    __syncthreads();
    multiply(acc, sa, sb, ty, tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ty * 4 + i < nm && tx * 4 + j < nn)
        dW[((int64_t)e * M + m0 + ty * 4 + i) * N + n0 + tx * 4 + j] = from_f32<T>(acc[i][j]);
}

template <typename T>
cudaError_t run_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da, cudaStream_t st) {
  const bool swi = (s.flags & MOE_FLAG_SWIGLU) != 0;
  const int N = swi ? 2 * s.F : s.F;
  const int64_t mtiles = max_rows / kB + s.E;
  if (mtiles > 65535 || (N + kB - 1) / kB > 65535 || (s.H + kB - 1) / kB > 65535) return cudaErrorNotSupported;
  cudaError_t e = cudaSuccess;
  auto tiles = [](int n) { return (unsigned)((n + kB - 1) / kB); };
  if (max_rows > 0 && (b.dx_perm || b.dW1 || b.db1)) {
    auto k = swi ? hidden_gradient_simt_kernel<T, true> : hidden_gradient_simt_kernel<T, false>;
    e = launch_kernel(k, dim3(tiles(s.F), (unsigned)mtiles), dim3(kThreads), 0, st, 1, (const T*)b.x_perm,
                      (const T*)b.dy_perm, b.offs, s.E, (const T*)b.W1, b.b1, (const T*)b.W2, s.H, s.F, da);
    if (e != cudaSuccess) return e;
    if (b.dx_perm)
      e = launch_kernel(input_gradient_simt_kernel<T>, dim3(tiles(s.H), (unsigned)mtiles), dim3(kThreads), 0, st, 1,
                        (const float*)da, b.offs, s.E, (const T*)b.W1, N, s.H, (T*)b.dx_perm);
    if (e != cudaSuccess) return e;
  }
  if (b.dW1)
    e = launch_kernel(weight_gradient_simt_kernel<float, T>, dim3(tiles(s.H), tiles(N), (unsigned)s.E),
                      dim3(kThreads), 0, st, 1, (const float*)da, (const T*)b.x_perm, b.offs, N, s.H, (T*)b.dW1);
  if (e == cudaSuccess && b.dW2)
    e = launch_kernel(weight_gradient_simt_kernel<T, T>, dim3(tiles(s.F), tiles(s.H), (unsigned)s.E),
                      dim3(kThreads), 0, st, 1, (const T*)b.dy_perm, (const T*)b.h_perm, b.offs, s.H, s.F,
                      (T*)b.dW2);
  if (e == cudaSuccess && b.db1) e = launch_row_sums(MOE_F32, da, b.offs, s.E, N, b.db1, st);
  if (e == cudaSuccess && b.db2) e = launch_row_sums(s.dtype, b.dy_perm, b.offs, s.E, s.H, b.db2, st);
  return e;
}

}  // namespace

cudaError_t launch_ffn_backward_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da,
                                     cudaStream_t st) {
  return s.dtype == MOE_BF16 ? run_simt<bf16>(s, max_rows, b, da, st) : run_simt<float>(s, max_rows, b, da, st);
}

// ---------------------------------------------------------------- bias gradients
namespace {

constexpr int kSumCols = 32, kSumRows = 8;

// out[e, c] = sum of column c over expert e's rows, in fp32: 32 columns x 8
// interleaved groups of rows a block, the groups added in order.
template <typename T>
__global__ void __launch_bounds__(kSumCols * kSumRows)
row_sums_kernel(const T* __restrict__ A, const int32_t* __restrict__ offs, int N, float* __restrict__ out) {
  __shared__ float part[kSumRows][kSumCols];
  pdl_enter();
  const int e = blockIdx.y, c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int r0 = offs[e], r1 = offs[e + 1];
  float sum = 0.f;
  if (c < N) {
#pragma unroll 4
    for (int r = r0 + g; r < r1; r += kSumRows) sum += to_f32(A[(int64_t)r * N + c]);
  }
  part[g][threadIdx.x % kSumCols] = sum;
  __syncthreads();
  if (g == 0 && c < N) {
    for (int i = 1; i < kSumRows; ++i) sum += part[i][threadIdx.x];
    out[(int64_t)e * N + c] = sum;
  }
}

}  // namespace

cudaError_t launch_row_sums(int dtype, const void* A, const int32_t* offs, int E, int N, float* out,
                            cudaStream_t st) {
  const dim3 grid((unsigned)((N + kSumCols - 1) / kSumCols), (unsigned)E);
  if (dtype == MOE_BF16)
    return launch_kernel(row_sums_kernel<bf16>, grid, dim3(kSumCols * kSumRows), 0, st, 1, (const bf16*)A, offs, N,
                         out);
  return launch_kernel(row_sums_kernel<float>, grid, dim3(kSumCols * kSumRows), 0, st, 1, (const float*)A, offs, N,
                       out);
}

}  // namespace moe
