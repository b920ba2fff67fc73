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
//
// Two launches: the tiles of da, then those of dx, dW1 and dW2 side by side
// (they need da and nothing of each other).  The bias gradients are the
// column sums of the weight gradients' left operand, added up by the blocks
// of the first column of tiles.  A block computes a kB x kB tile, the next 32
// reduction elements on their way to registers while it multiplies the last
// 32 in shared memory.  These layers are small (the fp32 ones are for
// checking): 32 x 32 tiles spread them over more SMs, and are used while
// 64 x 64 ones would not fill two rounds of blocks.  Measured on a layer of
// 64 tokens (H = 256, E = 8, F = 512): 12 us with tiles of 32, 21 with 64.
#include "common.cuh"
#include "ffn_backward.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kBK = 32, kThreads = 256;

// Row tile `tile` of kB rows: its expert, first row and the expert's end;
// false past the last tile.  A whole warp.
template <int kB>
__device__ __forceinline__ bool row_tile(const int32_t* __restrict__ offs, int E, int tile, int* e, int* r0, int* r1) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < E; base += 32) {
    const int i = base + lane, a = i < E ? offs[i] : 0, b = i < E ? offs[i + 1] : 0, n = (b - a + kB - 1) / kB;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    incl += before;
    const unsigned hit = __ballot_sync(0xffffffffu, tile >= incl - n && tile < incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      *e = base + src;
      *r0 = __shfl_sync(0xffffffffu, a + (tile - (incl - n)) * kB, src);
      *r1 = __shfl_sync(0xffffffffu, b, src);
      return true;
    }
    before = __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&u)[0]);
  const float2 b = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(&u)[1]);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(bf16* p, float4 v) {
  uint2 u;
  reinterpret_cast<__nv_bfloat162*>(&u)[0] = __floats2bfloat162_rn(v.x, v.y);
  reinterpret_cast<__nv_bfloat162*>(&u)[1] = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = u;
}

// An operand of a tile, kB indices i by kBK reduction indices k, in shared
// memory as [k][i].  In memory either k runs along a row (kAlongK: element
// i, k at i * stride + k) or i does (k * stride + i).  Rows start on 16 bytes
// and the dimension along them is a multiple of 8, so four elements are
// inside or outside together; outside (i >= ni, k >= nk) is zero.
template <int kB, bool kAlongK>
struct Stage {
  static constexpr int kLoads = kB * kBK / 4 / kThreads;
  float4 v[kLoads];
  template <typename T>
  __device__ __forceinline__ void fetch(const T* __restrict__ src, int64_t stride, int ni, int nk) {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const int at = c * kThreads + threadIdx.x;
      const int i = kAlongK ? at / (kBK / 4) : at % (kB / 4) * 4, k = kAlongK ? at % (kBK / 4) * 4 : at / (kB / 4);
      v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ni && k < nk) v[c] = load4(src + (kAlongK ? i * stride + k : k * stride + i));
    }
  }
  __device__ __forceinline__ void put(float (*s)[kB + 4]) const {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const int at = c * kThreads + threadIdx.x;
      if (kAlongK) {
        const int i = at / (kBK / 4), k = at % (kBK / 4) * 4;
        s[k][i] = v[c].x;
        s[k + 1][i] = v[c].y;
        s[k + 2][i] = v[c].z;
        s[k + 3][i] = v[c].w;
      } else {
        *reinterpret_cast<float4*>(&s[at / (kB / 4)][at % (kB / 4) * 4]) = v[c];
      }
    }
  }
};

// acc += A^T B over the staged reduction: thread (ty, tx) holds R x R values.
template <int kB, int R>
__device__ __forceinline__ void multiply(float (&acc)[R][R], const float (*A)[kB + 4], const float (*B)[kB + 4], int ty,
                                         int tx) {
#pragma unroll 8
  for (int k = 0; k < kBK; ++k) {
    float a[R], b[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      a[i] = A[k][ty * R + i];
      b[i] = B[k][tx * R + i];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// da for one kB-row x kB-column tile: the products a (one, or gate and up)
// and dh, all of length H, then the activation's slope.
template <typename T, bool kSwi, int kB>
__global__ void __launch_bounds__(kThreads)
hidden_gradient_simt_kernel(const T* __restrict__ x, const T* __restrict__ dy, const int32_t* __restrict__ offs,
                            int E, const T* __restrict__ W1, const float* __restrict__ b1, const T* __restrict__ W2,
                            int H, int F, float* __restrict__ da) {
  constexpr int G = kSwi ? 2 : 1, R = kB / 16;
  __shared__ float sx[kBK][kB + 4], sdy[kBK][kB + 4], sg[kBK][kB + 4], su[kSwi ? kBK : 1][kB + 4], s2[kBK][kB + 4];
  pdl_enter();
  int e, r0, r1;
  if (!row_tile<kB>(offs, E, blockIdx.y, &e, &r0, &r1)) return;
  const int f0 = blockIdx.x * kB, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nr = min(kB, r1 - r0), nf = min(kB, F - f0);
  const T* px = x + (int64_t)r0 * H;
  const T* pdy = dy + (int64_t)r0 * H;
  const T* pg = W1 + ((int64_t)e * G * F + f0) * H;
  const T* p2 = W2 + (int64_t)e * H * F + f0;
  Stage<kB, true> vx, vdy, vg, vu;
  Stage<kB, false> v2;
  auto fetch = [&](int k0) {
    const int nk = min(kBK, H - k0);
    vx.fetch(px + k0, H, nr, nk);
    vdy.fetch(pdy + k0, H, nr, nk);
    vg.fetch(pg + k0, H, nf, nk);
    if (kSwi) vu.fetch(pg + (int64_t)F * H + k0, H, nf, nk);
    v2.fetch(p2 + (int64_t)k0 * F, F, nf, nk);
  };
  float ag[R][R] = {}, au[R][R] = {}, ah[R][R] = {};
  fetch(0);
  for (int k0 = 0; k0 < H; k0 += kBK) {
    vx.put(sx);
    vdy.put(sdy);
    vg.put(sg);
    if (kSwi) vu.put(su);
    v2.put(s2);
    __syncthreads();
    if (k0 + kBK < H) fetch(k0 + kBK);
    multiply<kB, R>(ag, sx, sg, ty, tx);
    if (kSwi) multiply<kB, R>(au, sx, su, ty, tx);
    multiply<kB, R>(ah, sdy, s2, ty, tx);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = ty * R + i;
    if (r >= nr) continue;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int f = f0 + tx * R + j;
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

// out[i, j] for i < ni, j < nj (nj a multiple of 8) of this block's tile.
template <typename T, int R>
__device__ __forceinline__ void store_tile(T* out, int64_t stride, const float (&acc)[R][R], int ni, int nj, int ty,
                                           int tx) {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (ty * R + i >= ni || tx * R >= nj) continue;
    T* p = out + (int64_t)(ty * R + i) * stride + tx * R;
    if constexpr (R == 4) {
      store4(p, make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]));
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) p[j] = from_f32<T>(acc[i][j]);
    }
  }
}

// dx tile: da [rows, N] times W1[e] [N, H].
template <typename T, int kB>
__device__ __forceinline__ void input_tile(const float* __restrict__ da, const int32_t* __restrict__ offs, int E,
                                           const T* __restrict__ W1, int N, int H, T* __restrict__ dx, int row, int col,
                                           float (*sa)[kB + 4], float (*sb)[kB + 4]) {
  constexpr int R = kB / 16;
  int e, r0, r1;
  if (!row_tile<kB>(offs, E, row, &e, &r0, &r1)) return;
  const int h0 = col * kB, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nr = min(kB, r1 - r0), nh = min(kB, H - h0);
  const float* pa = da + (int64_t)r0 * N;
  const T* pw = W1 + (int64_t)e * N * H + h0;
  Stage<kB, true> va;
  Stage<kB, false> vw;
  float acc[R][R] = {};
  va.fetch(pa, N, nr, min(kBK, N));
  vw.fetch(pw, H, nh, min(kBK, N));
  for (int k0 = 0; k0 < N; k0 += kBK) {
    va.put(sa);
    vw.put(sb);
    __syncthreads();
    const int next = k0 + kBK;
    if (next < N) {
      va.fetch(pa + next, N, nr, min(kBK, N - next));
      vw.fetch(pw + (int64_t)next * H, H, nh, min(kBK, N - next));
    }
    multiply<kB, R>(acc, sa, sb, ty, tx);
    __syncthreads();
  }
  store_tile<T, R>(dx + (int64_t)r0 * H + h0, H, acc, nr, nh, ty, tx);
}

// One tile of dW[e] [M, N] = sum over expert e's rows of a_r b_r^T (zeros for
// an expert with no row); with n0 = 0 also db[e] = sum of a_r.  dW, db nullable.
template <typename TA, typename T, int kB>
__device__ __forceinline__ void weight_tile(const TA* __restrict__ A, const T* __restrict__ B,
                                            const int32_t* __restrict__ offs, int M, int N, T* __restrict__ dW,
                                            float* __restrict__ db, int e, int m0, int n0, float (*sa)[kB + 4],
                                            float (*sb)[kB + 4]) {
  constexpr int R = kB / 16;
  const int r0 = offs[e], rows = offs[e + 1] - r0, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int nm = min(kB, M - m0), nn = min(kB, N - n0);
  const TA* pa = A + (int64_t)r0 * M + m0;
  const T* pb = B + (int64_t)r0 * N + n0;
  Stage<kB, false> va, vb;
  float acc[R][R] = {}, sum = 0.f;
  const bool sums = db && n0 == 0;
  if (rows > 0) {
    va.fetch(pa, M, nm, min(kBK, rows));
    if (dW) vb.fetch(pb, N, nn, min(kBK, rows));
  }
  for (int k0 = 0; k0 < rows; k0 += kBK) {
    va.put(sa);
    if (dW) vb.put(sb);
    __syncthreads();
    const int next = k0 + kBK;
    if (next < rows) {
      va.fetch(pa + (int64_t)next * M, M, nm, min(kBK, rows - next));
      if (dW) vb.fetch(pb + (int64_t)next * N, N, nn, min(kBK, rows - next));
    }
    if (dW) multiply<kB, R>(acc, sa, sb, ty, tx);
    if (sums && threadIdx.x < kB)
      for (int k = 0; k < kBK; ++k) sum += sa[k][threadIdx.x];
    __syncthreads();
  }
  if (dW) store_tile<T, R>(dW + ((int64_t)e * M + m0) * N + n0, N, acc, nm, nn, ty, tx);
  if (sums && (int)threadIdx.x < nm) db[(int64_t)e * M + m0 + threadIdx.x] = sum;
}

// The tiles of dx, then those of dW1 and of dW2, in one grid.
struct Tiles {
  int dx, dx_cols;            // blocks of dx, columns of tiles
  int w1, w1_cols, w1_per;    // blocks of dW1, columns of tiles, tiles of an expert
  int w2_cols, w2_per;
};
template <typename T, int kB>
__global__ void __launch_bounds__(kThreads)
gradients_simt_kernel(const float* __restrict__ da, FfnBackward b, int E, int H, int F, int N, Tiles t) {
  __shared__ float sa[kBK][kB + 4], sb[kBK][kB + 4];
  pdl_enter();
  int i = blockIdx.x;
  if (i < t.dx) {
    input_tile<T, kB>(da, b.offs, E, (const T*)b.W1, N, H, (T*)b.dx_perm, i / t.dx_cols, i % t.dx_cols, sa, sb);
  } else if ((i -= t.dx) < t.w1) {
    const int e = i / t.w1_per, l = i % t.w1_per;
    weight_tile<float, T, kB>(da, (const T*)b.x_perm, b.offs, N, H, (T*)b.dW1, b.db1, e, l / t.w1_cols * kB,
                              l % t.w1_cols * kB, sa, sb);
  } else {
    i -= t.w1;
    const int e = i / t.w2_per, l = i % t.w2_per;
    weight_tile<T, T, kB>((const T*)b.dy_perm, (const T*)b.h_perm, b.offs, H, F, (T*)b.dW2, b.db2, e,
                          l / t.w2_cols * kB, l % t.w2_cols * kB, sa, sb);
  }
}

template <typename T, int kB>
cudaError_t run_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da, cudaStream_t st) {
  const bool swi = (s.flags & MOE_FLAG_SWIGLU) != 0;
  const int N = swi ? 2 * s.F : s.F;
  auto tiles = [](int64_t n) { return (n + kB - 1) / kB; };
  // at most one part-filled row tile for each expert with rows
  const int64_t mtiles = max_rows / kB + (max_rows < s.E ? max_rows : s.E);
  if (mtiles > 65535) return cudaErrorNotSupported;
  const bool hidden = max_rows > 0 && (b.dx_perm || b.dW1 || b.db1);
  if (hidden) {
    auto k = swi ? hidden_gradient_simt_kernel<T, true, kB> : hidden_gradient_simt_kernel<T, false, kB>;
    const cudaError_t e =
        launch_kernel(k, dim3((unsigned)tiles(s.F), (unsigned)mtiles), dim3(kThreads), 0, st, 1, (const T*)b.x_perm,
                      (const T*)b.dy_perm, b.offs, s.E, (const T*)b.W1, b.b1, (const T*)b.W2, s.H, s.F, da);
    if (e != cudaSuccess) return e;
  }
  // a bias gradient alone takes the first column of tiles
  const int64_t w1_cols = b.dW1 ? tiles(s.H) : b.db1 ? 1 : 0, w2_cols = b.dW2 ? tiles(s.F) : b.db2 ? 1 : 0;
  const int64_t w1_per = w1_cols * tiles(N), w2_per = w2_cols * tiles(s.H);
  const int64_t dx = hidden && b.dx_perm ? mtiles * tiles(s.H) : 0, w1 = w1_per * s.E, all = dx + w1 + w2_per * s.E;
  if (all == 0) return cudaSuccess;
  if (all >= ((int64_t)1 << 31)) return cudaErrorNotSupported;
  const Tiles t{(int)dx, (int)tiles(s.H), (int)w1, (int)w1_cols, (int)w1_per, (int)w2_cols, (int)w2_per};
  return launch_kernel(gradients_simt_kernel<T, kB>, dim3((unsigned)all), dim3(kThreads), 0, st, 1, (const float*)da,
                       b, s.E, s.H, s.F, N, t);
}

template <typename T>
cudaError_t pick_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da, cudaStream_t st) {
  const int64_t big = (max_rows / 64 + s.E) * ((s.F + 63) / 64);   // tiles of da
  return big < 2 * sm_count() ? run_simt<T, 32>(s, max_rows, b, da, st) : run_simt<T, 64>(s, max_rows, b, da, st);
}

}  // namespace

cudaError_t launch_ffn_backward_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da,
                                     cudaStream_t st) {
  return s.dtype == MOE_BF16 ? pick_simt<bf16>(s, max_rows, b, da, st) : pick_simt<float>(s, max_rows, b, da, st);
}

}  // namespace moe
