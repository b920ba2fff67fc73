// Gradients of the token exchange: the weighted combine's, and the
// dispatch's (tokens sorted by expert and back).
//
// Combine (Qwen2-MoE code walkthrough, jsqmd.com, section 3.1 item 2):
//   out[t] = sum_j w[t, j] y[pos[t, j]]
//   dy[pos[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[pos[t, j]]>
// A kept slot owns its row, so dy needs no sum; a dropped slot (pos < 0) has
// no row and dw = 0.
//
// Dispatch (section 3.1 item 3) copies x[t] to the rows of its kept slots:
//   dx[t] = sum_j dx_perm[pos[t, j]] (+ add[t])
// summed in fp32 in slot order, then the addend; both results are
// deterministic.
//
// Both are bound by memory.  Measured: combine 44.5 us for the prefill layer
// (8192 tokens, H = 3584, top-2, bf16: 294 MB, 6.6 TB/s), 76.6 us for 16384
// tokens of which a capacity keeps 26 k of 65 k slots; dispatch 168 us for
// 32768 tokens, H = 4096, top-2 with an addend (1.07 GB, 6.4 TB/s).
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 128;

// kWarps warps take a token: dout is read once for its K slots, and the K
// partial dot products are reduced over the warps in a fixed order.  A token
// without a kept slot reads no dout.  KP: K rounded up to 2, 4 or 8 so the
// slot arrays stay in registers.  All loads of a step (kUnroll vectors of dout
// and of every slot's row) are issued before the first is used.
template <typename T, int KP, int kWarps>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ y_perm,
                        const int32_t* __restrict__ pos, const float* __restrict__ w, int64_t Tn, int K,
                        int vec_per_row, uint4* __restrict__ dy_perm, float* __restrict__ dw) {
  constexpr int V = Vec<T>::N, kUnroll = KP <= 4 ? 2 : 1, kStep = 32 * kWarps;
  __shared__ float s_part[kWarps][KP];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = kWarps == 1 ? (int64_t)blockIdx.x * (kThreads / 32) + warp : (int64_t)blockIdx.x;
  if (t >= Tn) return;   // a whole warp (kWarps == 1); never with one token a block
  const int first = kWarps == 1 ? lane : (int)threadIdx.x;
  int p[KP];
  float wt[KP], dot[KP];
  bool any = false;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    p[j] = j < K ? pos[t * K + j] : -1;
    wt[j] = j < K ? w[t * K + j] : 0.f;
    dot[j] = 0.f;
    any |= p[j] >= 0;
  }
  const int end = any ? vec_per_row : 0;
  for (int v0 = first; v0 < end; v0 += kStep * kUnroll) {
    uint4 gr[kUnroll], yr[kUnroll][KP];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = v0 + u * kStep;
      if (v < end) gr[u] = __ldcs(dout + t * vec_per_row + v);
#pragma unroll
      for (int j = 0; j < KP; ++j)
        if (dw && p[j] >= 0 && v < end) yr[u][j] = __ldcs(y_perm + (int64_t)p[j] * vec_per_row + v);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = v0 + u * kStep;
      if (v >= end) break;
      float g[V];
      Vec<T>::unpack(gr[u], g);
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        if (p[j] < 0) continue;
        if (dw) {
          float y[V];
          Vec<T>::unpack(yr[u][j], y);
#pragma unroll
          for (int i = 0; i < V; ++i) dot[j] = fmaf(g[i], y[i], dot[j]);
        }
        if (dy_perm) {
          float d[V];
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] = wt[j] * g[i];
          __stcs(dy_perm + (int64_t)p[j] * vec_per_row + v, Vec<T>::pack(d));
        }
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int j = 0; j < KP; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
  }
  if (kWarps == 1) {
#pragma unroll
    for (int j = 0; j < KP; ++j)
      if (lane == j && j < K) dw[t * K + j] = dot[j];
    return;
  }
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < KP; ++j) s_part[warp % kWarps][j] = dot[j];
  }
  __syncthreads();
  if ((int)threadIdx.x < K) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += s_part[i][threadIdx.x];
    dw[t * K + threadIdx.x] = sum;
  }
}

// One thread for each 16-byte vector of dx.  dx may be the addend's buffer:
// a thread reads what it overwrites.
template <typename T>
__global__ void __launch_bounds__(256)
dispatch_backward_kernel(const uint4* __restrict__ dx_perm, const int32_t* __restrict__ pos, int64_t Tn, int K,
                         int vec_per_row, const uint4* add, uint4* dx) {
  constexpr int V = Vec<T>::N;
  pdl_enter();
  const int64_t n = Tn * vec_per_row;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / vec_per_row;
    const int v = (int)(i % vec_per_row);
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
    for (int j = 0; j < K; ++j) {
      const int p = pos[t * K + j];
      if (p < 0) continue;
      float f[V];
      Vec<T>::unpack(__ldcs(dx_perm + (int64_t)p * vec_per_row + v), f);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += f[c];
    }
    if (add) {
      float f[V];
      Vec<T>::unpack(add[i], f);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += f[c];
    }
    dx[i] = Vec<T>::pack(acc);
  }
}

template <typename T, int KP>
cudaError_t run_combine_backward(const Shape& s, const void* dout, const void* y_perm, const int32_t* pos,
                                 const float* w, void* dy_perm, float* dw, cudaStream_t st) {
  const int vec = (int)((int64_t)s.H * s.esize() / 16);
  const bool wide = vec > 64;   // a row of more than two vectors a lane is spread over the block
  const int64_t blocks = wide ? s.T : (s.T + kThreads / 32 - 1) / (kThreads / 32);
  auto k = wide ? combine_backward_kernel<T, KP, kThreads / 32> : combine_backward_kernel<T, KP, 1>;
  return launch_kernel(k, dim3((unsigned)blocks), dim3(kThreads), 0, st, 1, (const uint4*)dout, (const uint4*)y_perm,
                       pos, w, s.T, s.K, vec, (uint4*)dy_perm, dw);
}

template <typename T>
cudaError_t pick_combine_backward(const Shape& s, const void* dout, const void* y_perm, const int32_t* pos,
                                  const float* w, void* dy_perm, float* dw, cudaStream_t st) {
  if (s.K <= 2) return run_combine_backward<T, 2>(s, dout, y_perm, pos, w, dy_perm, dw, st);
  if (s.K <= 4) return run_combine_backward<T, 4>(s, dout, y_perm, pos, w, dy_perm, dw, st);
  return run_combine_backward<T, 8>(s, dout, y_perm, pos, w, dy_perm, dw, st);
}

}  // namespace

cudaError_t launch_combine_backward(const Shape& s, const void* dout, const void* y_perm, const int32_t* pos,
                                    const float* w, void* dy_perm, float* dw, cudaStream_t st) {
  if (s.T == 0 || (!dy_perm && !dw)) return cudaSuccess;
  return s.dtype == MOE_BF16 ? pick_combine_backward<bf16>(s, dout, y_perm, pos, w, dy_perm, dw, st)
                             : pick_combine_backward<float>(s, dout, y_perm, pos, w, dy_perm, dw, st);
}

cudaError_t launch_dispatch_backward(const Shape& s, const void* dx_perm, const int32_t* pos, const void* add,
                                     void* dx, cudaStream_t st) {
  if (s.T == 0) return cudaSuccess;
  const int vec = (int)((int64_t)s.H * s.esize() / 16);
  const int64_t need = (s.T * vec + 255) / 256, cap = (int64_t)sm_count() * 8;
  auto k = s.dtype == MOE_BF16 ? dispatch_backward_kernel<bf16> : dispatch_backward_kernel<float>;
  return launch_kernel(k, dim3((unsigned)(need < cap ? need : cap)), dim3(256), 0, st, 1, (const uint4*)dx_perm, pos,
                       s.T, s.K, vec, (const uint4*)add, (uint4*)dx);
}

}  // namespace moe
