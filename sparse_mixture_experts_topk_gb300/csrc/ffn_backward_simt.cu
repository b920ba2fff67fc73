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
// of the first column of tiles.  While a block multiplies the reduction
// elements in shared memory, the next (or the next two) are on their way to registers.
//
// A thread always holds 4 x 4 values (two 16-byte reads of shared memory for
// 16 multiply-adds).  A tile has 64 x 64 values, or 16 rows and 32 columns: eight
// warps then take an eighth of the reduction each, added up at the end.  These
// layers are small (the fp32 ones are for checking) and their experts have few
// rows: the small tiles are used while the experts have less than 32 rows on
// average, or while tiles of 64 would not be four for every three SMs.
// Measured, small against large: 64 tokens, H = 256, E = 8, top-2, F = 512:
// 23.7 us against 59.8; 250 tokens, H = 384, F = 640: 78 against 104, with top-4
// 137 against 121.
#include "common.cuh"
#include "ffn_backward.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
// Columns of a row product's tile of kM rows, and the reduction elements staged at a time.
template <int kM> constexpr int kCols = kM == 16 ? 32 : 64;
template <int kM> constexpr int kDepth = kM == 16 ? 64 : 32;
// Stages of dx's operands on their way to registers: a stage of the small tiles has too little to
// multiply to cover a load's time.
template <int kM> constexpr int kAhead = kM == 16 ? 2 : 1;

// Row tile `tile` of kM rows: its expert, first row and the expert's end;
// false past the last tile.  A whole warp.
template <int kM>
__device__ __forceinline__ bool row_tile(const int32_t* __restrict__ offs, int E, int tile, int* e, int* r0, int* r1) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < E; base += 32) {
    const int i = base + lane, a = i < E ? offs[i] : 0, b = i < E ? offs[i + 1] : 0, n = (b - a + kM - 1) / kM;
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
      *r0 = __shfl_sync(0xffffffffu, a + (tile - (incl - n)) * kM, src);
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
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&v)[4]) {
  uint2 u;
  reinterpret_cast<__nv_bfloat162*>(&u)[0] = __floats2bfloat162_rn(v[0], v[1]);
  reinterpret_cast<__nv_bfloat162*>(&u)[1] = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) = u;
}

// An operand of a tile, kI indices i by kBK reduction indices k, in shared
// memory as [k][i].  In memory either k runs along a row (kAlongK: element
// i, k at i * stride + k) or i does (k * stride + i).  Rows start on 16 bytes
// and the dimension along them is a multiple of 8, so four elements are
// inside or outside together; outside (i >= ni, k >= nk) is zero.
// The transposed writes of a 16-row operand would meet eight at a time in a bank
// with a warp's lanes along k.  It takes all 16 rows and two vectors along k
// instead (kSpread): rows of s have 20 floats, four rows are 16 banks apart.
// (64 tokens, H = 256, E = 8, top-2, F = 512: 25.5 -> 23.9 us, 16 tokens, H = 1024,
// E = 16: 68.5 -> 60.2; 64-row operands lose 9 % to loads that touch 16 rows.)
template <int kI, int kBK, bool kAlongK>
struct Stage {
  static constexpr bool kSpread = kAlongK && kI == 16;
  static constexpr int kVecs = kI * kBK / 4, kLoads = (kVecs + kThreads - 1) / kThreads;
  float4 v[kLoads];
  __device__ __forceinline__ static int at(int c) { return c * kThreads + threadIdx.x; }
  __device__ __forceinline__ static int i_of(int c) {
    return kSpread ? at(c) % 16 : kAlongK ? at(c) / (kBK / 4) : at(c) % (kI / 4) * 4;
  }
  __device__ __forceinline__ static int k_of(int c) {
    return kSpread ? at(c) / 16 * 4 : kAlongK ? at(c) % (kBK / 4) * 4 : at(c) / (kI / 4);
  }
  template <typename T>
  __device__ __forceinline__ void fetch(const T* __restrict__ src, int64_t stride, int ni, int nk) {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const int i = i_of(c), k = k_of(c);
      v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ni && k < nk) v[c] = load4(src + (kAlongK ? i * stride + k : k * stride + i));
    }
  }
  __device__ __forceinline__ void put(float (*s)[kI + 4]) const {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      if (at(c) >= kVecs) break;
      const int i = i_of(c), k = k_of(c);
      if (kAlongK) {
        s[k][i] = v[c].x;
        s[k + 1][i] = v[c].y;
        s[k + 2][i] = v[c].z;
        s[k + 3][i] = v[c].w;
      } else {
        *reinterpret_cast<float4*>(&s[k][i]) = v[c];
      }
    }
  }
};

// This thread's 4 x 4 values of a kM-row tile, and its share of the reduction.
template <int kM>
struct Place {
  static constexpr int kN = kCols<kM>;
  static constexpr int kTileThreads = kM / 4 * (kN / 4), kGroups = kThreads / kTileThreads;
  int ty, tx, group;
  __device__ Place() {
    const int i = threadIdx.x % kTileThreads;
    ty = i / (kN / 4);
    tx = i % (kN / 4);
    group = threadIdx.x / kTileThreads;
  }
};

// acc += A^T B over this group's share of the first nk staged elements.
template <int kM>
__device__ __forceinline__ void multiply(float (&acc)[4][4], const float (*A)[kM + 4], const float (*B)[kCols<kM> + 4],
                                         const Place<kM>& at, int nk) {
#pragma unroll 8
  for (int k = at.group; k < nk; k += Place<kM>::kGroups) {
    const float4 a4 = *reinterpret_cast<const float4*>(&A[k][at.ty * 4]);
    const float4 b4 = *reinterpret_cast<const float4*>(&B[k][at.tx * 4]);
    const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// The groups' accumulators added up, in order, in group 0's.
template <int kM>
__device__ __forceinline__ void gather(float (&acc)[4][4], const Place<kM>& at, float* s) {
  constexpr int kG = Place<kM>::kGroups, kT = Place<kM>::kTileThreads;
  if (kG == 1) return;
  __syncthreads();
  const int me = threadIdx.x % kT;
  if (at.group > 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) s[((at.group - 1) * 16 + i) * kT + me] = acc[i / 4][i % 4];
  }
  __syncthreads();
  if (at.group == 0) {
    for (int g = 1; g < kG; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] += s[((g - 1) * 16 + i) * kT + me];
  }
}
// Shared memory of gather: seven groups' accumulators of 32 threads.
constexpr int kGatherFloats = 7 * 16 * 32;

// da for one tile: the products a (one, or gate and up)
// and dh, all of length H, then the activation's slope.
template <typename T, bool kSwi, int kM>
__global__ void __launch_bounds__(kThreads)
hidden_gradient_simt_kernel(const T* __restrict__ x, const T* __restrict__ dy, const int32_t* __restrict__ offs,
                            int E, const T* __restrict__ W1, const float* __restrict__ b1, const T* __restrict__ W2,
                            int H, int F, float* __restrict__ da) {
  constexpr int G = kSwi ? 2 : 1, kN = kCols<kM>, kBK = kDepth<kM>;
  __shared__ __align__(16) float sx[kBK][kM + 4], sdy[kBK][kM + 4];
  __shared__ __align__(16) float sw[2 + (kSwi ? 1 : 0)][kBK][kN + 4];   // gate, W2, up
  static_assert(kM == 64 || sizeof(sw) >= kGatherFloats * sizeof(float), "the groups' sums reuse the weights' stage");
  pdl_enter();
  int e, r0, r1;
  // row tiles go on in the grid's third dimension where its second is full
  if (!row_tile<kM>(offs, E, blockIdx.z * gridDim.y + blockIdx.y, &e, &r0, &r1)) return;
  const Place<kM> at;
  const int f0 = blockIdx.x * kN, nr = min(kM, r1 - r0), nf = min(kN, F - f0);
  const T* px = x + (int64_t)r0 * H;
  const T* pdy = dy + (int64_t)r0 * H;
  const T* pg = W1 + ((int64_t)e * G * F + f0) * H;
  const T* p2 = W2 + (int64_t)e * H * F + f0;
  Stage<kM, kBK, true> vx, vdy;
  Stage<kN, kBK, true> vg, vu;
  Stage<kN, kBK, false> v2;
  auto fetch = [&](int k0) {
    const int nk = min(kBK, H - k0);
    vx.fetch(px + k0, H, nr, nk);
    vdy.fetch(pdy + k0, H, nr, nk);
    vg.fetch(pg + k0, H, nf, nk);
    if (kSwi) vu.fetch(pg + (int64_t)F * H + k0, H, nf, nk);
    v2.fetch(p2 + (int64_t)k0 * F, F, nf, nk);
  };
  float ag[4][4] = {}, au[4][4] = {}, ah[4][4] = {};
  fetch(0);
  for (int k0 = 0; k0 < H; k0 += kBK) {
    vx.put(sx);
    vdy.put(sdy);
    vg.put(sw[0]);
    v2.put(sw[1]);
    if (kSwi) vu.put(sw[kSwi ? 2 : 0]);
    __syncthreads();
    const int nk = min(kBK, H - k0);
    if (k0 + kBK < H) fetch(k0 + kBK);
    multiply<kM>(ag, sx, sw[0], at, nk);
    multiply<kM>(ah, sdy, sw[1], at, nk);
    if (kSwi) multiply<kM>(au, sx, sw[kSwi ? 2 : 0], at, nk);
    __syncthreads();
  }
  gather<kM>(ag, at, &sw[0][0][0]);
  gather<kM>(ah, at, &sw[0][0][0]);
  if (kSwi) gather<kM>(au, at, &sw[0][0][0]);
  if (at.group > 0 || at.tx * 4 >= nf) return;
  const int f = f0 + at.tx * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = at.ty * 4 + i;
    if (r >= nr) continue;
    float dg[4], du[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = ag[i][j] + (b1 ? b1[(int64_t)e * G * F + f + j] : 0.f);
      if (kSwi)
        swiglu_gradient(a, au[i][j] + (b1 ? b1[(int64_t)e * G * F + F + f + j] : 0.f), ah[i][j], &dg[j], &du[j]);
      else
        dg[j] = ah[i][j] * gelu_slope(a);
    }
    float* d = da + (int64_t)(r0 + r) * G * F + f;
    store4(d, dg);
    if (kSwi) store4(d + F, du);
  }
}

// acc[i][j] to out at row ty * 4 + i < ni, column tx * 4 + j < nj (a multiple of 8).
template <typename T, int kM>
__device__ __forceinline__ void store_tile(T* out, int64_t stride, const float (&acc)[4][4], int ni, int nj,
                                           const Place<kM>& at) {
  if (at.group > 0 || at.tx * 4 >= nj) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at.ty * 4 + i < ni) store4(out + (int64_t)(at.ty * 4 + i) * stride + at.tx * 4, acc[i]);
}

union Shared {
  struct { float a[kDepth<64>][64 + 4], b[kDepth<64>][kCols<64> + 4]; } w;
  struct { float a[kDepth<16>][16 + 4], b[kDepth<16>][kCols<16> + 4]; } r;
  float sums[kGatherFloats];
};

// dx tile: da [rows, N] times W1[e] [N, H].
template <typename T, int kM>
__device__ __forceinline__ void input_tile(const float* __restrict__ da, const int32_t* __restrict__ offs, int E,
                                           const T* __restrict__ W1, int N, int H, T* __restrict__ dx, int row, int col,
                                           float (*sa)[kM + 4], float (*sb)[kCols<kM> + 4], float* sums) {
  constexpr int kN = kCols<kM>, kBK = kDepth<kM>;
  int e, r0, r1;
  if (!row_tile<kM>(offs, E, row, &e, &r0, &r1)) return;
  const Place<kM> at;
  const int h0 = col * kN, nr = min(kM, r1 - r0), nh = min(kN, H - h0);
  const float* pa = da + (int64_t)r0 * N;
  const T* pw = W1 + (int64_t)e * N * H + h0;
  struct {
    Stage<kM, kBK, true> a;
    Stage<kN, kBK, false> w;
  } v[kAhead<kM>];
  float acc[4][4] = {};
  auto fetch = [&](auto& s, int k0) {
    const int nk = min(kBK, N - k0);
    if (nk <= 0) return;
    s.a.fetch(pa + k0, N, nr, nk);
    s.w.fetch(pw + (int64_t)k0 * H, H, nh, nk);
  };
#pragma unroll
  for (int j = 0; j < kAhead<kM>; ++j) fetch(v[j], j * kBK);
  for (int kj = 0; kj < N; kj += kAhead<kM> * kBK) {
#pragma unroll
    for (int j = 0; j < kAhead<kM>; ++j) {
      const int k0 = kj + j * kBK, nk = min(kBK, N - k0);
      if (nk <= 0) break;
      v[j].a.put(sa);
      v[j].w.put(sb);
      __syncthreads();
      fetch(v[j], k0 + kAhead<kM> * kBK);
      multiply<kM>(acc, sa, sb, at, nk);
      __syncthreads();
    }
  }
  gather<kM>(acc, at, sums);
  store_tile<T, kM>(dx + (int64_t)r0 * H + h0, H, acc, nr, nh, at);
}

// One tile of dW[e] [M, N] = sum over expert e's rows of a_r b_r^T (zeros for
// an expert with no row); with n0 = 0 also db[e] = sum of a_r.  dW, db nullable.
template <typename TA, typename T>
__device__ __forceinline__ void weight_tile(const TA* __restrict__ A, const T* __restrict__ B,
                                            const int32_t* __restrict__ offs, int M, int N, T* __restrict__ dW,
                                            float* __restrict__ db, int e, int m0, int n0, float (*sa)[64 + 4],
                                            float (*sb)[64 + 4]) {
  constexpr int kN = 64, kBK = kDepth<64>;
  const Place<64> at;
  const int r0 = offs[e], rows = offs[e + 1] - r0, nm = min(64, M - m0), nn = min(kN, N - n0);
  const TA* pa = A + (int64_t)r0 * M + m0;
  const T* pb = B + (int64_t)r0 * N + n0;
  Stage<64, kBK, false> va, vb;
  float acc[4][4] = {}, sum = 0.f;
  const bool sums = db && n0 == 0;
  auto fetch = [&](int k0) {
    va.fetch(pa + (int64_t)k0 * M, M, nm, min(kBK, rows - k0));
    if (dW) vb.fetch(pb + (int64_t)k0 * N, N, nn, min(kBK, rows - k0));
  };
  if (rows > 0) fetch(0);
  for (int k0 = 0; k0 < rows; k0 += kBK) {
    const int nk = min(kBK, rows - k0);
    va.put(sa);
    if (dW) vb.put(sb);
    __syncthreads();
    if (k0 + kBK < rows) fetch(k0 + kBK);
    if (dW) multiply<64>(acc, sa, sb, at, nk);
    if (sums && threadIdx.x < 64)
      for (int k = 0; k < nk; ++k) sum += sa[k][threadIdx.x];
    __syncthreads();
  }
  if (dW) store_tile<T, 64>(dW + ((int64_t)e * M + m0) * N + n0, N, acc, nm, nn, at);
  if (sums && (int)threadIdx.x < nm) db[(int64_t)e * M + m0 + threadIdx.x] = sum;
}

// The tiles of dx, then those of dW1 and of dW2, in one grid.
struct Tiles {
  int dx, dx_cols;            // blocks of dx, columns of tiles
  int w1, w1_cols, w1_per;    // blocks of dW1, columns of tiles, tiles of an expert
  int w2_cols, w2_per;
};
template <typename T, int kM>
__global__ void __launch_bounds__(kThreads)
gradients_simt_kernel(const float* __restrict__ da, const __grid_constant__ FfnBackward b, int E, int H, int F, int N,
                      Tiles t) {
  __shared__ __align__(16) Shared s;
  pdl_enter();
  int i = blockIdx.x;
  if (i < t.dx) {
    if constexpr (kM == 64)
      input_tile<T, kM>(da, b.offs, E, (const T*)b.W1, N, H, (T*)b.dx_perm, i / t.dx_cols, i % t.dx_cols, s.w.a, s.w.b,
                        s.sums);
    else
      input_tile<T, kM>(da, b.offs, E, (const T*)b.W1, N, H, (T*)b.dx_perm, i / t.dx_cols, i % t.dx_cols, s.r.a, s.r.b,
                        s.sums);
  } else if ((i -= t.dx) < t.w1) {
    const int e = i / t.w1_per, l = i % t.w1_per;
    weight_tile(da, (const T*)b.x_perm, b.offs, N, H, (T*)b.dW1, b.db1, e, l / t.w1_cols * 64, l % t.w1_cols * 64,
                s.w.a, s.w.b);
  } else {
    i -= t.w1;
    const int e = i / t.w2_per, l = i % t.w2_per;
    weight_tile((const T*)b.dy_perm, (const T*)b.h_perm, b.offs, H, F, (T*)b.dW2, b.db2, e, l / t.w2_cols * 64,
                l % t.w2_cols * 64, s.w.a, s.w.b);
  }
}

template <typename T, int kM>
cudaError_t run_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da, cudaStream_t st) {
  const bool swi = (s.flags & MOE_FLAG_SWIGLU) != 0;
  const int N = swi ? 2 * s.F : s.F;
  auto tiles = [](int64_t n) { return (n + 63) / 64; };            // weight products
  auto cols = [](int64_t n) { return (n + kCols<kM> - 1) / kCols<kM>; };   // row products
  // at most one part-filled row tile for each expert with rows
  const int64_t mtiles = max_rows / kM + (max_rows < s.E ? max_rows : s.E);
  const int64_t lim = (int64_t)1 << 31;
  if (max_rows + 64 >= lim) return cudaErrorNotSupported;   // row numbers go a stage or tile past an expert's end
  const bool hidden = max_rows > 0 && (b.dx_perm || b.dW1 || b.db1);
  if (hidden) {
    constexpr int64_t kMost = 65535;   // of a grid's second and third dimensions; 2^31 / 16 tiles take 2048 layers
    const int64_t layers = (mtiles + kMost - 1) / kMost;
    auto k = swi ? hidden_gradient_simt_kernel<T, true, kM> : hidden_gradient_simt_kernel<T, false, kM>;
    const cudaError_t e =
        launch_kernel(k, dim3((unsigned)cols(s.F), (unsigned)(mtiles < kMost ? mtiles : kMost), (unsigned)layers),
                      dim3(kThreads), 0, st, 1, (const T*)b.x_perm, (const T*)b.dy_perm, b.offs, s.E,
                      (const T*)b.W1, b.b1, (const T*)b.W2, s.H, s.F, da);
    if (e != cudaSuccess) return e;
  }
  // a bias gradient alone takes the first column of tiles
  const int64_t w1_cols = b.dW1 ? tiles(s.H) : b.db1 ? 1 : 0, w2_cols = b.dW2 ? tiles(s.F) : b.db2 ? 1 : 0;
  const int64_t w1_per = w1_cols * tiles(N), w2_per = w2_cols * tiles(s.H);
  const int64_t dx = hidden && b.dx_perm ? mtiles * cols(s.H) : 0, w1 = w1_per * s.E, all = dx + w1 + w2_per * s.E;
  if (all == 0) return cudaSuccess;
  if (all >= lim) return cudaErrorNotSupported;
  const Tiles t{(int)dx, (int)cols(s.H), (int)w1, (int)w1_cols, (int)w1_per, (int)w2_cols, (int)w2_per};
  return launch_kernel(gradients_simt_kernel<T, kM>, dim3((unsigned)all), dim3(kThreads), 0, st, 1, (const float*)da,
                       b, s.E, s.H, s.F, N, t);
}

template <typename T>
cudaError_t pick_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da, cudaStream_t st) {
  const int64_t large = (max_rows / 64 + s.E) * ((s.F + 63) / 64);   // da's tiles of 64 rows, about
  const bool small = max_rows < 32 * (int64_t)s.E || large * 3 < (int64_t)sm_count() * 4;
  return small ? run_simt<T, 16>(s, max_rows, b, da, st) : run_simt<T, 64>(s, max_rows, b, da, st);
}

}  // namespace

cudaError_t launch_ffn_backward_simt(const Shape& s, int64_t max_rows, const FfnBackward& b, float* da,
                                     cudaStream_t st) {
  return s.dtype == MOE_BF16 ? pick_simt<bf16>(s, max_rows, b, da, st) : pick_simt<float>(s, max_rows, b, da, st);
}

}  // namespace moe
