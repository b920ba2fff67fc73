// Matrices made nearly orthogonal by Newton-Schulz products, and the Muon step
// around them.
//
// For a matrix u, X = u / |u| (Frobenius norm), its short side as rows (s <= L):
//   A = X X^T,  B = a I + b A + c A A,  X <- B X      `iterations` times
// B is a polynomial of the symmetric A, so A and B are symmetric: their tiles
// below the diagonal are the mirrored ones above it and are not computed.
//
// X, A and B are held in fp16 times 2^12.  Their values are at most 1.2, 1.5
// and 3.45 in magnitude (the largest singular value never passes 1.21), which
// leaves a factor of 4, and nothing above 2^-26 loses bits; fp16 has three bits
// more than bf16 at the same rate of the tensor cores.  Rounded to bf16
// instead, the result is 1.1 % off (in the 2-norm, for a gradient of four
// strong directions over noise), with fp16 0.13 %.
//
// The products run on SM pairs (tcgen05 .cta_group::2, tiles of 256 x 256, fp32
// accumulators in TMEM, operands staged by TMA), all matrices of one size
// together.  A and the short products read both operands along their rows; X
// as the second operand of B X is read as it lies ("MN-major").
//
// Roles per CTA: warps 0 and 10 TMA producers, one for each operand, warp 1
// MMA issuer (leader CTA of the pair), warps 2-9 epilogue.  Every wait is
// bounded: on expiry the kernel records a timeout in the workspace's error
// word, drains what it has in flight, frees its tensor memory and returns.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;   // the quintic's coefficients
constexpr float kHeld = 4096.f;                              // factor of every value held in fp16

// ---------------------------------------------------------------- products

constexpr int kBM = 128;                  // operand rows (or columns) per CTA: the pair covers 256
constexpr int kTile = 2 * kBM;
constexpr int kBK = 64;                   // reduction elements per stage
constexpr int kGroup = 16;                // reduction elements per MMA
constexpr int kOperand = kBM * kBK * 2;   // bytes of one operand in a stage
constexpr int kHalf = kOperand / 2;       // an MN-major operand is two boxes of 64 columns x 64 rows
constexpr int kStages = 7;
constexpr int kTmemCols = 512;            // two accumulators of 256 columns
constexpr int kEpiWarps = 8;              // per CTA: two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kEpiWarps + 32, kSecondProducer = 2 + kEpiWarps;
constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kOperand;
// The limit of a wait, and what the epilogue's wait for a tile has on top for each stage of its reduction.
constexpr uint64_t kWaitNs = 2000000000ull, kStageNs = 2000;

// MN-major operand of 128 x 64: two boxes (64 columns of 128 bytes, 64 rows, 128-byte swizzle) one after the other.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  return tc::sdesc_k128(saddr) | ((uint64_t)(kHalf >> 4) << 16);
}
constexpr uint32_t kMajorB = 1u << 16;    // instruction descriptor: B is MN-major
constexpr int kStepK = 32, kStepMN = 2048;   // bytes from one group of 16 to the next
// Instruction descriptor of kind::f16: D fp32, A and B fp16 (formats 0), K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// out = alpha A B^T (kMN: A B) + beta add + diag I, for `batch` matrices.
struct Product {
  CUtensorMap a, b;
  __half* out;
  const __half* add;     // as out, or null
  int rows, cols, k;     // of out, and the reduction
  int64_t pitch, plane;  // of out, in elements
  int batch;
  bool symmetric;        // out is: tiles on and above the diagonal
  float alpha, beta, diag;
  const int32_t* skip;
  int* err;
};

__device__ __forceinline__ void advance(int& stage, uint32_t& phase) {
  if (++stage == kStages) {
    stage = 0;
    phase ^= 1u;
  }
}

__device__ __forceinline__ void give_up(int* err, volatile int* abort) {
  set_error(err, kDevTimeout);
  *abort = 1;
}

struct Tile {
  int matrix, m0, n0;
};

template <bool kMN>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Product P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  const uint32_t sA = (tc::smem_u32(smem_raw) + 1023u) & ~1023u, sB = sA + kStages * kOperand;
  const uint32_t bars = tc::smem_u32(s_bar);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto tfull = [&](int a) { return bars + 8 * (2 * kStages + a); };
  auto tempty = [&](int a) { return bars + 8 * (2 * kStages + 2 + a); };
  const uint32_t done = bars + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();

  pdl_enter();
  if (P.skip && *P.skip) return;   // every thread of both CTAs
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(full(s), 1);
        tc::mbar_init(empty(s), 1);
      }
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(tfull(a), 1);
        tc::mbar_init(tempty(a), 2 * kEpiWarps);   // one arrival for each epilogue warp of the pair
      }
      tc::mbar_init(done, 1);
      s_abort = 0;
      tc::fence_barrier_init();
      tc::fence_proxy_async_smem();
    }
  } else if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(&s_tmem), kTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = s_tmem;

  const int mt = (P.rows + kTile - 1) / kTile, nt = (P.cols + kTile - 1) / kTile;
  const int per = P.symmetric ? mt * (mt + 1) / 2 : mt * nt;
  const int64_t total = (int64_t)per * P.batch;
  const int nk = (P.k + kBK - 1) / kBK;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  // Columns of an MMA: those that the tile has, to 16, or to 128 where each CTA reads its half along the rows.
  auto mma_n = [&](const Tile& d) {
    constexpr int to = kMN ? 128 : 16;
    return min(kTile, (P.cols - d.n0 + to - 1) / to * to);
  };
  auto decode = [&](int64_t t) {
    Tile d;
    d.matrix = (int)(t / per);
    int i = 0, j = (int)(t - (int64_t)d.matrix * per);
    if (P.symmetric) {
      while (j >= mt - i) j -= mt - i++;   // row i has mt - i tiles
      j += i;
    } else {
      i = j % mt;
      j /= mt;
    }
    d.m0 = i * kTile;
    d.n0 = j * kTile;
    return d;
  };

  uint32_t filled = 0, fill_par = 0;
  bool producer = false;
  if (warp == 0 || warp == kSecondProducer) {
    // ------------------------------------------------------------ TMA producers (both CTAs)
    const bool second = warp == kSecondProducer;
    if (tc::elect_one()) {
      producer = !second;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t to = second ? sB : sA;
      const CUtensorMap* map = second ? &P.b : &P.a;
      for (int64_t t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const int r = second ? d.n0 + rank * (mma_n(d) / 2) : d.m0 + rank * kBM;   // B's columns are split evenly
        for (int kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(empty(stage), phase ^ 1u, &s_abort, kWaitNs)) {
            ok = false;
            break;
          }
          if (rank == 0 && !second) tc::mbar_arrive_expect_tx(full(stage), 4 * kOperand);
          const uint32_t at = to + stage * kOperand, fbar = tc::map_peer(full(stage), 0);
          if (kMN && second) {
            tc::tma_load_3d_pair(at, map, fbar, r, kb * kBK, d.matrix);
            tc::tma_load_3d_pair(at + kHalf, map, fbar, r + 64, kb * kBK, d.matrix);
          } else {
            tc::tma_load_3d_pair(at, map, fbar, kb * kBK, r, d.matrix);
          }
          filled |= 1u << stage;
          fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
          advance(stage, phase);
        }
      }
      if (!ok) give_up(P.err, &s_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && tc::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;   // ready: the stage at hand was seen full
      const uint64_t a0 = tc::sdesc_k128(sA), b0 = kMN ? sdesc_mn128(sB) : tc::sdesc_k128(sB);
      constexpr uint32_t as = kStepK >> 4, bs = (kMN ? kStepMN : kStepK) >> 4;
      for (int64_t t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const uint32_t idesc = idesc_f16_f32(kTile, mma_n(d)) | (kMN ? kMajorB : 0u);
        if (!tc::mbar_wait(tempty(acc), acc_phase ^ 1u, &s_abort, kWaitNs)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t dst = tmem + (uint32_t)(acc * kTile);
#pragma unroll 1
        for (int kb = 0; kb < nk; ++kb) {
          if (!ready && !tc::mbar_wait(full(stage), phase, &s_abort, kWaitNs)) {
            ok = false;
            break;
          }
          const int here = stage, ng = min(kBK / kGroup, (P.k - kb * kBK + kGroup - 1) / kGroup);
          advance(stage, phase);
          // looked at under the MMAs still running (the wait itself costs 200 cycles)
          ready = tc::mbar_try_wait(full(stage), phase);
          const uint64_t a = a0 + (uint32_t)(here * (kOperand >> 4)), b = b0 + (uint32_t)(here * (kOperand >> 4));
          tc::mma_bf16_pair(dst, a, b, idesc, kb != 0);
#pragma unroll
          for (int g = 1; g < kBK / kGroup; ++g)
            if (g < ng) tc::mma_bf16_pair(dst, a + g * as, b + g * bs, idesc, 1);
          tc::tc_commit_pair_mc(empty(here), 0x3);
        }
        if (!ok) break;
        tc::tc_commit_pair_mc(tfull(acc), 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) give_up(P.err, &s_abort);
      tc::tc_commit_pair_mc(done, 0x3);   // both CTAs learn when every MMA has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q .. 32 q + 31 belong to this warp
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint64_t limit = kWaitNs + (uint64_t)nk * kStageNs;
    for (int64_t t = first; t < total; t += step) {
      const Tile d = decode(t);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(tfull(acc), acc_phase, &s_abort, limit))) {
        give_up(P.err, &s_abort);
        break;
      }
      tc::tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile);
      const int row = d.m0 + rank * kBM + q * 32 + lane;
      __half* out = P.out + (int64_t)d.matrix * P.plane;
      const __half* add = P.add ? P.add + (int64_t)d.matrix * P.plane : nullptr;
      const bool mirror = P.symmetric && d.m0 != d.n0;
#pragma unroll 1
      for (int c = half * 4; c < half * 4 + 4; ++c) {
        const int col = d.n0 + c * 32;
        if (col >= P.cols) break;
        uint32_t r[32];
        tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
        uint4 more[4] = {};
        // rows are padded to 8 elements: a vector that starts inside the row lies inside it
        if (add && row < P.rows)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (col + g * 8 < P.cols) more[g] = *reinterpret_cast<const uint4*>(add + row * P.pitch + col + g * 8);
        tc::tmem_wait_ld();
        uint32_t packed[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float v[2];
          const float2 m = __half22float2(reinterpret_cast<const __half2*>(more)[j]);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            v[x] = P.alpha * __uint_as_float(r[2 * j + x]);
            v[x] = fmaf(P.beta, x ? m.y : m.x, v[x]);
            if (row == col + 2 * j + x) v[x] += P.diag;
          }
          const __half2 h = __floats2half2_rn(v[0], v[1]);
          packed[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if (row < P.rows) {
          uint4* to = reinterpret_cast<uint4*>(out + row * P.pitch + col);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (col + g * 8 < P.cols)
              to[g] = make_uint4(packed[4 * g], packed[4 * g + 1], packed[4 * g + 2], packed[4 * g + 3]);
          if (mirror) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (col + j < P.cols)
                reinterpret_cast<uint16_t*>(out)[(int64_t)(col + j) * P.pitch + row] =
                    (uint16_t)(packed[j >> 1] >> (16 * (j & 1)));
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) tc::mbar_arrive(tempty(acc));
        else tc::mbar_arrive_remote_relaxed(tc::map_peer(tempty(acc), 0));
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  // every MMA has finished before the CTAs part
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(done, 0, nullptr, kWaitNs)) set_error(P.err, kDevTimeout);
    __syncwarp();
  }
  // after an abort the leader drains its stage barriers, on which both CTAs'
  // loads complete, before either CTA may leave; loads into a stage that it
  // had not armed yet are given a millisecond to land
  if (producer && s_abort) {
    if (rank == 0)
      for (int s = 0; s < kStages; ++s)
        if ((filled >> s) & 1u) tc::mbar_wait(full(s), (fill_par >> s) & 1u, nullptr, kWaitNs);
    const uint64_t t0 = tc::globaltimer();
    while (tc::globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncwarp();         // the cluster's barrier takes whole warps
  tc::cluster_sync();   // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Matrices [rows, cols], `pitch` elements a row, one after the other.
struct Held {
  __half* p;
  int rows, cols;
  int64_t pitch;
  int64_t plane() const { return (int64_t)rows * pitch; }
};

template <bool kMN>
cudaError_t product(const Held& a, const Held& b, const Held& out, int batch, bool symmetric, float alpha,
                    const Held* add, float beta, float diag, const int32_t* skip, int* err, cudaStream_t st) {
  Product P = {};
  if (!tma_map_16bit_3d(&P.a, a.p, batch, a.rows, a.cols, a.pitch, a.plane(), kBM) ||
      !tma_map_16bit_3d(&P.b, b.p, batch, b.rows, b.cols, b.pitch, b.plane(), kMN ? kBK : kBM))
    return cudaErrorNotSupported;
  P.out = out.p;
  P.add = add ? add->p : nullptr;
  P.rows = out.rows;
  P.cols = out.cols;
  P.k = a.cols;
  P.pitch = out.pitch;
  P.plane = out.plane();
  P.batch = batch;
  P.symmetric = symmetric;
  P.alpha = alpha;
  P.beta = beta;
  P.diag = diag;
  P.skip = skip;
  P.err = err;
  const int64_t mt = (out.rows + kTile - 1) / kTile, nt = (out.cols + kTile - 1) / kTile;
  const int64_t tiles = batch * (symmetric ? mt * (mt + 1) / 2 : mt * nt), pairs = sm_count() / 2;
  auto kern = product_kernel<kMN>;
  const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (r != cudaSuccess) return r;
  return launch_kernel(kern, dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs))), dim3(kThreads), kSmem, st, 2, P);
}

// ---------------------------------------------------------------- what surrounds them

// A part of a tensor: `count` of its matrices, which are matrices `first` and
// on of the ones at hand.
struct Segment {
  float* p;
  bf16* p16;
  const void* g;
  float* m;
  void* out;             // raw: receives the result
  int rows, cols;
  int first, count;
  float keep, step;      // p = p keep - step O
};
constexpr int kSegments = 24;
struct Matrices {
  Segment seg[kSegments];
  int n;                 // segments
  int s, L;              // of X
  int64_t pitch, plane;  // of X
  int parts;             // partial sums of a matrix
  int tiles_s, tiles_L;  // tiles of 64 x 64
  float mu;              // m = mu m + g, u = g + mu m (nesterov) or m
  bool nesterov, raw;
  int out_dtype;
  const float* grad_scale;
  const int32_t* skip;
};

__device__ __forceinline__ const Segment& segment_of(const Matrices& M, int matrix) {
  int i = 0;
  while (i + 1 < M.n && M.seg[i + 1].first <= matrix) ++i;
  return M.seg[i];
}

// Four elements of fp32 or bf16, of which the first n exist.
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, int n, float* v) {
  if (vec && n == 4) {
    if (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
      v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
      const float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]);
      v[0] = a.x;
      v[1] = a.y;
      v[2] = b.x;
      v[3] = b.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, bool vec, int n, const float* v) {
  if (vec && n == 4) {
    if (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 q;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
      h[0] = __floats2bfloat162_rn(v[0], v[1]);
      h[1] = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(p) = q;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) p[i] = from_f32<T>(v[i]);
}
__device__ __forceinline__ bool aligned_to(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Sums of squares that neither overflow nor vanish: of u, and of u 2^-90 and u 2^90.
struct Squares {
  float mid, big, small;
};
__device__ __forceinline__ Squares warp_sum(Squares v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.mid += __shfl_xor_sync(0xffffffffu, v.mid, o);
    v.big += __shfl_xor_sync(0xffffffffu, v.big, o);
    v.small += __shfl_xor_sync(0xffffffffu, v.small, o);
  }
  return v;
}

constexpr int kPart = 8192;   // elements of a partial sum
constexpr float kUp = 1.2379400392853803e27f, kDown = 8.077935669463161e-28f;   // 2^90, 2^-90

// The momentum's step, and the sums of squares of each matrix' update.
template <typename T>
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ Matrices M, Squares* __restrict__ part) {
  __shared__ Squares s_w[8];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const int matrix = blockIdx.x / M.parts, k = blockIdx.x % M.parts;
  const Segment& S = segment_of(M, matrix);
  const int64_t n = (int64_t)S.rows * S.cols, base = (int64_t)(matrix - S.first) * n;
  const T* g = reinterpret_cast<const T*>(S.g) + base;
  float* m = M.raw ? nullptr : S.m + base;
  const float scale = M.grad_scale ? *M.grad_scale : 1.f;
  const bool vg = aligned_to(g, 4 * sizeof(T)), vm = aligned_to(m, 16);
  Squares q = {0.f, 0.f, 0.f};
#pragma unroll
  for (int it = 0; it < kPart / 1024; ++it) {
    const int64_t i = (int64_t)k * kPart + it * 1024 + threadIdx.x * 4;
    const int left = i < n ? (int)(n - i < 4 ? n - i : 4) : 0;
    if (left == 0) continue;
    float u[4];
    load4(g + i, vg, left, u);
    if (!M.raw) {
      float mm[4];
      load4(m + i, vm, left, mm);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float gx = u[x] * scale;
        mm[x] = fmaf(M.mu, mm[x], gx);
        u[x] = M.nesterov ? fmaf(M.mu, mm[x], gx) : mm[x];
      }
      store4(m + i, vm, left, mm);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x >= left) continue;
      const float b = u[x] * kDown, s = u[x] * kUp;
      q.mid = fmaf(u[x], u[x], q.mid);
      q.big = fmaf(b, b, q.big);
      q.small = fmaf(s, s, q.small);
    }
  }
  q = warp_sum(q);
  if (threadIdx.x % 32 == 0) s_w[threadIdx.x / 32] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) {
      q.mid += s_w[w].mid;
      q.big += s_w[w].big;
      q.small += s_w[w].small;
    }
    part[blockIdx.x] = q;
  }
}

// One block for each matrix: the two factors that take u to X as it is held,
// 2^-e first, so that no product overflows or vanishes on the way.
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ Matrices M, const Squares* __restrict__ part,
                                                   float2* __restrict__ factor) {
  __shared__ double s_w[3][8];
  pdl_enter();
  if (M.skip && *M.skip) return;
  double v[3] = {};
  for (int i = threadIdx.x; i < M.parts; i += 256) {
    const Squares q = part[(int64_t)blockIdx.x * M.parts + i];
    v[0] += q.mid;
    v[1] += q.big;
    v[2] += q.small;
  }
#pragma unroll
  for (int c = 0; c < 3; ++c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
    if (threadIdx.x % 32 == 0) s_w[c][threadIdx.x / 32] = v[c];
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int c = 0; c < 3; ++c) {
    v[c] = s_w[c][0];
    for (int w = 1; w < 8; ++w) v[c] += s_w[c][w];
  }
  // a sum above 1e-20 has no share worth mentioning of squares that vanished
  double norm;
  if (v[0] != v[0]) norm = v[0];
  else if (isinf(v[0])) norm = sqrt(v[1]) * (double)kUp;
  else if (v[0] > 1e-20) norm = sqrt(v[0]);
  else norm = sqrt(v[2]) * (double)kDown;
  float2 f = make_float2(0.f, 0.f);
  if (norm > 0 && !isinf(norm)) {
    int e;
    frexp(norm, &e);
    e = e > 126 ? 126 : e < -126 ? -126 : e;
    f.x = (float)ldexp(1.0, -e);
    f.y = (float)((double)kHeld / ldexp(norm, -e));
  } else if (!(norm == 0)) {
    f.x = f.y = NAN;   // a NaN or an infinity in u
  }
  factor[blockIdx.x] = f;
}

// A block's tile of 64 x 64 elements of a matrix: rows r0.., columns c0.. as it
// lies in the tensor; `flip`: X is its transpose.
struct Place {
  const Segment* S;
  int matrix, r0, c0;
  bool flip;
};
__device__ __forceinline__ Place place_of(const Matrices& M) {
  const int per = M.tiles_s * M.tiles_L;
  Place p;
  p.matrix = blockIdx.x / per;
  const int t = blockIdx.x % per;
  p.S = &segment_of(M, p.matrix);
  p.flip = p.S->rows > p.S->cols;
  const int a = t / M.tiles_L * 64, b = t % M.tiles_L * 64;   // in X
  p.r0 = p.flip ? b : a;
  p.c0 = p.flip ? a : b;
  return p;
}

__device__ __forceinline__ uint2 pack_half4(const float* v) {
  const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// X = u / |u|, as it is held, its columns padded with zeros to the pitch.
template <typename T>
__global__ void __launch_bounds__(256)
build_kernel(const __grid_constant__ Matrices M, const float2* __restrict__ factor, __half* __restrict__ X) {
  __shared__ float tile[64][65];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const Place at = place_of(M);
  const Segment& S = *at.S;
  const int64_t base = (int64_t)(at.matrix - S.first) * S.rows * S.cols;
  const T* g = reinterpret_cast<const T*>(S.g) + base;
  const float* m = M.raw ? nullptr : S.m + base;
  const float scale = M.grad_scale ? *M.grad_scale : 1.f;
  const float2 f = factor[at.matrix];
  const bool vg = aligned_to(g, 4 * sizeof(T)) && S.cols % 4 == 0, vm = aligned_to(m, 16) && S.cols % 4 == 0;
  __half* out = X + (int64_t)at.matrix * M.plane;
  const int x4 = threadIdx.x % 16 * 4, y = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = at.r0 + y + 16 * i, c = at.c0 + x4;
    const int left = r < S.rows && c < S.cols ? min(4, S.cols - c) : 0;
    float u[4] = {0.f, 0.f, 0.f, 0.f};
    if (left > 0) {
      const int64_t o = (int64_t)r * S.cols + c;
      load4(g + o, vg, left, u);
      if (!M.raw) {
        float mm[4];
        load4(m + o, vm, left, mm);
#pragma unroll
        for (int x = 0; x < 4; ++x) u[x] = M.nesterov ? fmaf(M.mu, mm[x], u[x] * scale) : mm[x];
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) u[x] = u[x] * f.x * f.y;
    if (at.flip) {
#pragma unroll
      for (int x = 0; x < 4; ++x) tile[y + 16 * i][x4 + x] = u[x];
    } else if (r < M.s && c < M.pitch) {
      *reinterpret_cast<uint2*>(out + (int64_t)r * M.pitch + c) = pack_half4(u);
    }
  }
  if (!at.flip) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = at.c0 + y + 16 * i, c = at.r0 + x4;   // in X
    if (r >= M.s || c >= M.pitch) continue;
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = tile[x4 + x][y + 16 * i];
    *reinterpret_cast<uint2*>(out + (int64_t)r * M.pitch + c) = pack_half4(v);
  }
}

// p = p keep - step O, and its bf16 copy; raw: out = O.
__global__ void __launch_bounds__(256)
apply_kernel(const __grid_constant__ Matrices M, const __half* __restrict__ X) {
  __shared__ float tile[64][65];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const Place at = place_of(M);
  const Segment& S = *at.S;
  const int64_t base = (int64_t)(at.matrix - S.first) * S.rows * S.cols;
  const __half* in = X + (int64_t)at.matrix * M.plane;
  const int x4 = threadIdx.x % 16 * 4, y = threadIdx.x / 16;
  auto held4 = [&](int r, int c, float* v) {   // 4 elements of X; the pitch is a multiple of 8
    const uint2 q = r < M.s && c < M.L ? *reinterpret_cast<const uint2*>(in + (int64_t)r * M.pitch + c)
                                       : make_uint2(0u, 0u);
    const __half2* h = reinterpret_cast<const __half2*>(&q);
    const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
    v[0] = a.x * (1.f / kHeld);
    v[1] = a.y * (1.f / kHeld);
    v[2] = b.x * (1.f / kHeld);
    v[3] = b.y * (1.f / kHeld);
  };
  if (at.flip) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4];
      held4(at.c0 + y + 16 * i, at.r0 + x4, v);
#pragma unroll
      for (int x = 0; x < 4; ++x) tile[x4 + x][y + 16 * i] = v[x];
    }
    __syncthreads();
  }
  const bool even = S.cols % 4 == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = at.r0 + y + 16 * i, c = at.c0 + x4;
    const int left = r < S.rows && c < S.cols ? min(4, S.cols - c) : 0;
    if (left <= 0) continue;
    float o[4];
    if (at.flip) {
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = tile[y + 16 * i][x4 + x];
    } else {
      held4(r, c, o);
    }
    const int64_t e = base + (int64_t)r * S.cols + c;
    if (M.raw) {
      if (M.out_dtype == MOE_BF16) {
        bf16* to = reinterpret_cast<bf16*>(S.out) + e;
        store4(to, even && aligned_to(to, 8), left, o);
      } else {
        float* to = reinterpret_cast<float*>(S.out) + e;
        store4(to, even && aligned_to(to, 16), left, o);
      }
      continue;
    }
    float* p = S.p + e;
    const bool vp = even && aligned_to(p, 16);
    float v[4];
    load4(p, vp, left, v);
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = v[x] * S.keep - S.step * o[x];
    store4(p, vp, left, v);
    if (S.p16) store4(S.p16 + e, even && aligned_to(S.p16 + e, 8), left, v);
  }
}

// ---------------------------------------------------------------- the order of it all

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Matrices of s x L (s <= L) that run together, and their buffers.
constexpr size_t kMostBytes = (size_t)4 << 30;   // a larger batch runs in parts of this size
struct Sizes {
  int s, L, parts;
  int64_t pitch, square;   // of X, and of A and B
  Sizes(int rows, int cols) {
    s = rows < cols ? rows : cols;
    L = rows < cols ? cols : rows;
    pitch = round8(L);
    square = round8(s);
    parts = (int)(((int64_t)s * L + kPart - 1) / kPart);
  }
  size_t x() const { return (size_t)s * pitch * 2; }
  size_t a() const { return (size_t)s * square * 2; }
  size_t bytes(int64_t n) const {   // X and its successor, A, B, sums, factors
    return 2 * round256(n * x()) + 2 * round256(n * a()) + round256(n * parts * sizeof(Squares)) +
           round256(n * sizeof(float2));
  }
  int64_t most() const {
    int64_t n = (int64_t)(kMostBytes / (2 * x() + 2 * a() + parts * sizeof(Squares) + sizeof(float2)));
    const int64_t grid = ((int64_t)1 << 30) / ((int64_t)((s + 63) / 64) * ((L + 63) / 64));   // blocks of a launch
    if (n > grid) n = grid;
    return n < 1 ? 1 : n;
  }
};

bool empty(const moe_muon_tensor& t) { return t.batch == 0 || t.rows == 0 || t.cols == 0; }
bool alike(const moe_muon_tensor& a, const moe_muon_tensor& b) {
  return (a.rows == b.rows && a.cols == b.cols) || (a.rows == b.cols && a.cols == b.rows);
}
// Whether tensor i is the first of its size.
bool leads(const moe_muon_tensor* t, int i) {
  if (empty(t[i])) return false;
  for (int j = 0; j < i; ++j)
    if (!empty(t[j]) && alike(t[i], t[j])) return false;
  return true;
}

cudaError_t run_matrices(const Matrices& M, const Sizes& z, int n, bool grad_bf16, int iterations, char* ws,
                         cudaStream_t st) {
  int* err = (int*)ws;
  char* at = ws + 256;
  auto take = [&](size_t bytes) {
    char* p = at;
    at += round256(bytes);
    return p;
  };
  Held X{(__half*)take(n * z.x()), z.s, z.L, z.pitch}, Y{(__half*)take(n * z.x()), z.s, z.L, z.pitch};
  Held A{(__half*)take(n * z.a()), z.s, z.s, z.square}, B{(__half*)take(n * z.a()), z.s, z.s, z.square};
  Squares* part = (Squares*)take((size_t)n * z.parts * sizeof(Squares));
  float2* factor = (float2*)take((size_t)n * sizeof(float2));
  const dim3 sums((unsigned)(n * z.parts)), tiles((unsigned)((int64_t)n * M.tiles_s * M.tiles_L)), threads(256);
  cudaError_t e = grad_bf16 ? launch_kernel(momentum_kernel<bf16>, sums, threads, 0, st, 1, M, part)
                            : launch_kernel(momentum_kernel<float>, sums, threads, 0, st, 1, M, part);
  if (e == cudaSuccess) e = launch_kernel(norm_kernel, dim3((unsigned)n), threads, 0, st, 1, M, part, factor);
  if (e == cudaSuccess)
    e = grad_bf16 ? launch_kernel(build_kernel<bf16>, tiles, threads, 0, st, 1, M, factor, X.p)
                  : launch_kernel(build_kernel<float>, tiles, threads, 0, st, 1, M, factor, X.p);
  // what is held is 2^12 times the value: a product of two comes out 2^24 times
  const float back = 1.f / kHeld;
  for (int i = 0; i < iterations && e == cudaSuccess; ++i) {
    e = product<false>(X, X, A, n, true, back, nullptr, 0.f, 0.f, M.skip, err, st);
    if (e == cudaSuccess) e = product<false>(A, A, B, n, true, kC * back, &A, kB, kA * kHeld, M.skip, err, st);
    if (e == cudaSuccess) e = product<true>(B, X, Y, n, false, back, nullptr, 0.f, 0.f, M.skip, err, st);
    const Held t = X;
    X = Y;
    Y = t;
  }
  if (e == cudaSuccess) e = launch_kernel(apply_kernel, tiles, threads, 0, st, 1, M, X.p);
  return e;
}

}  // namespace

size_t orthogonal_workspace(const moe_muon_tensor* tensors, int count) {
  size_t most = 0;
  for (int i = 0; i < count; ++i) {
    if (!leads(tensors, i)) continue;
    const Sizes z(tensors[i].rows, tensors[i].cols);
    int64_t n = 0;
    for (int j = i; j < count; ++j)
      if (!empty(tensors[j]) && alike(tensors[i], tensors[j])) n += tensors[j].batch;
    const int64_t cap = z.most();
    const size_t bytes = z.bytes(n < cap ? n : cap);
    if (bytes > most) most = bytes;
  }
  return 256 + most;
}

cudaError_t launch_orthogonal(const moe_muon_tensor* tensors, int count, int grad_dtype, const moe_muon_params& h,
                              const OrthogonalRaw* raw, const float* grad_scale, const int32_t* skip, void* ws,
                              cudaStream_t st) {
  for (int i = 0; i < count; ++i) {
    if (!leads(tensors, i)) continue;
    const Sizes z(tensors[i].rows, tensors[i].cols);
    const int64_t cap = z.most();
    Matrices M = {};
    M.s = z.s;
    M.L = z.L;
    M.pitch = z.pitch;
    M.plane = z.s * z.pitch;
    M.parts = z.parts;
    M.tiles_s = (z.s + 63) / 64;
    M.tiles_L = (z.L + 63) / 64;
    M.mu = (float)h.momentum;
    M.nesterov = h.nesterov != 0;
    M.raw = raw != nullptr;
    M.out_dtype = raw ? raw->out_dtype : MOE_F32;
    M.grad_scale = grad_scale;
    M.skip = skip;
    int held = 0;   // matrices in M
    auto flush = [&]() {
      if (held == 0) return cudaSuccess;
      const cudaError_t e = run_matrices(M, z, held, grad_dtype == MOE_BF16, h.iterations, (char*)ws, st);
      M.n = held = 0;
      return e;
    };
    for (int j = i; j < count; ++j) {
      const moe_muon_tensor& t = tensors[j];
      if (empty(t) || !alike(tensors[i], t)) continue;
      const int64_t size = (int64_t)t.rows * t.cols;
      for (int64_t b = 0; b < t.batch;) {
        if (held == cap || M.n == kSegments) {
          const cudaError_t e = flush();
          if (e != cudaSuccess) return e;
        }
        const int64_t n = t.batch - b < cap - held ? t.batch - b : cap - held;
        Segment& S = M.seg[M.n++];
        S = {};
        S.rows = t.rows;
        S.cols = t.cols;
        S.first = held;
        S.count = (int)n;
        if (raw) {
          S.g = (const char*)raw->x + b * size * (raw->x_dtype == MOE_BF16 ? 2 : 4);
          S.out = (char*)raw->out + b * size * (raw->out_dtype == MOE_BF16 ? 2 : 4);
        } else {
          S.p = t.p + b * size;
          S.p16 = t.p_bf16 ? (bf16*)t.p_bf16 + b * size : nullptr;
          S.g = (const char*)t.grad + b * size * (grad_dtype == MOE_BF16 ? 2 : 4);
          S.m = t.m + b * size;
          S.keep = (float)(1.0 - h.lr * t.weight_decay);
          S.step = (float)(h.lr * t.scale);
        }
        held += (int)n;
        b += n;
      }
    }
    const cudaError_t e = flush();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
