// Gradient of the expert FFN on the tensor cores: grouped products on SM
// pairs (tcgen05 .cta_group::2, tiles of 256 x 256, fp32 accumulators in
// TMEM, operands staged by TMA).
//
// For expert e and its rows r (formulas as in ffn_backward_simt.cu):
//   dh = dy W2[e]           [rows, F]    tokens K-major, weights read along their rows
//   a  = x W1[e]^T (+ b1)   [rows, G F]  both K-major; the epilogue reads dh and writes da
//   dx = da W1[e]           [rows, H]    tokens K-major, weights read along their rows
//   dW1[e] = da^T x, dW2[e] = dy^T h     reduction over the rows, both operands read along their rows
// Nothing is transposed in memory: an operand whose reduction index runs
// along the rows of its matrix ("MN-major") is staged as it lies, and the MMA
// descriptors say so.
//
// dh goes through fp32 scratch between its product and the one that uses it,
// tile by tile in the order in which the epilogue's threads hold it, so that
// every access of a warp is 512 bytes in a row.
// Computing both products of a da tile together would spare that traffic
// (4 bytes a value, written and read once), but two accumulators of 256
// columns fill TMEM, so the epilogue could not overlap the next tile, and two
// of 128 columns would raise the operand bytes per MMA by half, which bounds
// a tile already.  da is rounded to bf16, as an operand of the next products.
//
// Rows kernel (dh, da, dx).  A block of 256 rows has its rows on the MMA's M
// side; an expert's last block of at most 128 rows runs swapped (256 weight
// columns on M, the rows on N rounded up to 16), so that few rows do not cost
// a full tile.  Weights kernel (dW1, dW2): the reduction runs over an
// expert's rows in blocks of 64, 16 to an MMA.  The rows that do not fill a
// group of 16 come from copies of them, padded with zeros to 16, that a small
// kernel makes first: in place the group goes on with rows of the next expert
// or with memory that nobody wrote, in both operands, and 0 x NaN is NaN.
// (Zeroing those rows in shared memory was measured: the second CTA's zeroing
// has to reach the MMA thread through a release and an acquire at cluster
// scope, 2300 cycles of a tile's 4300.)
//
// Roles per CTA: warp 0 TMA producer, warp 1 MMA issuer (leader CTA of the
// pair), warps 2-9 epilogue.  Two epilogue warps share a quarter of the TMEM lanes and halve its columns: with
// one, the slopes of a da tile took longer than its MMAs.  Every wait
// is bounded: on expiry the kernel records a timeout in the workspace's error
// word, drains what it has in flight, frees its tensor memory and returns.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "ffn_backward.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kBM = 128;                  // operand rows (or columns) per CTA: the pair covers 256
constexpr int kTile = 2 * kBM;            // rows and columns of a pair's tile
constexpr int kBK = 64;                   // reduction elements per stage
constexpr int kBoxRows = 32;              // swapped: token rows per box
constexpr int kSwapRows = 128;            // a last block of at most this many rows runs swapped
constexpr int kOperand = kBM * kBK * 2;   // bytes of one operand in a stage
constexpr int kHalf = kOperand / 2;       // an MN-major operand is two boxes of 64 columns x 64 rows
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kTmemCols = 512;            // two accumulators of 256 columns
constexpr int kEpiWarps = 8;              // per CTA: two for each quarter of the TMEM lanes
constexpr int kStoreBytes = 32 * 128;     // weights kernel: an epilogue warp's 32 rows of 64 columns
constexpr size_t kSmemRows = 1024 + (size_t)kStages * kStageBytes, kSmemWeights = kSmemRows + kEpiWarps * kStoreBytes;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint64_t kWaitNs = 2000000000ull;

enum Product { kDh, kDaGelu, kDaSwiglu, kDx };

// Shared-memory descriptor of an MN-major operand of 128 x 64: two boxes (64
// columns of 128 bytes, 64 rows, 128-byte swizzle) one after the other.
//   bits 16-29: bytes >> 4 between groups of 64 columns; bits 32-45: between groups of 8 rows
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kHalf >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;   // instruction descriptor: operand is MN-major
// 16 reduction elements on: along a K-major row, or two groups of 8 rows
constexpr int kStepK = 32, kStepMN = 2048;

// Per-expert tile counts' prefix into tstart [E + 1] and a copy of offs; one warp.
template <typename Count>
__device__ __forceinline__ void tile_table(const int32_t* __restrict__ offs, int E, int lane, int* s_offs, int* tstart,
                                           Count count) {
  int loc[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    loc[i] = 0;
    if (e < E) {
      const int o0 = offs[e], o1 = offs[e + 1];
      loc[i] = count(o1 - o0);
      s_offs[e] = o0;
      if (e == E - 1) s_offs[E] = o1;
    }
    sum += loc[i];
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    if (e < E) tstart[e] = run;
    run += loc[i];
  }
  if (lane == 31) tstart[E] = incl;
}

// The last expert whose first tile is at or before t.
__device__ __forceinline__ int expert_of(const int* tstart, int E, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tstart[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void advance(int& stage, uint32_t& phase) {
  if (++stage == kStages) {
    stage = 0;
    phase ^= 1u;
  }
}

// What the rows kernel's epilogue reads and writes.
struct RowsOut {
  float* dh;            // kTile x kTile fp32 for each dh tile (see dh_at): written by kDh, read by kDa*
  bf16* da;             // [rows, G F]
  bf16* dx;             // [rows, H]
  const float* bias;    // b1 or null
  float* part;          // [blocks * 8, G F] partial sums of da over rows, or null
  bool sectors;         // what this product writes has rows that start on 32 bytes
};

// Where a dh tile holds row r, column f: 32 x 32 blocks, in each of them the
// 32 rows' first four columns, then the next four, ...
__device__ __forceinline__ int dh_at(int r, int f) {
  return ((r >> 5) * (kTile / 32) + (f >> 5)) * 1024 + ((f & 31) >> 2) * 128 + (r & 31) * 4 + (f & 3);
}

// Sum over the warp's lanes of 32 values each: lane l returns the sum of v[l].
__device__ __forceinline__ float column_sum(float* v, int lane) {
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const bool up = (lane & w) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
    }
  }
  return v[0];
}

// n of 32 values (n a multiple of 8) to a row; whole 32-byte sectors where
// every row starts on one (`sectors`), else 16 bytes at a time.
template <typename T>
__device__ __forceinline__ void store_row(T* dst, const float* v, int n, bool sectors) {
  constexpr int V = Vec<T>::N;
#pragma unroll
  for (int g = 0; g < 32 / (2 * V); ++g) {
    const uint4 lo = Vec<T>::pack(v + 2 * g * V), hi = Vec<T>::pack(v + (2 * g + 1) * V);
    if (sectors && (2 * g + 2) * V <= n) {
      tc::st_global_32(dst + 2 * g * V, lo, hi);
    } else {
      if (2 * g * V < n) *reinterpret_cast<uint4*>(dst + 2 * g * V) = lo;
      if ((2 * g + 1) * V < n) *reinterpret_cast<uint4*>(dst + (2 * g + 1) * V) = hi;
    }
  }
}

// One tile of the rows kernel, this warp's half of it.  Row orientation: this
// thread's row, 32 columns at a time, the tile's left or right half.  Swapped:
// this thread's column, every other group of 32 rows.  dh: the dh tile of
// these rows, f0 this tile's first column in it.
template <int kKind>
__device__ __forceinline__ void rows_epilogue(uint32_t tbase, bool swap, int e, int row_base, int nrows, int n0,
                                              int block, float* dh, int f0, int rank, int q, int half, int lane,
                                              int N, const RowsOut& o) {
  constexpr bool kSwi = kKind == kDaSwiglu, kDa = kKind == kDaGelu || kSwi;
  constexpr int kOut = kSwi ? kBM : kTile;
  const int wide = kSwi ? 2 * N : N;     // columns of da and of the bias
  const float* be = kDa && o.bias ? o.bias + (int64_t)e * wide : nullptr;
  if (swap) {
    const int f = n0 + rank * kBM + q * 32 + lane;
    const bool ok = f < N;
    const float bf = be && ok ? be[f] : 0.f;
    float sum = 0.f;
#pragma unroll 1
    for (int c = half; c * 32 < nrows; c += 2) {
      const int64_t at = (int64_t)(row_base + c * 32) * N + f;
      const int left = ok ? nrows - c * 32 : 0;
      float* dt = dh + dh_at(c * 32, f0 + rank * kBM + q * 32 + lane);   // row c * 32 + j at + 4 j
      float g[kDa ? 32 : 1];
      if (kDa) {
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j % (kDa ? 32 : 1)] = j < left ? __ldcs(dt + 4 * j) : 0.f;
      }
      uint32_t r[32];
      tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j < left) {
          const float v = __uint_as_float(r[j]);
          if (kKind == kDh) {
            dt[4 * j] = v;
          } else if (kKind == kDx) {
            o.dx[at + (int64_t)j * N] = __float2bfloat16_rn(v);
          } else {
            const float d = g[j % (kDa ? 32 : 1)] * gelu_slope_fast(v + bf);
            sum += d;
            o.da[at + (int64_t)j * N] = __float2bfloat16_rn(d);
          }
        }
      }
    }
    if (kDa && o.part && ok) o.part[((int64_t)block * 8 + half) * wide + f] = sum;
    return;
  }
  const int r0 = rank * kBM + q * 32;          // this warp's first row of the block
  const int64_t row = row_base + r0 + lane;
  const bool ok = r0 + lane < nrows;
#pragma unroll 1
  for (int c = half * (kOut / 64); c < (half + 1) * (kOut / 64); ++c) {
    const int col = n0 + c * 32;
    if (col >= N) break;
    const int left = min(32, N - col);     // a multiple of 8
    float4* dt = reinterpret_cast<float4*>(dh + dh_at(r0 + lane, f0 + c * 32));   // columns 4 g .. 4 g + 3 at + 32 g
    float4 d[kDa ? 8 : 1];
    if (kDa) {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        d[g % (kDa ? 8 : 1)] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok && g * 4 < left) d[g % (kDa ? 8 : 1)] = __ldcs(dt + 32 * g);
      }
    }
    uint32_t r[32], u[kSwi ? 32 : 1];
    tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
    if (kSwi) tc::tmem_ld_32x32b_x32(tbase + kBM + c * 32, u);
    tc::tmem_wait_ld();
    float v[32];
    if (!kDa) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      if (kKind == kDh) {
#pragma unroll
        for (int g = 0; g < 8; ++g)
          if (ok && g * 4 < left) dt[32 * g] = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
      } else if (ok) {
        store_row(o.dx + row * N + col, v, left, o.sectors);
      }
    } else {
      float w[kSwi ? 32 : 1];
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float ba[4] = {0.f, 0.f, 0.f, 0.f}, bb[4] = {0.f, 0.f, 0.f, 0.f};
        if (be && g * 4 < left) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ba[i] = be[col + g * 4 + i];
            if (kSwi) bb[i] = be[N + col + g * 4 + i];
          }
        }
        const float4 dg = d[g % (kDa ? 8 : 1)];
        const float dh[4] = {dg.x, dg.y, dg.z, dg.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = g * 4 + i;
          const float a = __uint_as_float(r[j]) + ba[i];
          if (kSwi)
            swiglu_gradient_fast(a, __uint_as_float(u[j % (kSwi ? 32 : 1)]) + bb[i], dh[i], &v[j],
                            &w[j % (kSwi ? 32 : 1)]);
          else
            v[j] = dh[i] * gelu_slope_fast(a);
        }
      }
      if (ok) {
        store_row(o.da + row * wide + col, v, left, o.sectors);
        if (kSwi) store_row(o.da + row * wide + N + col, w, left, o.sectors);
      }
      if (o.part) {
        // rows past the block's end and columns past N are other data: they count as zeros
        const int64_t p = ((int64_t)block * 8 + rank * 4 + q) * wide + col + lane;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!ok || j >= left) {
            v[j] = 0.f;
            if (kSwi) w[j % (kSwi ? 32 : 1)] = 0.f;
          }
        const float s = column_sum(v, lane);
        if (lane < left) o.part[p] = s;
        if (kSwi) {
          const float s2 = column_sum(w, lane);
          if (lane < left) o.part[p + N] = s2;
        }
      }
    }
  }
}

__device__ __forceinline__ int row_blocks(int rows) { return (rows + kTile - 1) / kTile; }

// Barriers of a CTA: full and empty per stage, full and empty per accumulator, the end.
struct Bars {
  uint32_t base;
  __device__ uint32_t full(int s) const { return base + 8 * s; }
  __device__ uint32_t empty(int s) const { return base + 8 * (kStages + s); }
  __device__ uint32_t tfull(int a) const { return base + 8 * (2 * kStages + a); }
  __device__ uint32_t tempty(int a) const { return base + 8 * (2 * kStages + 2 + a); }
  __device__ uint32_t done() const { return base + 8 * (2 * kStages + 4); }
};

__device__ __forceinline__ void give_up(int* err, volatile int* abort) {
  set_error(err, kDevTimeout);
  *abort = 1;
}

// tmX, tmXs: token rows [rows, K] in boxes of 128 and 32 rows.  tmW: weights
// K-major [E N, K] (kDa*) or [E, K, N] in 64 x 64 boxes (kDh, kDx).
template <int kKind>
__global__ void __launch_bounds__(kThreads, 1)
backward_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmXs,
                     const __grid_constant__ CUtensorMap tmW, const int32_t* __restrict__ offs, int E, int N, int K,
                     RowsOut out, int* err) {
  constexpr bool kSwi = kKind == kDaSwiglu, kMN = kKind == kDh || kKind == kDx;
  constexpr int kOut = kSwi ? kBM : kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_offs[257], s_tstart[257];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  const uint32_t sA = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sB = sA + kStages * kOperand;
  const Bars bar{tc::smem_u32(s_bar)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();
  const int nt = (N + kOut - 1) / kOut, nk = (K + kBK - 1) / kBK;

  if (warp == 0) {
    pdl_enter();
    tile_table(offs, E, lane, s_offs, s_tstart, [&](int rows) { return row_blocks(rows) * nt; });
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(bar.full(s), 1);
        tc::mbar_init(bar.empty(s), 1);
      }
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(bar.tfull(a), 1);
        tc::mbar_init(bar.tempty(a), 2 * 32 * kEpiWarps);
      }
      tc::mbar_init(bar.done(), 1);
      s_abort = 0;
      tc::fence_barrier_init();
      tc::fence_proxy_async_smem();
      tc::prefetch_tmap(&tmX);
      tc::prefetch_tmap(&tmXs);
      tc::prefetch_tmap(&tmW);
    }
  } else if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(&s_tmem), kTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  if (warp != 0) pdl_wait();
  const uint32_t tmem = s_tmem;
  const int total = s_tstart[E], first = blockIdx.x / 2, step = gridDim.x / 2;

  struct Tile {
    int e, row_base, nrows, mma_n, n0, block, dh_tile;
    bool swap;
  };
  const int dh_nt = (N + kTile - 1) / kTile;   // kDh, kDa*: N = F
  auto decode = [&](int t) {
    Tile d;
    d.e = expert_of(s_tstart, E, t);
    const int mt = row_blocks(s_offs[d.e + 1] - s_offs[d.e]);
    const int local = t - s_tstart[d.e], rb = local % mt;
    d.row_base = s_offs[d.e] + rb * kTile;
    d.nrows = min(kTile, s_offs[d.e + 1] - d.row_base);
    d.swap = !kSwi && d.nrows <= kSwapRows;
    d.mma_n = d.swap ? (d.nrows + 15) / 16 * 16 : kTile;
    d.n0 = (local / mt) * kOut;
    d.block = (s_offs[d.e] >> 8) + d.e + rb;
    d.dh_tile = s_tstart[d.e] / nt * dh_nt + d.n0 / kTile * mt + rb;
    return d;
  };

  uint32_t filled = 0, fill_par = 0;
  bool producer = false;
  if (warp == 0) {
    if (tc::elect_one()) {
      producer = true;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const int half = d.mma_n / 2, nbox = d.swap ? (half + kBoxRows - 1) / kBoxRows : 0;
        const uint32_t tx = 2u * (uint32_t)(kOperand + (d.swap ? nbox * kBoxRows * 128 : kOperand));
        for (int kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(bar.empty(stage), phase ^ 1u, &s_abort, kWaitNs)) { ok = false; break; }
          const uint32_t fbar = tc::map_peer(bar.full(stage), 0);
          if (rank == 0) tc::mbar_arrive_expect_tx(bar.full(stage), tx);
          const uint32_t tok = (d.swap ? sB : sA) + stage * kOperand, wgt = (d.swap ? sA : sB) + stage * kOperand;
          const int n = d.n0 + rank * kBM;
          if (kMN) {
            tc::tma_load_3d_pair(wgt, &tmW, fbar, n, kb * kBK, d.e);
            tc::tma_load_3d_pair(wgt + kHalf, &tmW, fbar, n + 64, kb * kBK, d.e);
          } else {
            tc::tma_load_2d_pair(wgt, &tmW, fbar, kb * kBK, kSwi ? (2 * d.e + rank) * N + d.n0 : d.e * N + n);
          }
          if (d.swap) {
            for (int i = 0; i < nbox; ++i)
              tc::tma_load_2d_pair(tok + i * kBoxRows * 128, &tmXs, fbar, kb * kBK,
                                   d.row_base + rank * half + i * kBoxRows);
          } else {
            tc::tma_load_2d_pair(tok, &tmX, fbar, kb * kBK, d.row_base + rank * kBM);
          }
          filled |= 1u << stage;
          fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
          advance(stage, phase);
        }
      }
      if (!ok) give_up(err, &s_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && tc::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const uint32_t idesc = tc::idesc_bf16_f32(kTile, d.mma_n) | (kMN ? (d.swap ? kMajorA : kMajorB) : 0u);
        if (!tc::mbar_wait(bar.tempty(acc), acc_phase ^ 1u, &s_abort, kWaitNs)) { ok = false; break; }
        tc::tc_fence_after();
        const uint32_t dst = tmem + (uint32_t)(acc * kTile);
        for (int kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(bar.full(stage), phase, &s_abort, kWaitNs)) { ok = false; break; }
          tc::tc_fence_after();
          const uint32_t a0 = sA + stage * kOperand, b0 = sB + stage * kOperand;
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            uint64_t da, db;
            if (kMN && d.swap) da = sdesc_mn128(a0 + k * kStepMN);
            else da = tc::sdesc_k128(a0 + k * kStepK);
            if (kMN && !d.swap) db = sdesc_mn128(b0 + k * kStepMN);
            else db = tc::sdesc_k128(b0 + k * kStepK);
            tc::mma_bf16_pair(dst, da, db, idesc, (kb | k) != 0);
          }
          tc::tc_commit_pair_mc(bar.empty(stage), 0x3);
          advance(stage, phase);
        }
        if (!ok) break;
        tc::tc_commit_pair_mc(bar.tfull(acc), 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) give_up(err, &s_abort);
      tc::tc_commit_pair_mc(bar.done(), 0x3);   // both CTAs learn when every MMA has finished
    }
    __syncwarp();
    if (lane == 0 && !tc::mbar_wait(bar.done(), 0, nullptr, kWaitNs)) set_error(err, kDevTimeout);
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q .. 32 q + 31 belong to this warp
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = first; t < total; t += step) {
      const Tile d = decode(t);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar.tfull(acc), acc_phase, &s_abort, kWaitNs))) {
        give_up(err, &s_abort);
        break;
      }
      tc::tc_fence_after();
      rows_epilogue<kKind>(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile), d.swap, d.e, d.row_base,
                           d.nrows, d.n0, d.block, out.dh + (int64_t)d.dh_tile * kTile * kTile, d.n0 % kTile, rank, q, half,
                           lane, N, out);
      tc::tc_fence_before();
      if (rank == 0) tc::mbar_arrive(bar.tempty(acc));
      else tc::mbar_arrive_remote(tc::map_peer(bar.tempty(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (producer && rank == 0 && s_abort)
    for (int s = 0; s < kStages; ++s)
      if ((filled >> s) & 1u) tc::mbar_wait(bar.full(s), (fill_par >> s) & 1u, nullptr, kWaitNs);
  tc::cluster_sync();   // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// What is left of the smaller work, in one launch beside one another.
//
// Tails: the rows of each expert past its last whole group of 16, padded with
// zeros to 16, [E, 16, cols] for each of up to four operands.
struct Operand {
  const uint4* rows;
  uint4* tails;
  int vec;              // 16-byte vectors in a row
};
constexpr int kTailRows = 16, kTailSplit = 4;   // blocks for an expert's tail of one operand
constexpr int kRedCols = 32, kRedGroups = 8, kSumVecs = 8, kSumGroups = 32;
struct Extras {
  Operand o[4];
  int tails;            // blocks of tails
  const float* part;    // db1's partial sums, n columns
  float* db1;
  int n, swaps, cols1;  // columns of blocks
  int db1_blocks;
  const uint4* dy;      // db2 = the sum of an expert's dy rows, h columns
  float* db2;
  int h, cols2;
};

// One expert's rows past its last whole group of 16, a quarter of them.
__device__ __forceinline__ void copy_tail(const Operand& o, const int32_t* __restrict__ offs, int e, int part) {
  const int r0 = offs[e], rows = offs[e + 1] - r0, whole = rows / kTailRows * kTailRows;
  if (rows == whole) return;   // no tail: never read
  const int per = kTailRows / kTailSplit * o.vec;
  for (int i = threadIdx.x; i < per; i += blockDim.x) {
    const int r = part * (kTailRows / kTailSplit) + i / o.vec, v = i % o.vec;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (whole + r < rows) x = o.rows[(int64_t)(r0 + whole + r) * o.vec + v];
    o.tails[((int64_t)e * kTailRows + r) * o.vec + v] = x;
  }
}

// db1[e, c]: the row blocks' partial sums, added in a fixed order.  A swapped
// block has two partials, another eight; 8 threads of a column take them in turn.
__device__ __forceinline__ void reduce_bias(const Extras& x, const int32_t* __restrict__ offs, int e, int col,
                                            float* s) {
  const int g = threadIdx.x / kRedCols, c = col * kRedCols + threadIdx.x % kRedCols;
  const int r0 = offs[e], rows = offs[e + 1] - r0, mt = row_blocks(rows);
  const int last = mt > 0 ? rows - (mt - 1) * kTile : 0;
  const int parts = 8 * mt - (x.swaps && mt > 0 && last <= kSwapRows ? 6 : 0);
  const float* p = x.part + ((int64_t)(r0 >> 8) + e) * 8 * x.n + c;
  float sum = 0.f;
  if (c < x.n) {
#pragma unroll 4
    for (int i = g; i < parts; i += kRedGroups) sum += p[(int64_t)i * x.n];
  }
  s[threadIdx.x] = sum;
  __syncthreads();
  if (g == 0 && c < x.n) {
    for (int i = 1; i < kRedGroups; ++i) sum += s[i * kRedCols + threadIdx.x];
    x.db1[(int64_t)e * x.n + c] = sum;
  }
}

// db2[e, 64 columns]: 32 threads of a 16-byte vector take the rows in turn,
// their sums are added in order.
__device__ __forceinline__ void sum_rows(const Extras& x, const int32_t* __restrict__ offs, int e, int col, float* s) {
  const int g = threadIdx.x / kSumVecs, v = col * kSumVecs + threadIdx.x % kSumVecs, vec = x.h / 8;
  const int r1 = offs[e + 1];
  float sum[8] = {};
  if (v < vec) {
#pragma unroll 4
    for (int r = offs[e] + g; r < r1; r += kSumGroups) {
      float f[8];
      Vec<bf16>::unpack(__ldg(x.dy + (int64_t)r * vec + v), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += f[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[(g * kSumVecs + threadIdx.x % kSumVecs) * 8 + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;   // one column of the block's 64
  if (c < kSumVecs * 8 && col * kSumVecs * 8 + c < x.h) {
    float total = 0.f;
    for (int i = 0; i < kSumGroups; ++i) total += s[i * kSumVecs * 8 + c];
    x.db2[(int64_t)e * x.h + col * kSumVecs * 8 + c] = total;
  }
}

__global__ void __launch_bounds__(256)
backward_extras_kernel(const __grid_constant__ Extras x, const int32_t* __restrict__ offs, int E) {
  __shared__ float s[256 * 8];
  pdl_enter();
  int i = blockIdx.x;
  if (i < x.tails) {
    const int e = i % E, k = i / E;
    copy_tail(x.o[k / kTailSplit], offs, e, k % kTailSplit);
  } else if ((i -= x.tails) < x.db1_blocks) {
    reduce_bias(x, offs, i / x.cols1, i % x.cols1, s);
  } else {
    i -= x.db1_blocks;
    sum_rows(x, offs, i / x.cols2, i % x.cols2, s);
  }
}

// One weight gradient: out [E, M, N] = sum over an expert's rows of A's row
// (M columns) times B's row (N columns).
struct WeightProduct {
  int M, N;
};

// tmA, tmB: an operand's rows in boxes of 64 x 64; tmAt, tmBt: its tails in
// boxes of 64 columns x 16 rows; tmO: out in boxes of 32 rows x 64 columns.
// Products 0 and 1 follow one another.  An accumulator leaves through shared
// memory by TMA: stored by its threads, a row each, it took 594 us instead of
// 440 at the prefill layer with 16 bytes a store (450 with 32, which needs
// rows that start on 32 bytes).
__global__ void __launch_bounds__(kThreads, 1)
backward_weights_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
                        const __grid_constant__ CUtensorMap tmAt0, const __grid_constant__ CUtensorMap tmBt0,
                        const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
                        const __grid_constant__ CUtensorMap tmAt1, const __grid_constant__ CUtensorMap tmBt1,
                        const __grid_constant__ CUtensorMap tmO0, const __grid_constant__ CUtensorMap tmO1,
                        const int32_t* __restrict__ offs, int E, WeightProduct P0, WeightProduct P1, int* err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_offs[257];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  const uint32_t sA = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sB = sA + kStages * kOperand, sOut = sB + kStages * kOperand;
  const Bars bar{tc::smem_u32(s_bar)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();
  auto tiles = [](int n) { return (n + kTile - 1) / kTile; };
  const int per0 = tiles(P0.M) * tiles(P0.N), per1 = tiles(P1.M) * tiles(P1.N);

  if (warp == 0) {
    pdl_enter();
    for (int e = lane; e <= E; e += 32) s_offs[e] = offs[e];
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(bar.full(s), 1);
        tc::mbar_init(bar.empty(s), 1);
      }
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(bar.tfull(a), 1);
        tc::mbar_init(bar.tempty(a), 2 * 32 * kEpiWarps);
      }
      tc::mbar_init(bar.done(), 1);
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
  if (warp != 0) pdl_wait();
  const uint32_t tmem = s_tmem;
  const int total0 = E * per0, total = total0 + E * per1, first = blockIdx.x / 2, step = gridDim.x / 2;

  struct Tile {
    int p, e, m0, n0, row0, groups, nk;   // groups of 16 rows, the tail's included; stages
    bool tail;                            // the last stage is the tail's, one group
  };
  auto decode = [&](int t) {
    Tile d;
    d.p = t >= total0 ? 1 : 0;
    const int tl = t - (d.p ? total0 : 0), per = d.p ? per1 : per0, nt = tiles(d.p ? P1.N : P0.N);
    d.e = tl / per;
    const int local = tl - d.e * per, mi = local / nt;
    d.m0 = mi * kTile;
    d.n0 = (local - mi * nt) * kTile;
    d.row0 = s_offs[d.e];
    const int rows = s_offs[d.e + 1] - d.row0, whole = rows / kTailRows;
    d.tail = rows % kTailRows != 0;
    d.nk = (whole * kTailRows + kBK - 1) / kBK + (d.tail ? 1 : 0);
    d.groups = whole + (d.tail ? 1 : 0);
    return d;
  };

  uint32_t filled = 0, fill_par = 0;
  bool producer = false;
  if (warp == 0) {
    if (tc::elect_one()) {
      producer = true;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const CUtensorMap* mA = d.p ? &tmA1 : &tmA0;
        const CUtensorMap* mB = d.p ? &tmB1 : &tmB0;
        const int m = d.m0 + rank * kBM, n = d.n0 + rank * kBM;
        for (int kb = 0; kb < d.nk; ++kb) {
          if (!tc::mbar_wait(bar.empty(stage), phase ^ 1u, &s_abort, kWaitNs)) { ok = false; break; }
          const uint32_t fbar = tc::map_peer(bar.full(stage), 0);
          const bool tail = d.tail && kb == d.nk - 1;
          int r = d.row0 + kb * kBK;
          if (tail) {
            mA = d.p ? &tmAt1 : &tmAt0;
            mB = d.p ? &tmBt1 : &tmBt0;
            r = d.e * kTailRows;
          }
          if (rank == 0)
            tc::mbar_arrive_expect_tx(bar.full(stage), tail ? 2 * kStageBytes * kTailRows / kBK : 2 * kStageBytes);
          const uint32_t a = sA + stage * kOperand, b = sB + stage * kOperand;
          tc::tma_load_2d_pair(a, mA, fbar, m, r);
          tc::tma_load_2d_pair(a + kHalf, mA, fbar, m + 64, r);
          tc::tma_load_2d_pair(b, mB, fbar, n, r);
          tc::tma_load_2d_pair(b + kHalf, mB, fbar, n + 64, r);
          filled |= 1u << stage;
          fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
          advance(stage, phase);
        }
      }
      if (!ok) give_up(err, &s_abort);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && tc::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint32_t idesc = tc::idesc_bf16_f32(kTile, kTile) | kMajorA | kMajorB;
      Tile next = first < total ? decode(first) : Tile{};
      for (int t = first; t < total && ok; t += step) {
        const Tile d = next;
        if (!tc::mbar_wait(bar.tempty(acc), acc_phase ^ 1u, &s_abort, kWaitNs)) { ok = false; break; }
        tc::tc_fence_after();
        const uint32_t dst = tmem + (uint32_t)(acc * kTile);
        for (int kb = 0; kb < d.nk; ++kb) {
          if (!tc::mbar_wait(bar.full(stage), phase, &s_abort, kWaitNs)) { ok = false; break; }
          tc::tc_fence_after();
          const uint32_t a0 = sA + stage * kOperand, b0 = sB + stage * kOperand;
          // the tail's stage holds the last group alone, the one before it what is left of the whole ones
          const bool tail = d.tail && kb == d.nk - 1;
          const int groups = tail ? 1 : min(kBK / 16, d.groups - (d.tail ? 1 : 0) - kb * (kBK / 16));
          for (int k = 0; k < groups; ++k)
            tc::mma_bf16_pair(dst, sdesc_mn128(a0 + k * kStepMN), sdesc_mn128(b0 + k * kStepMN), idesc, (kb | k) != 0);
          tc::tc_commit_pair_mc(bar.empty(stage), 0x3);
          advance(stage, phase);
          if (kb == 0 && t + step < total) next = decode(t + step);   // its divisions run beside the MMAs
        }
        if (!ok) break;
        tc::tc_commit_pair_mc(bar.tfull(acc), 0x3);
        if (d.nk == 0 && t + step < total) next = decode(t + step);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) give_up(err, &s_abort);
      tc::tc_commit_pair_mc(bar.done(), 0x3);
    }
    __syncwarp();
    if (lane == 0 && !tc::mbar_wait(bar.done(), 0, nullptr, kWaitNs)) set_error(err, kDevTimeout);
    __syncwarp();
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t buf = sOut + (warp - 2) * kStoreBytes;
    uint8_t* g = smem_raw + (buf - tc::smem_u32(smem_raw)) + lane * 128;   // this thread's row of it
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = first; t < total; t += step) {
      const Tile d = decode(t);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar.tfull(acc), acc_phase, &s_abort, kWaitNs))) {
        give_up(err, &s_abort);
        break;
      }
      tc::tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile);
      const int m = d.m0 + rank * kBM + q * 32;
      if (m < (d.p ? P1.M : P0.M)) {
#pragma unroll 1
        for (int c = half * (kTile / 128); c < (half + 1) * (kTile / 128); ++c) {
          const int n = d.n0 + c * 64;
          if (n >= (d.p ? P1.N : P0.N)) break;
          if (lane == 0) tc::bulk_wait_read();   // the buffer's previous store has been read
          __syncwarp();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
            if (d.nk > 0) {
              uint32_t r[32];
              tc::tmem_ld_32x32b_x32(tbase + c * 64 + h * 32, r);
              tc::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)   // 16 bytes at the place that the 128-byte swizzle gives them
              *reinterpret_cast<uint4*>(g + (((h * 4 + j) ^ (lane & 7)) << 4)) = Vec<bf16>::pack(v + j * 8);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::tma_store_3d(d.p ? &tmO1 : &tmO0, buf, n, m, d.e);
        }
      }
      tc::tc_fence_before();
      if (rank == 0) tc::mbar_arrive(bar.tempty(acc));
      else tc::mbar_arrive_remote(tc::map_peer(bar.tempty(acc), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) tc::bulk_wait_all();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (producer && rank == 0 && s_abort)
    for (int s = 0; s < kStages; ++s)
      if ((filled >> s) & 1u) tc::mbar_wait(bar.full(s), (fill_par >> s) & 1u, nullptr, kWaitNs);
  tc::cluster_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// One persistent launch of CTA pairs, never more than fit at once.
template <typename... KArgs, typename... Args>
cudaError_t launch_pairs(void (*kern)(KArgs...), size_t smem, cudaStream_t st, Args... args) {
  cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (r != cudaSuccess) return r;
  return launch_kernel(kern, dim3((unsigned)(sm_count() / 2 * 2)), dim3(kThreads), smem, st, 2, args...);
}

// Whether every row of [.., cols] elements of `size` bytes starts on a 32-byte sector.
bool starts_on_sectors(const void* p, int cols, int size) {
  return ((uintptr_t)p % 32 == 0) && ((int64_t)cols * size % 32 == 0);
}

template <int kKind>
cudaError_t run_rows(const void* tokens, int64_t rows, int K, const void* W, int E, int N, const int32_t* offs,
                     const RowsOut& out, int* err, cudaStream_t st) {
  constexpr bool kMN = kKind == kDh || kKind == kDx;
  CUtensorMap mx, mxs, mw;
  if (!tma_map_bf16(&mx, tokens, (uint64_t)rows, (uint64_t)K, kBM) ||
      !tma_map_bf16(&mxs, tokens, (uint64_t)rows, (uint64_t)K, kBoxRows))
    return cudaErrorNotSupported;
  if (kMN ? !tma_map_bf16_3d(&mw, W, (uint64_t)E, (uint64_t)K, (uint64_t)N, kBK)
          : !tma_map_bf16(&mw, W, (uint64_t)E * N * (kKind == kDaSwiglu ? 2 : 1), (uint64_t)K, kBM))
    return cudaErrorNotSupported;
  return launch_pairs(backward_rows_kernel<kKind>, kSmemRows, st, mx, mxs, mw, offs, E, N, K, out, err);
}

}  // namespace

int64_t backward_blocks(int64_t rows, int E) { return rows / kTile + E + 1; }
size_t backward_dh_floats(int64_t rows, int E, int F) {
  const int64_t blocks = rows / kTile + (rows < E ? rows : E);   // at most: one partial block for each expert with rows
  return (size_t)blocks * ((F + kTile - 1) / kTile) * kTile * kTile;
}
size_t backward_tail_bytes(int E, int H, int N, int F) {
  return (size_t)E * kTailRows * ((size_t)N + 2 * (size_t)H + (size_t)F) * sizeof(bf16);
}

cudaError_t launch_ffn_backward_tc(const Shape& s, int64_t max_rows, const FfnBackward& b, void* da, float* dh,
                                   float* part, void* tails, int* err, cudaStream_t st) {
  const bool swi = (s.flags & MOE_FLAG_SWIGLU) != 0;
  const int G = swi ? 2 : 1, N = G * s.F;
  const int64_t lim = (int64_t)1 << 31;
  if (max_rows + kTile >= lim || (int64_t)s.E * N >= lim || (int64_t)s.E * s.H >= lim) return cudaErrorNotSupported;
  cudaError_t e = cudaSuccess;
  if (max_rows == 0) {
    // no row of any expert: every gradient is zero
    if (b.dW1) e = cudaMemsetAsync(b.dW1, 0, (size_t)s.E * N * s.H * 2, st);
    if (e == cudaSuccess && b.dW2) e = cudaMemsetAsync(b.dW2, 0, (size_t)s.E * s.F * s.H * 2, st);
    if (e == cudaSuccess && b.db1) e = cudaMemsetAsync(b.db1, 0, (size_t)s.E * N * 4, st);
    if (e == cudaSuccess && b.db2) e = cudaMemsetAsync(b.db2, 0, (size_t)s.E * s.H * 4, st);
    return e;
  }
  CUtensorMap m[8];
  CUtensorMap mo[2];
  WeightProduct P[2] = {{0, 0}, {0, 0}};
  Extras x = {};
  int n = 0;   // weight products
  bf16* at = (bf16*)tails;
  auto add_operand = [&](int i, const void* rows, int cols) {   // operand i of product n
    bf16* t = at;
    at += (int64_t)s.E * kTailRows * cols;
    x.o[2 * n + i] = {(const uint4*)rows, (uint4*)t, cols / 8};
    return tma_map_bf16(&m[4 * n + i], rows, (uint64_t)max_rows, (uint64_t)cols, kBK) &&
           tma_map_bf16(&m[4 * n + 2 + i], t, (uint64_t)s.E * kTailRows, (uint64_t)cols, kTailRows);
  };
  auto add = [&](const void* A, int M, const void* Bm, int Nn, void* dW) {
    P[n] = {M, Nn};
    const bool ok = add_operand(0, A, M) && add_operand(1, Bm, Nn) &&
                    tma_map_bf16_3d(&mo[n], dW, (uint64_t)s.E, (uint64_t)M, (uint64_t)Nn, 32);
    ++n;
    return ok;
  };
  if (b.dW1 && !add(da, N, b.x_perm, s.H, b.dW1)) return cudaErrorNotSupported;
  if (b.dW2 && !add(b.dy_perm, s.H, b.h_perm, s.F, b.dW2)) return cudaErrorNotSupported;
  x.tails = 2 * n * kTailSplit * s.E;
  RowsOut out{dh, (bf16*)da, (bf16*)b.dx_perm, b.b1, b.db1 ? part : nullptr, starts_on_sectors(da, s.F, 2)};
  if (b.dx_perm || b.dW1 || b.db1) {
    e = run_rows<kDh>(b.dy_perm, max_rows, s.H, b.W2, s.E, s.F, b.offs, out, err, st);
    if (e == cudaSuccess)
      e = swi ? run_rows<kDaSwiglu>(b.x_perm, max_rows, s.H, b.W1, s.E, s.F, b.offs, out, err, st)
              : run_rows<kDaGelu>(b.x_perm, max_rows, s.H, b.W1, s.E, s.F, b.offs, out, err, st);
    x.part = part;
    x.db1 = b.db1;
    x.n = N;
    x.swaps = swi ? 0 : 1;
    x.cols1 = (N + kRedCols - 1) / kRedCols;
    x.db1_blocks = b.db1 ? x.cols1 * s.E : 0;
  }
  x.dy = (const uint4*)b.dy_perm;
  x.db2 = b.db2;
  x.h = s.H;
  x.cols2 = (s.H / 8 + kSumVecs - 1) / kSumVecs;
  const int64_t extras = (int64_t)x.tails + x.db1_blocks + (b.db2 ? (int64_t)x.cols2 * s.E : 0);
  if (e == cudaSuccess && extras > 0)
    e = launch_kernel(backward_extras_kernel, dim3((unsigned)extras), dim3(256), 0, st, 1, x, b.offs, s.E);
  out.sectors = starts_on_sectors(b.dx_perm, s.H, 2);
  if (e == cudaSuccess && b.dx_perm)
    e = run_rows<kDx>(da, max_rows, N, b.W1, s.E, s.H, b.offs, out, err, st);
  if (n == 1) {
    for (int i = 0; i < 4; ++i) m[4 + i] = m[i];
    mo[1] = mo[0];
  }
  if (e == cudaSuccess && n > 0)
    e = launch_pairs(backward_weights_kernel, kSmemWeights, st, m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], mo[0],
                     mo[1], b.offs, s.E, P[0], P[1], err);
  return e;
}

}  // namespace moe
