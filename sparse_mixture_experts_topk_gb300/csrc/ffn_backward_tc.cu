// Gradient of the expert FFN on the tensor cores: grouped products on SM
// pairs (tcgen05 .cta_group::2, tiles of 256 x 256, fp32 accumulators in
// TMEM, operands staged by TMA).
//
// For expert e and its rows r (formulas as in ffn_backward_simt.cu):
//   dh = dy W2[e]           [rows, F]    tokens K-major, weights read along their rows
//   a  = x W1[e]^T (+ b1)   [rows, G F]  both K-major
//   dx = da W1[e]           [rows, H]    tokens K-major, weights read along their rows
//   dW1[e] = da^T x, dW2[e] = dy^T h     reduction over the rows, both operands read along their rows
// Nothing is transposed in memory: an operand whose reduction index runs
// along the rows of its matrix ("MN-major") is staged as it lies, and the MMA
// descriptors say so.
//
// Three launches.  (1) da: a pair computes a tile of dh and then the same
// tile of a (with SwiGLU its two halves, gate and up side by side), and the
// epilogue of the second turns both into da, rounded to bf16 as an operand of
// what follows.  dh waits in a scratch of 128 KB for each CTA, where every
// thread reads back what it wrote itself: it stays in L2 and needs no
// synchronisation.  (Both accumulators of a tile side by side would fill TMEM,
// and no epilogue could overlap the next tile; through memory, with a launch
// for each product, the two took 435 us instead of 425 at the prefill layer.)
// (2) The smaller work: see Extras.  (3) dx, dW1 and dW2, which need nothing of
// one another, the long tiles of dx first.
//
// Row products (dh, a, dx).  A block of 256 rows has its rows on the MMA's M
// side; an expert's last block of at most 128 rows runs swapped (256 weight
// columns on M, the rows on N rounded up to 16), so that few rows do not cost
// a full tile.  (With SwiGLU it then has three products of 256 columns, dh,
// gate and up, and the gate waits in the scratch as dh does.)
// Weight products: the reduction runs over an expert's rows in blocks of 64,
// 16 to an MMA.  The rows that do not fill a group of 16 come from copies of
// them, padded with zeros to 16, that the second launch makes: in place the
// group goes on with rows of the next expert or with memory that nobody wrote,
// in both operands, and 0 x NaN is NaN.  (Zeroing those rows in shared memory
// was measured: the second CTA's zeroing has to reach the MMA thread through a
// release and an acquire at cluster scope, 2300 cycles of a tile's 4300.)
//
// Roles per CTA: warps 0 and 10 TMA producers, one for each operand (a thread
// takes 600 cycles to fill a stage by itself, more than its MMAs take), warp 1
// MMA issuer (leader CTA of the pair), warps 2-9 epilogue.  Two epilogue warps share a quarter of the TMEM
// lanes and halve its columns: with one, the slopes of a da tile took longer
// than its MMAs.  The other CTA's arrivals that free an accumulator release
// nothing (only tensor memory was read): with a release each of its tiles
// took 1000 cycles more, and a layer of 512 tokens and 32 experts (H = 2048,
// F = 1024) 162 us instead of 140.  Tiles go round the pairs by number.  Every wait is bounded:
// on expiry the kernel records a timeout in the workspace's error word, drains
// what it has in flight, frees its tensor memory and returns.
//
// What bounds it is what a stage costs whatever its MMAs take: 590 to 605
// cycles where a row product's take 512, 570 where a swapped block's take 64,
// 610 to 700 for a weight product.  (The tensor pipe is active 77 % of the
// cycles in launch 1 and 83 % in 3 on 4096 tokens of 8 experts, where there are
// few short blocks: 1.6 PFLOP/s.)  Measured: the prefill layer (8192 tokens, H =
// 3584, E = 32, top-2, F = 2560, 1.5 TFLOP) 425 + 7 + 589 us launch by launch,
// 1.12 to 1.23 ms in a program that runs nothing else (SM clock 1.7 of 2.07 GHz,
// at which 1.27 PFLOP/s are 60 % of what the tensor cores could do, so the power
// cap is not the limit); with SwiGLU 617 + 9 + 986 us, 1.77 to 1.92 ms.
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
constexpr int kGroup = 16;                // reduction elements per MMA
constexpr int kBoxRows = 32;              // swapped: token rows per box
constexpr int kSwapRows = 128;            // a last block of at most this many rows runs swapped
constexpr int kOperand = kBM * kBK * 2;   // bytes of one operand in a stage
constexpr int kHalf = kOperand / 2;       // an MN-major operand is two boxes of 64 columns x 64 rows
constexpr int kStageBytes = 2 * kOperand;
constexpr int kTmemCols = 512;            // two accumulators of 256 columns
constexpr int kEpiWarps = 8;              // per CTA: two for each quarter of the TMEM lanes
constexpr int kStoreBytes = 32 * 128;     // an epilogue warp's 32 rows of 64 columns on their way to TMA
constexpr size_t kSmem = 1024 + (size_t)7 * kStageBytes;   // seven stages, or six and the eight store tiles
static_assert(kEpiWarps * kStoreBytes == kStageBytes, "the store tiles take a stage's place");
constexpr int kThreads = 64 + 32 * kEpiWarps + 32, kSecondProducer = 2 + kEpiWarps;
constexpr int kMaxPairs = 80;             // bounds the dh scratch: 128 KB for each CTA
constexpr int kStash = kBM * kTile;       // its fp32 values
// The limit of a wait, and what the epilogue's wait for a tile has on top for
// each stage of its reduction: a weight product's goes over all of an expert's
// rows (264 ns a stage of 64 rows at H = F = 8: two seconds are 485 M rows).
constexpr uint64_t kWaitNs = 2000000000ull, kStageNs = 2000;

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

// Per-expert tile counts' prefix into tstart [E + 1]; one warp.
template <typename Count>
__device__ __forceinline__ void tile_table(const int32_t* __restrict__ offs, int E, int lane, int* tstart,
                                           Count count) {
  int loc[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane * 8 + i;
    loc[i] = e < E ? count(offs[e + 1] - offs[e]) : 0;
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

template <int kStages>
__device__ __forceinline__ void advance(int& stage, uint32_t& phase) {
  if (++stage == kStages) {
    stage = 0;
    phase ^= 1u;
  }
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

__device__ __forceinline__ int row_blocks(int rows) { return (rows + kTile - 1) / kTile; }

// Barriers of a CTA: full and empty per stage, full and empty per accumulator, the end.
template <int kStages>
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

// What is left of the smaller work, in one launch beside one another, what takes longest first.
//
// Tails: the rows of each expert past its last whole group of 16, padded with
// zeros to 16, [E, 16, cols] for each of up to four operands.
struct Operand {
  const uint4* rows;
  uint4* tails;
  int vec;              // 16-byte vectors in a row
};
constexpr int kTailSplit = 4;   // blocks for an expert's tail of one operand
constexpr int kRedCols = 32, kRedGroups = 8;
constexpr int kSumVecs = 4, kSumGroups = 64, kSumBatch = 8;
struct Extras {
  Operand o[4];
  int tails;            // blocks of tails
  const float* part;    // db1's partial sums, n columns
  float* db1;
  int n, cols1;         // columns of blocks
  int db1_blocks;
  const uint4* dy;      // db2 = the sum of an expert's dy rows, h columns
  float* db2;
  int h, cols2;
};

// One expert's rows past its last whole group of 16, a quarter of them.
__device__ __forceinline__ void copy_tail(const Operand& o, const int32_t* __restrict__ offs, int e, int part) {
  const int r0 = offs[e], rows = offs[e + 1] - r0, whole = rows / kGroup * kGroup;
  if (rows == whole) return;   // no tail: never read
  const int per = kGroup / kTailSplit * o.vec;
  for (int i = threadIdx.x; i < per; i += blockDim.x) {
    const int r = part * (kGroup / kTailSplit) + i / o.vec, v = i % o.vec;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (whole + r < rows) x = o.rows[(int64_t)(r0 + whole + r) * o.vec + v];
    o.tails[((int64_t)e * kGroup + r) * o.vec + v] = x;
  }
}

// db1[e, c]: the row blocks' partial sums, added in a fixed order.  A swapped
// block has two partials, another eight; 8 threads of a column take them in turn.
__device__ __forceinline__ void reduce_bias(const Extras& x, const int32_t* __restrict__ offs, int e, int col,
                                            float* s) {
  const int g = threadIdx.x / kRedCols, c = col * kRedCols + threadIdx.x % kRedCols;
  const int r0 = offs[e], rows = offs[e + 1] - r0, mt = row_blocks(rows);
  const int last = mt > 0 ? rows - (mt - 1) * kTile : 0;
  const int parts = 8 * mt - (mt > 0 && last <= kSwapRows ? 6 : 0);
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

// db2[e, 32 columns]: 64 threads of a 16-byte vector take the rows in turn,
// their sums are added in order.  A batch of loads takes 3 us of an expert's
// time whatever its size, so most experts should need one (777 tokens, H =
// 1000, E = 12, top-3: 96.1 -> 92.8 us, with 32 threads and loads four by four before).
__device__ __forceinline__ void sum_rows(const Extras& x, const int32_t* __restrict__ offs, int e, int col, float* s) {
  const int g = threadIdx.x / kSumVecs, v = col * kSumVecs + threadIdx.x % kSumVecs, vec = x.h / 8;
  const uint32_t r1 = offs[e + 1];
  float sum[8] = {};
  if (v < vec) {
    // unsigned: rows go past r1, which may be near 2^31
    for (uint32_t r = offs[e] + g; r < r1; r += kSumBatch * kSumGroups) {
      uint4 u[kSumBatch];   // in flight together, zeros past the expert's end
#pragma unroll
      for (int b = 0; b < kSumBatch; ++b) {
        const uint32_t row = r + b * kSumGroups;
        u[b] = row < r1 ? __ldg(x.dy + (int64_t)row * vec + v) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int b = 0; b < kSumBatch; ++b) {
        float f[8];
        Vec<bf16>::unpack(u[b], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += f[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[(g * kSumVecs + threadIdx.x % kSumVecs) * 8 + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x;   // one column of the block's 32
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
  if (i < x.cols2 * E) {
    sum_rows(x, offs, i / x.cols2, i % x.cols2, s);
  } else if ((i -= x.cols2 * E) < x.db1_blocks) {
    reduce_bias(x, offs, i / x.cols1, i % x.cols1, s);
  } else {
    i -= x.db1_blocks;
    const int e = i % E, k = i / E;
    copy_tail(x.o[k / kTailSplit], offs, e, k % kTailSplit);
  }
}

// The kernels: da of GELU or SwiGLU experts, or the gradients that need it.
enum Job { kDaGelu, kDaSwiglu, kGradients };

struct Params {
  // kDa*: dy and x rows (boxes of 128 and of 32 rows), W2 [E, H, F], W1 [E G F, H]
  // kGradients: da rows (128, 32), W1 [E, G F, H]; the operands of dW1 and dW2
  // (A, B, and their tails in boxes of 16 rows); dW1 and dW2 (boxes of 32 rows)
  CUtensorMap map[13];
  const int32_t* offs;
  int E, H, F, N;          // N = G F
  float* stash;            // kDa*: dh of the tile at hand, kStash for each CTA
  bf16* da;                // [rows, N]
  const float* b1;         // [E, N] or null
  float* part;             // [blocks * 8, N] partial sums of da over rows, or null
  bf16* dx;                // [rows, H] or null
  int wm[2], wn[2];        // the weight products' M and N, 0 for none
  bool sectors;            // the rows of da or dx start on 32 bytes
  int* err;
  int stall;               // testing: 1 = the first stage's barrier waits for an arrival that nobody makes
};
enum Map { kDy = 0, kDyBox, kW2, kX, kXBox, kW1, kDaRows = 0, kDaBox, kW1MN, kWeightMaps, kOutMaps = 11 };

// A tile: a row product's (expert e, rows row0 .. row0 + nrows, columns n0 ..),
// or a weight product's (p, rows m0 .., columns n0 ..).
struct Tile {
  int e, row0, nrows, n0, block, m0, p;
  bool rows, swap;
};

// This thread's dh values, in groups of four: group k at [32 k].
__device__ __forceinline__ float4* stash_of(float* stash, int epi_warp, int lane) {
  return reinterpret_cast<float4*>(stash + (int64_t)blockIdx.x * kStash) + epi_warp * 32 * 32 + lane;
}

// The i-th of the four groups of 32 columns that an epilogue warp has of a dh
// tile.  SwiGLU: two of each half of the tile, those that it will have of
// that half's gate and up columns.
template <bool kSwi>
__device__ __forceinline__ int dh_chunk(int i, int half) {
  return kSwi ? (i >> 1) * 4 + half * 2 + (i & 1) : half * 4 + i;
}

// 32 values of this thread's from an accumulator to its scratch.
__device__ __forceinline__ void stash32(uint32_t taddr, float4* st) {
  uint32_t r[32];
  tc::tmem_ld_32x32b_x32(taddr, r);
  tc::tmem_wait_ld();
#pragma unroll
  for (int g = 0; g < 8; ++g)
    st[g * 32] = make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]), __uint_as_float(r[4 * g + 2]),
                             __uint_as_float(r[4 * g + 3]));
}
// dh of a tile in row orientation.
template <bool kSwi>
__device__ __forceinline__ void stash_rows(uint32_t tbase, const Tile& d, int half, int F, float4* st) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const int c = dh_chunk<kSwi>(i, half);
    if (d.n0 + c * 32 < F) stash32(tbase + c * 32, st + i * 8 * 32);
  }
}
// dh (which = 0) or the gate (1) of a swapped tile: at most two groups of 32 rows.
__device__ __forceinline__ void stash_swapped(uint32_t tbase, const Tile& d, int half, int which, float4* st) {
#pragma unroll 1
  for (int i = 0; (half + 2 * i) * 32 < d.nrows; ++i)
    stash32(tbase + (half + 2 * i) * 32, st + (which * 2 + i) * 8 * 32);
}
__device__ __forceinline__ float part_of(const float4& v, int j) {
  return (j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w;
}

// da of a swapped tile: this thread's column, every other group of 32 rows.
template <bool kSwi>
__device__ __forceinline__ void da_swapped(uint32_t tbase, const Tile& d, int rank, int q, int half, int lane,
                                           const Params& P, const float4* st) {
  const int f = d.n0 + rank * kBM + q * 32 + lane;
  const bool ok = f < P.F;
  const float* be = P.b1 && ok ? P.b1 + (int64_t)d.e * P.N + f : nullptr;
  const float bf = be ? be[0] : 0.f, bu = be && kSwi ? be[P.F] : 0.f;
  float sum = 0.f, sum_up = 0.f;
#pragma unroll 1
  for (int i = 0; (half + 2 * i) * 32 < d.nrows; ++i) {
    const int c = half + 2 * i, left = ok ? d.nrows - c * 32 : 0;
    float4 dh[8], gate[kSwi ? 8 : 1];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      dh[g] = __ldcg(st + (i * 8 + g) * 32);
      if (kSwi) gate[g % (kSwi ? 8 : 1)] = __ldcg(st + ((2 + i) * 8 + g) * 32);
    }
    uint32_t r[32];
    tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
    tc::tmem_wait_ld();
    bf16* out = P.da + (int64_t)(d.row0 + c * 32) * P.N + f;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j < left) {
        const float h = part_of(dh[j >> 2], j), v = __uint_as_float(r[j]);
        float g;
        if (kSwi) {
          float u;
          swiglu_gradient_fast(part_of(gate[(j >> 2) % (kSwi ? 8 : 1)], j) + bf, v + bu, h, &g, &u);
          sum_up += u;
          out[(int64_t)j * P.N + P.F] = __float2bfloat16_rn(u);
        } else {
          g = h * gelu_slope_fast(v + bf);
        }
        sum += g;
        out[(int64_t)j * P.N] = __float2bfloat16_rn(g);
      }
    }
  }
  if (P.part && ok) {
    float* p = P.part + ((int64_t)d.block * 8 + half) * P.N + f;
    p[0] = sum;
    if (kSwi) p[P.F] = sum_up;
  }
}

// da of a tile in row orientation: this thread's row, 32 columns at a time.
// SwiGLU: `sub` is the half of the dh tile whose gate and up columns the
// accumulator holds.
template <bool kSwi>
__device__ __forceinline__ void da_rows(uint32_t tbase, const Tile& d, int sub, int rank, int q, int half, int lane,
                                        const Params& P, const float4* st) {
  const int F = P.F, r0 = rank * kBM + q * 32;
  const int64_t row = d.row0 + r0 + lane;
  const bool ok = r0 + lane < d.nrows;
  const float* be = P.b1 ? P.b1 + (int64_t)d.e * P.N : nullptr;
#pragma unroll 1
  for (int k = 0; k < (kSwi ? 2 : 4); ++k) {
    const int i = kSwi ? sub * 2 + k : k, c = dh_chunk<kSwi>(i, half);   // of the dh tile
    const int acc = kSwi ? c - sub * 4 : c;                               // of the accumulator
    const int col = d.n0 + c * 32;
    if (col >= F) break;
    const int left = min(32, F - col);     // a multiple of 8
    float4 dh[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) dh[g] = __ldcg(st + (i * 8 + g) * 32);
    uint32_t r[32], u[kSwi ? 32 : 1];
    tc::tmem_ld_32x32b_x32(tbase + acc * 32, r);
    if (kSwi) tc::tmem_ld_32x32b_x32(tbase + kBM + acc * 32, u);
    tc::tmem_wait_ld();
    float v[32], w[kSwi ? 32 : 1];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float ba[4] = {0.f, 0.f, 0.f, 0.f}, bb[4] = {0.f, 0.f, 0.f, 0.f};
      if (be && g * 4 < left) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          ba[x] = be[col + g * 4 + x];
          if (kSwi) bb[x] = be[F + col + g * 4 + x];
        }
      }
      const float h[4] = {dh[g].x, dh[g].y, dh[g].z, dh[g].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int j = g * 4 + x;
        const float a = __uint_as_float(r[j]) + ba[x];
        if (kSwi)
          swiglu_gradient_fast(a, __uint_as_float(u[j % (kSwi ? 32 : 1)]) + bb[x], h[x], &v[j],
                               &w[j % (kSwi ? 32 : 1)]);
        else
          v[j] = h[x] * gelu_slope_fast(a);
      }
    }
    if (ok) {
      store_row(P.da + row * P.N + col, v, left, P.sectors);
      if (kSwi) store_row(P.da + row * P.N + F + col, w, left, P.sectors);
    }
    if (P.part) {
      // rows past the block's end and columns past F are other data: they count as zeros
      const int64_t p = ((int64_t)d.block * 8 + rank * 4 + q) * P.N + col + lane;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (!ok || j >= left) {
          v[j] = 0.f;
          if (kSwi) w[j % (kSwi ? 32 : 1)] = 0.f;
        }
      const float s = column_sum(v, lane);
      if (lane < left) P.part[p] = s;
      if (kSwi) {
        const float s2 = column_sum(w, lane);
        if (lane < left) P.part[p + F] = s2;
      }
    }
  }
}

// A tile of dx, in either orientation.
__device__ __forceinline__ void dx_tile(uint32_t tbase, const Tile& d, int rank, int q, int half, int lane,
                                        const Params& P) {
  if (d.swap) {
    const int f = d.n0 + rank * kBM + q * 32 + lane;
#pragma unroll 1
    for (int c = half; c * 32 < d.nrows; c += 2) {
      uint32_t r[32];
      tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
      tc::tmem_wait_ld();
      bf16* out = P.dx + (int64_t)(d.row0 + c * 32) * P.H + f;
      const int left = f < P.H ? d.nrows - c * 32 : 0;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j < left) out[(int64_t)j * P.H] = __float2bfloat16_rn(__uint_as_float(r[j]));
    }
    return;
  }
  const int r0 = rank * kBM + q * 32 + lane;
#pragma unroll 1
  for (int c = half * 4; c < half * 4 + 4; ++c) {
    const int col = d.n0 + c * 32;
    if (col >= P.H) break;
    uint32_t r[32];
    tc::tmem_ld_32x32b_x32(tbase + c * 32, r);
    tc::tmem_wait_ld();
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
    if (r0 < d.nrows) store_row(P.dx + (int64_t)(d.row0 + r0) * P.H + col, v, min(32, P.H - col), P.sectors);
  }
}

// A tile of a weight gradient, zeros for an expert without rows.  It leaves
// through shared memory by TMA: stored by its threads, a row each, the
// products took 594 us instead of 440 at the prefill layer with 16 bytes a
// store (450 with 32, which needs rows that start on 32 bytes).
__device__ __forceinline__ void weight_tile(uint32_t tbase, const Tile& d, bool zero, int rank, int q, int half,
                                            int lane, const Params& P, uint32_t buf, uint8_t* g) {
  const int m = d.m0 + rank * kBM + q * 32;
  if (m >= P.wm[d.p]) return;
#pragma unroll 1
  for (int c = half * 2; c < half * 2 + 2; ++c) {
    const int n = d.n0 + c * 64;
    if (n >= P.wn[d.p]) break;
    if (lane == 0) tc::bulk_wait_read();   // the buffer's previous store has been read
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      if (!zero) {
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
    if (lane == 0) tc::tma_store_3d(&P.map[kOutMaps + d.p], buf, n, m, d.e);
  }
}

template <int kJob>
__global__ void __launch_bounds__(kThreads, 1) backward_pair_kernel(const __grid_constant__ Params P) {
  constexpr bool kSwi = kJob == kDaSwiglu, kDa = kJob != kGradients;
  constexpr int kStages = kDa ? 7 : 6;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_tstart[257];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  const uint32_t sA = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sB = sA + kStages * kOperand, sOut = sB + kStages * kOperand;
  const Bars<kStages> bar{tc::smem_u32(s_bar)};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();
  auto tiles = [](int n) { return (n + kTile - 1) / kTile; };
  const int E = P.E, nt = kDa ? tiles(P.F) : P.dx ? tiles(P.H) : 0;   // columns of a row product's tiles
  const int per0 = kDa ? 0 : tiles(P.wm[0]) * tiles(P.wn[0]), per1 = kDa ? 0 : tiles(P.wm[1]) * tiles(P.wn[1]);

  if (warp == 0) {
    pdl_enter();
    tile_table(P.offs, E, lane, s_tstart, [&](int rows) { return row_blocks(rows) * nt; });
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(bar.full(s), s == 0 ? 1 + P.stall : 1);
        tc::mbar_init(bar.empty(s), 1);
      }
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(bar.tfull(a), 1);
        tc::mbar_init(bar.tempty(a), 2 * kEpiWarps);   // one arrival for each epilogue warp of the pair
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
  const int total_rows = s_tstart[E], total0 = total_rows + E * per0, total = total0 + E * per1;
  const int first = blockIdx.x / 2, step = gridDim.x / 2;

  auto decode = [&](int t) {
    Tile d = {};
    if (kDa || t < total_rows) {
      d.rows = true;
      d.e = expert_of(s_tstart, E, t);
      const int r0 = P.offs[d.e], r1 = P.offs[d.e + 1], mt = row_blocks(r1 - r0);
      const int local = t - s_tstart[d.e], col = local / mt, rb = local - col * mt;
      d.row0 = r0 + rb * kTile;
      d.nrows = min(kTile, r1 - d.row0);
      d.swap = d.nrows <= kSwapRows;
      d.n0 = col * kTile;
      d.block = (r0 >> 8) + d.e + rb;
    } else {
      d.p = t >= total0 ? 1 : 0;
      const int tl = t - (d.p ? total0 : total_rows), per = d.p ? per1 : per0, cols = tiles(P.wn[d.p]);
      d.e = tl / per;
      const int local = tl - d.e * per, mi = local / cols;
      d.m0 = mi * kTile;
      d.n0 = (local - mi * cols) * kTile;
      d.row0 = P.offs[d.e];
      d.nrows = P.offs[d.e + 1] - d.row0;
    }
    return d;
  };
  // The products of a tile, one accumulator after the other (SwiGLU: dh, then
  // a's halves as far as F goes, or gate and up), their stages, and the MMAs
  // of a stage.
  auto products = [&](const Tile& d) { return kSwi ? (d.swap || P.F - d.n0 > kBM ? 3 : 2) : kDa ? 2 : 1; };
  auto has_tail = [&](const Tile& d) { return !d.rows && d.nrows % kGroup != 0; };
  const int row_k = kDa ? P.H : P.N;   // a row product's reduction
  auto stages = [&](const Tile& d) {
    return d.rows ? (row_k + kBK - 1) / kBK
                  : (d.nrows / kGroup * kGroup + kBK - 1) / kBK + (has_tail(d) ? 1 : 0);
  };
  auto groups = [&](const Tile& d, int kb, int nk) {
    if (d.rows) return min(kBK / kGroup, (row_k - kb * kBK + kGroup - 1) / kGroup);
    if (has_tail(d) && kb == nk - 1) return 1;   // the tail's stage holds its group alone
    return min(kBK / kGroup, d.nrows / kGroup - kb * (kBK / kGroup));
  };

  uint32_t filled = 0, fill_par = 0;
  bool producer = false;
  if (warp == 0 || warp == kSecondProducer) {
    // ------------------------------------------------------------ TMA producers (both CTAs)
    const bool second = warp == kSecondProducer;   // this warp's operand: tokens or B; else weights or A
    if (tc::elect_one()) {
      producer = !second;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // Waits for a free stage and has `load` fill this warp's operand; the
      // first producer arms the leader's barrier for the pair's bytes.  The
      // kinds of loads have loops of their own: what a stage costs this thread
      // bounds the kernel.
      auto fill = [&](int nk, uint32_t bytes, auto load) {
        for (int kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(bar.empty(stage), phase ^ 1u, &s_abort, kWaitNs)) return false;
          if (rank == 0 && !second) tc::mbar_arrive_expect_tx(bar.full(stage), bytes);
          load(kb, stage * kOperand, tc::map_peer(bar.full(stage), 0));
          filled |= 1u << stage;
          fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
          advance<kStages>(stage, phase);
        }
        return true;
      };
      for (int t = first; t < total && ok; t += step) {
        const Tile d = decode(t);
        const int nk = stages(d), n = d.n0 + rank * kBM;
        if (!d.rows) {
          const CUtensorMap* m = &P.map[kWeightMaps + 4 * d.p + (second ? 1 : 0)];
          const int c = second ? n : d.m0 + rank * kBM, whole = nk - (has_tail(d) ? 1 : 0);
          const uint32_t to = second ? sB : sA;
          auto load = [&](const CUtensorMap* op, int r, uint32_t at, uint32_t fbar) {
            tc::tma_load_2d_pair(to + at, op, fbar, c, r);
            tc::tma_load_2d_pair(to + at + kHalf, op, fbar, c + 64, r);
          };
          ok = fill(whole, 2 * kStageBytes,
                    [&](int kb, uint32_t at, uint32_t fbar) { load(m, d.row0 + kb * kBK, at, fbar); }) &&
               fill(nk - whole, 2 * kStageBytes * kGroup / kBK,
                    [&](int, uint32_t at, uint32_t fbar) { load(m + 2, d.e * kGroup, at, fbar); });
          continue;
        }
        const int tokens = d.swap ? (d.nrows + 15) / 16 * 8 : kBM;   // this CTA's token rows
        const int nbox = d.swap ? (tokens + kBoxRows - 1) / kBoxRows : 1;
        const uint32_t bytes = 2 * (kOperand + (d.swap ? nbox * kBoxRows * 128 : kOperand));
        if (second) {
          const int row = d.row0 + rank * tokens;
          const uint32_t to = d.swap ? sB : sA;
          for (int sub = 0; sub < products(d) && ok; ++sub) {
            const CUtensorMap* m = &P.map[(!kDa ? kDaRows : sub == 0 ? kDy : kX) + (d.swap ? 1 : 0)];
            ok = fill(nk, bytes, [&](int kb, uint32_t at, uint32_t fbar) {
              for (int i = 0; i < nbox; ++i)
                tc::tma_load_2d_pair(to + at + i * kBoxRows * 128, m, fbar, kb * kBK, row + i * kBoxRows);
            });
          }
          continue;
        }
        // the weights: read along their rows (dh, dx) ...
        const uint32_t to = d.swap ? sA : sB;
        const CUtensorMap* mw = &P.map[kDa ? kW2 : kW1MN];
        ok = fill(nk, bytes, [&](int kb, uint32_t at, uint32_t fbar) {
          tc::tma_load_3d_pair(to + at, mw, fbar, n, kb * kBK, d.e);
          tc::tma_load_3d_pair(to + at + kHalf, mw, fbar, n + 64, kb * kBK, d.e);
        });
        // ... or K-major (a)
        if (kDa) {
          for (int sub = 1; sub < products(d) && ok; ++sub) {
            const int wrow = !kSwi ? d.e * P.F + n
                                   : d.swap ? (2 * d.e + sub - 1) * P.F + n
                                            : (2 * d.e + rank) * P.F + d.n0 + (sub - 1) * kBM;
            ok = fill(nk, bytes, [&](int kb, uint32_t at, uint32_t fbar) {
              tc::tma_load_2d_pair(to + at, &P.map[kW1], fbar, kb * kBK, wrow);
            });
          }
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
      // A stage's MMAs.  This thread's own latency counts: a wait takes 200
      // cycles even on a barrier that is complete, so the next stage's is
      // looked at before this one's MMAs are issued, under those still running
      // (1 to 2 % at every size), and what does not change from stage to stage
      // is kept out of here.  The look may suspend the thread for a while: when
      // the ring is dry, and at a pair's last stage, which no other follows,
      // MMAs that could start wait with it.
      auto issue = [&](uint32_t dst, uint64_t a0, uint64_t b0, uint64_t as, uint64_t bs, uint32_t idesc, int ng,
                       uint32_t accumulate) {
        if (!ready && !tc::mbar_wait(bar.full(stage), phase, &s_abort, kWaitNs)) return false;
        const int here = stage;
        advance<kStages>(stage, phase);
        ready = tc::mbar_try_wait(bar.full(stage), phase);
        const uint64_t a = a0 + (uint32_t)(here * (kOperand >> 4)), b = b0 + (uint32_t)(here * (kOperand >> 4));
        tc::mma_bf16_pair(dst, a, b, idesc, accumulate);
#pragma unroll
        for (int k = 1; k < kBK / kGroup; ++k)
          if (k < ng) tc::mma_bf16_pair(dst, a + k * as, b + k * bs, idesc, 1);
        tc::tc_commit_pair_mc(bar.empty(here), 0x3);
        return true;
      };
      Tile next = first < total ? decode(first) : Tile{};
      for (int t = first; t < total && ok; t += step) {
        const Tile d = next;
        const int nk = stages(d), np = products(d), mma_n = d.swap ? (d.nrows + 15) / 16 * 16 : kTile;
        const int full = d.rows ? row_k / kBK : d.nrows / kBK;   // stages of four groups
        for (int sub = 0; sub < np && ok; ++sub) {
          const bool weights_mn = kDa ? sub == 0 : true;
          const bool a_mn = !d.rows || (d.swap && weights_mn), b_mn = !d.rows || (!d.swap && weights_mn);
          const uint32_t idesc = tc::idesc_bf16_f32(kTile, mma_n) | (a_mn ? kMajorA : 0u) | (b_mn ? kMajorB : 0u);
          if (!tc::mbar_wait(bar.tempty(acc), acc_phase ^ 1u, &s_abort, kWaitNs)) { ok = false; break; }
          tc::tc_fence_after();
          const uint32_t dst = tmem + (uint32_t)(acc * kTile);
          // a descriptor's address is in units of 16 bytes, and no operand leaves its field
          const uint64_t a0 = a_mn ? sdesc_mn128(sA) : tc::sdesc_k128(sA), as = (a_mn ? kStepMN : kStepK) >> 4;
          const uint64_t b0 = b_mn ? sdesc_mn128(sB) : tc::sdesc_k128(sB), bs = (b_mn ? kStepMN : kStepK) >> 4;
          int kb = 0;
#pragma unroll 1
          for (; kb < full && ok; ++kb) ok = issue(dst, a0, b0, as, bs, idesc, kBK / kGroup, kb != 0);
          // the next tile's divisions run beside the MMAs issued so far
          if (sub == np - 1 && t + step < total) next = decode(t + step);
#pragma unroll 1
          for (; kb < nk && ok; ++kb) ok = issue(dst, a0, b0, as, bs, idesc, groups(d, kb, nk), kb != 0);
          if (!ok) break;
          tc::tc_commit_pair_mc(bar.tfull(acc), 0x3);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      if (!ok) give_up(P.err, &s_abort);
      tc::tc_commit_pair_mc(bar.done(), 0x3);   // both CTAs learn when every MMA has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q .. 32 q + 31 belong to this warp
    const uint32_t buf = sOut + (warp - 2) * kStoreBytes;
    uint8_t* row = smem_raw + (buf - tc::smem_u32(smem_raw)) + lane * 128;
    float4* st = kDa ? stash_of(P.stash, warp - 2, lane) : nullptr;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const Tile d = decode(t);
      const int np = products(d);
      const uint64_t limit = kWaitNs + (uint64_t)stages(d) * kStageNs;
      for (int sub = 0; sub < np; ++sub) {
        if (!__all_sync(0xffffffffu, tc::mbar_wait(bar.tfull(acc), acc_phase, &s_abort, limit))) {
          give_up(P.err, &s_abort);
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile);
        if (kDa) {
          if (d.swap && sub < np - 1) stash_swapped(tbase, d, half, sub, st);
          else if (d.swap) da_swapped<kSwi>(tbase, d, rank, q, half, lane, P, st);
          else if (sub == 0) stash_rows<kSwi>(tbase, d, half, P.F, st);
          else da_rows<kSwi>(tbase, d, sub - 1, rank, q, half, lane, P, st);
        } else if (d.rows) {
          dx_tile(tbase, d, rank, q, half, lane, P);
        } else {
          weight_tile(tbase, d, d.nrows == 0, rank, q, half, lane, P, buf, row);
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) tc::mbar_arrive(bar.tempty(acc));
          else tc::mbar_arrive_remote_relaxed(tc::map_peer(bar.tempty(acc), 0));
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }
  tc::tc_fence_before();
  __syncthreads();
  // Every MMA has finished before the CTAs part.  Asked for only now that this
  // CTA's roles are done: warp 1 of the pair's other CTA has no role, and
  // waiting from the start it would hold the launch, not a wait, to the limit.
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(bar.done(), 0, nullptr, kWaitNs)) set_error(P.err, kDevTimeout);
    __syncwarp();
  }
  // after an abort the leader drains its stage barriers, on which both CTAs'
  // loads complete, before either CTA may leave; loads into a stage that it
  // had not armed yet are given a millisecond to land
  if (producer && s_abort) {
    if (rank == 0)
      for (int s = 0; s < kStages; ++s)
        if ((filled >> s) & 1u) tc::mbar_wait(bar.full(s), (fill_par >> s) & 1u, nullptr, kWaitNs);
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

// One persistent launch of CTA pairs.
template <int kJob>
cudaError_t launch_pairs(const Params& P, cudaStream_t st) {
  auto kern = backward_pair_kernel<kJob>;
  const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (r != cudaSuccess) return r;
  const int pairs = sm_count() / 2;
  return launch_kernel(kern, dim3((unsigned)(2 * (pairs < kMaxPairs ? pairs : kMaxPairs))), dim3(kThreads), kSmem, st, 2,
                       P);
}

// Whether every row of [.., cols] bf16 elements starts on a 32-byte sector.
bool starts_on_sectors(const void* p, int cols) { return ((uintptr_t)p % 32 == 0) && (cols % 16 == 0); }

}  // namespace

int64_t backward_blocks(int64_t rows, int E) { return rows / kTile + E + 1; }
size_t backward_stash_floats() { return (size_t)2 * kMaxPairs * kStash; }
size_t backward_tail_bytes(int E, int H, int N, int F) {
  return (size_t)E * kGroup * ((size_t)N + 2 * (size_t)H + (size_t)F) * sizeof(bf16);
}

cudaError_t launch_ffn_backward_tc(const Shape& s, int64_t max_rows, const FfnBackward& b, void* da, float* stash,
                                   float* part, void* tails, int* err, cudaStream_t st) {
  const bool swi = (s.flags & MOE_FLAG_SWIGLU) != 0;
  const int N = swi ? 2 * s.F : s.F;
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
  const uint64_t R = (uint64_t)max_rows, E = (uint64_t)s.E, H = (uint64_t)s.H, F = (uint64_t)s.F, n = (uint64_t)N;
  Params P = {};
  P.offs = b.offs;
  P.E = s.E;
  P.H = s.H;
  P.F = s.F;
  P.N = N;
  P.da = (bf16*)da;
  P.err = err;
  P.stall = (s.flags & MOE_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
  const bool hidden = b.dx_perm || b.dW1 || b.db1;   // what needs da
  if (hidden) {
    P.stash = stash;
    P.b1 = b.b1;
    P.part = b.db1 ? part : nullptr;
    P.sectors = starts_on_sectors(da, s.F);
    if (!tma_map_bf16(&P.map[kDy], b.dy_perm, R, H, kBM) || !tma_map_bf16(&P.map[kDyBox], b.dy_perm, R, H, kBoxRows) ||
        !tma_map_bf16_3d(&P.map[kW2], b.W2, E, H, F, kBK) || !tma_map_bf16(&P.map[kX], b.x_perm, R, H, kBM) ||
        !tma_map_bf16(&P.map[kXBox], b.x_perm, R, H, kBoxRows) || !tma_map_bf16(&P.map[kW1], b.W1, E * n, H, kBM))
      return cudaErrorNotSupported;
    e = swi ? launch_pairs<kDaSwiglu>(P, st) : launch_pairs<kDaGelu>(P, st);
    if (e != cudaSuccess) return e;
  }
  Extras x = {};
  int nw = 0;   // weight products
  bf16* at = (bf16*)tails;
  auto add = [&](const void* A, int M, const void* Bm, int Nn, void* dW) {
    const void* rows[2] = {A, Bm};
    const int cols[2] = {M, Nn};
    CUtensorMap* m = &P.map[kWeightMaps + 4 * nw];
    bool ok = tma_map_bf16_3d(&P.map[kOutMaps + nw], dW, E, (uint64_t)M, (uint64_t)Nn, 32);
    for (int i = 0; i < 2; ++i) {
      x.o[2 * nw + i] = {(const uint4*)rows[i], (uint4*)at, cols[i] / 8};
      ok = ok && tma_map_bf16(m + i, rows[i], R, (uint64_t)cols[i], kBK) &&
           tma_map_bf16(m + 2 + i, at, E * kGroup, (uint64_t)cols[i], kGroup);
      at += (int64_t)s.E * kGroup * cols[i];
    }
    P.wm[nw] = M;
    P.wn[nw] = Nn;
    ++nw;
    return ok;
  };
  if (b.dW1 && !add(da, N, b.x_perm, s.H, b.dW1)) return cudaErrorNotSupported;
  if (b.dW2 && !add(b.dy_perm, s.H, b.h_perm, s.F, b.dW2)) return cudaErrorNotSupported;
  x.tails = 2 * nw * kTailSplit * s.E;
  x.part = part;
  x.db1 = b.db1;
  x.n = N;
  x.cols1 = (N + kRedCols - 1) / kRedCols;
  x.db1_blocks = b.db1 ? x.cols1 * s.E : 0;
  x.dy = (const uint4*)b.dy_perm;
  x.db2 = b.db2;
  x.h = s.H;
  x.cols2 = b.db2 ? (s.H / 8 + kSumVecs - 1) / kSumVecs : 0;
  const int64_t extras = (int64_t)x.tails + x.db1_blocks + (int64_t)x.cols2 * s.E;
  if (extras > 0)
    e = launch_kernel(backward_extras_kernel, dim3((unsigned)extras), dim3(256), 0, st, 1, x, b.offs, s.E);
  if (e != cudaSuccess || !(b.dx_perm || nw > 0)) return e;
  P.dx = (bf16*)b.dx_perm;
  P.sectors = starts_on_sectors(b.dx_perm, s.H);
  if (b.dx_perm && (!tma_map_bf16(&P.map[kDaRows], da, R, n, kBM) || !tma_map_bf16(&P.map[kDaBox], da, R, n, kBoxRows) ||
                    !tma_map_bf16_3d(&P.map[kW1MN], b.W1, E, n, H, kBK)))
    return cudaErrorNotSupported;
  return launch_pairs<kGradients>(P, st);
}

}  // namespace moe
