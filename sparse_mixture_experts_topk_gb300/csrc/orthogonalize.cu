// Matrices made nearly orthogonal by Newton-Schulz products, and the Muon step
// around them.
//
// For a matrix u, X = u / |u| (Frobenius norm), its short side as rows (s <= L):
//   A = X X^T,  B = a I + b A + c A A,  X <- B X      `iterations` times
// B is a polynomial of the symmetric A, so A and B are symmetric: their tiles
// below the diagonal are the mirrored ones above it and are not computed.
//
// X, A and B are held in fp16 times 2^12 (but in fp32 on the CUDA cores for a
// short side of up to 16, see small_kernel).  Their values are at most 1.21, 1.46
// and 3.45 in magnitude (no singular value passes 1.21), those of a product of
// two B at most 11.9 of the 15.9 that fit, and nothing above 2^-26 loses bits;
// fp16 has three bits more than bf16 at the same rate of the tensor cores.
// Rounded to bf16 instead, the result is 1.1 % off (in the 2-norm, for a
// gradient of four strong directions over noise), with fp16 0.13 %.
//
// All products of a call are one launch: running CTAs take tiles by number from
// a counter, step after step, and a tile starts once every tile of its matrix'
// step before is written (a counter for each step and matrix).  A tile waits for
// lower numbers only, and those are taken by CTAs that run: no CTA needs
// another one to be resident.  Launched one by one, the steps of a few small
// matrices took twice as long, and those of many large ones lost their tails.
//
// Tiles are 256 x 256 on SM pairs (tcgen05 .cta_group::2), or 256 x 128 where
// those would leave SMs idle; fp32 accumulators in TMEM, operands staged by TMA.
// A and the short products read both operands along their rows; X as the second
// operand of B X is read as it lies ("MN-major").
//
// What bounds it: 64 elements of a reduction take a tile's MMAs 512 cycles on a
// pair, and the 32 KB for each SM that go with them as long at the 64 bytes a
// cycle that L2 gives an SM (half a tile loads 24 KB); with few matrices the
// latency of a step, 7 us beside its MMAs.
// Measured: a Muon step on 16 matrices of 2560 x 3584 (6.3 TFLOP in the order
// below) 4.7 to 5.1 ms, 0.25 of them before the products, on 48 of 1408 x 4096
// 4.7 to 5.0 and 0.47; 3 matrices of 1416 x 1001 201 us, 16 of 256 x 512 102 us,
// one of 64 x 96 18 us.
//
// Roles per CTA: warps 0 and 10 TMA producers, one for each operand, warp 1
// MMA issuer (leader CTA of a pair), warps 2-9 epilogue.  Every wait is
// bounded: on expiry the kernel records a timeout in the workspace's error
// word, drains what it has in flight, frees its tensor memory and returns.
#include <algorithm>

#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;   // the quintic's coefficients
constexpr float kHeld = 4096.f;                              // factor of every value held in fp16

// ---------------------------------------------------------------- the tensors

// A part of a tensor: matrices of it, which are matrices `first` and on of the
// ones at hand, up to the next segment's.
struct Segment {
  float* p;
  bf16* p16;
  const void* g;
  float* m;
  void* out;             // raw: receives the result
  int rows, cols;
  int first;
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

// Four elements of p, of which `left` exist, from e on, to go with put4; nothing for raw.
__device__ __forceinline__ void get4(const Matrices& M, const Segment& S, int64_t e, bool even, int left, float* p) {
  if (!M.raw) load4(S.p + e, even && aligned_to(S.p + e, 16), left, p);
}
// p = p keep - step o there, and its bf16 copy; raw: out = o.
__device__ __forceinline__ void put4(const Matrices& M, const Segment& S, int64_t e, bool even, int left, const float* p,
                                     const float* o) {
  if (M.raw) {
    if (M.out_dtype == MOE_BF16) {
      bf16* to = reinterpret_cast<bf16*>(S.out) + e;
      store4(to, even && aligned_to(to, 8), left, o);
    } else {
      float* to = reinterpret_cast<float*>(S.out) + e;
      store4(to, even && aligned_to(to, 16), left, o);
    }
    return;
  }
  float v[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = p[x] * S.keep - S.step * o[x];
  store4(S.p + e, even && aligned_to(S.p + e, 16), left, v);
  if (S.p16) store4(S.p16 + e, even && aligned_to(S.p16 + e, 8), left, v);
}

// ---------------------------------------------------------------- products

constexpr int kRows = 256;                // of a tile
constexpr int kBM = 128;                  // of them in a CTA
constexpr int kBox = 64;                  // reduction elements of a box
constexpr int kSub = 2;                   // boxes of an operand in a stage
constexpr int kBK = kSub * kBox;          // reduction elements per stage
constexpr int kGroup = 16;                // reduction elements per MMA
constexpr int kBlock = kBM * kBox * 2;    // bytes of 128 rows of a box
constexpr int kOperand = kSub * kBlock;   // and of a's in a stage
constexpr int kHalf = kBlock / 2;         // a box of 64 columns x 64 rows: b read across is made of those
constexpr int kRing = 6 * 2 * kBlock;     // bytes of all stages
constexpr int kEpiWarps = 8;              // per CTA: two for each quarter of the TMEM lanes
constexpr int kThreads = 64 + 32 * kEpiWarps + 32, kSecondProducer = 2 + kEpiWarps;
constexpr int kStoreBytes = 32 * 128;     // an epilogue warp's 32 rows of 64 columns on their way to TMA, or their transpose
constexpr size_t kSmem = 1024 + (size_t)kRing + kEpiWarps * kStoreBytes;
// The limit of a wait, and what it has on top for each stage of the tiles that a CTA has of a step: those may
// have to be written first.
constexpr uint64_t kWaitNs = 2000000000ull, kStageNs = 2000;
constexpr int kQueue = 16, kNoTile = -1, kAborted = -2;

// MN-major operand: boxes of 64 columns (128 bytes, 128-byte swizzle) and 64 rows one after the other.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr) {
  return tc::sdesc_k128(saddr) | ((uint64_t)(kHalf >> 4) << 16);
}
constexpr uint32_t kMajorB = 1u << 16;       // instruction descriptor: B is MN-major
constexpr int kStepK = 32, kStepMN = 2048;   // bytes from one group of 16 to the next
// Instruction descriptor of kind::f16: D fp32, A and B fp16 (formats 0), K-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The buffers: X and its successor [s, L], three symmetric matrices [s, s].
enum Buffer : int8_t { kX = 0, kY, kG, kP, kQ, kBuffers, kNone = -1 };

// out = alpha a b^T + beta add + diag I, or, where b is X (read as it lies), alpha a b.
struct Step {
  Buffer a, b, out, add;
  bool gram;         // a = b = X: the reduction is over L
  int8_t opens;      // operands that are the X before the first step, off by its correction
  float alpha, beta, diag;
  __host__ __device__ bool wide() const { return out <= kY; }   // else out is symmetric: tiles from the diagonal on
  __host__ __device__ bool mn() const { return out <= kY; }
};
constexpr int kMaxSteps = 7 * MOE_ORTHOGONALIZE_MAX_ITERATIONS / 2;

// X as it is held before the first step: u times a times b, times which `correction` it is u / |u| 2^12.
struct Scale {
  float a, b, correction;
  int build;   // not written yet
};

struct Chain {
  CUtensorMap along[kBuffers];   // boxes of 128 rows of 64 elements
  CUtensorMap across[kBuffers];  // 64 rows of 64 elements
  CUtensorMap store[kBuffers];   // 32 rows of 64 elements
  CUtensorMap mirror[kBuffers];  // the symmetric ones: 64 rows of 32 elements, not swizzled
  __half* buf[kBuffers];
  int s, L, batch, steps;
  int64_t pitch, plane, square, square_plane;   // elements of a row and of a matrix
  Step step[kMaxSteps];
  int* written;                  // [steps, batch] zeros: warps that have written their share of a tile
  int* next;                     // zero: the first tile that nobody has taken
  const Scale* scale;            // of each matrix
  bool beside;                   // launches that run beside this one follow
  uint64_t limit;
  const int32_t* skip;
  int* err;
  bool stall;   // testing: each pair's waits run out in one of three ways
};

// The tiles of a chain in the order in which they are taken.
// kN: columns of a tile.
template <int kN>
struct Tiles {
  static constexpr int kSteps = kRows / kN;   // tiles beside the diagonal in a row of them
  const Chain& C;
  int mt, nt, nL;      // rows of tiles, and columns over s and L
  int p, per;          // the step at hand, and its tiles of a matrix
  int64_t base;        // the first of its tiles (all are below 2^31: see Sizes::most)
  int matrix, m0, n0;
  __device__ explicit Tiles(const Chain& c)
      : C(c), mt((c.s + kRows - 1) / kRows), nt((c.s + kN - 1) / kN), nL((c.L + kN - 1) / kN), p(0), base(0) {
    per = tiles(0);
  }
  __device__ int tiles(int step) const {
    return C.step[step].wide() ? mt * nL : mt * nt - kSteps * (mt * (mt - 1) / 2);
  }
  // Tile t, not before the last one asked for; false behind the last.
  __device__ bool seek(int64_t t) {
    while (t >= base + (int64_t)per * C.batch) {
      base += (int64_t)per * C.batch;
      if (++p == C.steps) return false;
      per = tiles(p);
    }
    const uint32_t local = (uint32_t)(t - base);
    matrix = (int)(local / (uint32_t)per);
    int i = 0, j = (int)(local % (uint32_t)per);
    if (C.step[p].wide()) {
      i = j % mt;
      j /= mt;
    } else {
      while (j >= nt - kSteps * i) {   // those of row i from the diagonal on
        j -= nt - kSteps * i;
        ++i;
      }
      j += kSteps * i;
    }
    m0 = i * kRows;
    n0 = j * kN;
    return true;
  }
  __device__ int k() const { return C.step[p].gram ? C.L : C.s; }
  __device__ int cols() const { return C.step[p].wide() ? C.L : C.s; }
  // Columns of an MMA: those that the tile has, to 16; to whole groups of 64 for each CTA where b is read across
  __device__ int mma_n() const {
    const int to = C.step[p].mn() ? 128 : 16;
    return min(kN, (cols() - n0 + to - 1) / to * to);
  }
};

template <int kStages>
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

// Wait (bounded) until the counter reaches `need`; what was written before is
// then visible to this thread's loads and to the tensor copies it issues.
__device__ __forceinline__ bool wait_written(const int* counter, int need, volatile int* abort, uint64_t limit) {
  const uint64_t t0 = tc::globaltimer();
  while (true) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
    if (v >= need) {
      asm volatile("fence.proxy.async.global;" ::: "memory");
      return true;
    }
    if (*abort || tc::globaltimer() - t0 > limit) return false;
  }
}

// 32 rows and 64 columns of the result, from (row0, col) of X on, to the
// tensor, by one warp: turned through its buffer so that the lanes' accesses lie
// along the tensor's rows.  packed: this lane's row, as held.  kWhole: with a
// loop of its own for what lies inside the tensor (where the epilogue's
// instructions count; cold code costs a few short products 2 %).
template <bool kWhole>
__device__ __forceinline__ void finish(const Matrices& M, const Segment& S, int64_t base, uint8_t* buf,
                                       const uint32_t (&packed)[2][16], int row0, int col, int lane) {
  const bool flip = S.rows > S.cols, even = S.cols % 4 == 0;
  __half* tile = reinterpret_cast<__half*>(buf);
  __syncwarp();   // the lanes have read the tile before
  if (flip) {
    // 64 rows of 32 of the tensor; 8 bytes of a row exchanged by its number
#pragma unroll
    for (int j = 0; j < 64; ++j)
      reinterpret_cast<uint16_t*>(tile)[j * 32 + ((((lane >> 2) ^ (j & 7)) << 2) | (lane & 3))] =
          (uint16_t)(packed[j >> 5][(j & 31) >> 1] >> (16 * (j & 1)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)   // 32 rows of 64; 16 bytes of a row exchanged by its number
      *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
          make_uint4(packed[j >> 2][j % 4 * 4], packed[j >> 2][j % 4 * 4 + 1], packed[j >> 2][j % 4 * 4 + 2],
                     packed[j >> 2][j % 4 * 4 + 3]);
  }
  __syncwarp();
  // four elements of a row to a lane, 16 or 8 lanes to a row; eight loads in flight
  const int tr0 = flip ? col : row0, tc0 = flip ? row0 : col, along = flip ? 8 : 16;
  if (kWhole && !M.raw && even && aligned_to(S.p, 16) && aligned_to(S.p16, 8) && tr0 + 512 / along <= S.rows &&
      tc0 + 4 * along <= S.cols) {
    // all of it lies inside: with the bounds and alignments of each group
    // checked, the instructions of this took longer than a tile's MMAs
    const int r = lane / along, x = lane % along;
    const int64_t e = base + (int64_t)(tr0 + r) * S.cols + tc0 + x * 4, step = (int64_t)(32 / along) * S.cols;
    float4* p = reinterpret_cast<float4*>(S.p + e);
    uint2* p16 = S.p16 ? reinterpret_cast<uint2*>(S.p16 + e) : nullptr;
    const float keep = S.keep, by = S.step * (1.f / kHeld);
#pragma unroll 1
    for (int i0 = 0; i0 < 16; i0 += 8) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldcs(p + (i0 + i) * step / 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (i0 + i) * (32 / along) + r;
        const uint2 u = *reinterpret_cast<const uint2*>(
            buf + (flip ? row * 64 + ((x ^ (row & 7)) << 3) : row * 128 + (((x >> 1) ^ (row & 7)) << 4) + (x & 1) * 8));
        const __half2* h = reinterpret_cast<const __half2*>(&u);
        const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
        v[i] = make_float4(v[i].x * keep - by * a.x, v[i].y * keep - by * a.y, v[i].z * keep - by * b.x,
                           v[i].w * keep - by * b.y);
        __stcs(p + (i0 + i) * step / 4, v[i]);
        if (p16) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v[i].x, v[i].y), hi = __floats2bfloat162_rn(v[i].z, v[i].w);
          __stcs(p16 + (i0 + i) * step / 4,
                 make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi)));
        }
      }
    }
    return;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 8) {
    float p[8][4];
    int64_t e[8];
    int left[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = (i0 + i) * 32 + lane, r = flip ? at / 8 : at / 16, x = flip ? at % 8 : at % 16;
      const int tr = (flip ? col : row0) + r, tc = (flip ? row0 : col) + x * 4;
      left[i] = tr < S.rows ? min(4, S.cols - tc) : 0;
      e[i] = base + (int64_t)tr * S.cols + tc;
      if (left[i] > 0) get4(M, S, e[i], even, left[i], p[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (left[i] <= 0) continue;
      const int at = (i0 + i) * 32 + lane, r = flip ? at / 8 : at / 16, x = flip ? at % 8 : at % 16;
      const uint2 u = *reinterpret_cast<const uint2*>(
          buf + (flip ? r * 64 + ((x ^ (r & 7)) << 3) : r * 128 + (((x >> 1) ^ (r & 7)) << 4) + (x & 1) * 8));
      const __half2* h = reinterpret_cast<const __half2*>(&u);
      const float2 a = __half22float2(h[0]), b = __half22float2(h[1]);
      const float o[4] = {a.x * (1.f / kHeld), a.y * (1.f / kHeld), b.x * (1.f / kHeld), b.y * (1.f / kHeld)};
      put4(M, S, e[i], even, left[i], p[i], o);
    }
  }
}

// Tiles of 256 x kN on the two CTAs of a cluster.
template <int kN>
__global__ void __launch_bounds__(kThreads, 1)
chain_kernel(const __grid_constant__ Chain C, const __grid_constant__ Matrices M) {
  constexpr int kChunks = kN / 128;   // of 64 columns, for each of a lane quarter's two epilogue warps
  constexpr int kBlockB = kN / 2 * kBox * 2, kOperandB = kSub * kBlockB;   // b's part in a CTA, as kBlock and kOperand
  constexpr int kStages = kRing / (kOperand + kOperandB);
  constexpr uint32_t kTmemCols = 2 * kN;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ unsigned long long s_queue[kQueue], s_copies[4];
  __shared__ uint32_t s_gave_up[2];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 5];
  const uint32_t sA = (tc::smem_u32(smem_raw) + 1023u) & ~1023u, sB = sA + kStages * kOperand;
  const uint32_t sOut = sB + kStages * kOperandB;
  const uint32_t bars = tc::smem_u32(s_bar);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto tfull = [&](int a) { return bars + 8 * (2 * kStages + a); };
  auto tempty = [&](int a) { return bars + 8 * (2 * kStages + 2 + a); };
  const uint32_t done = bars + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)tc::cluster_ctarank();
  auto commit = [&](uint32_t bar) {
    tc::tc_commit_pair_mc(bar, 0x3);
  };

  // What comes after the call waits for the end of this kernel: a next call's few
  // first blocks, started beside it, made it slower (steps on 8 matrices of 1024 x
  // 1024 one after another 85 -> 121 us, 16 of 256 x 512 101 -> 110).
  pdl_wait();
  if (C.beside) pdl_trigger();
  if (C.skip && *C.skip) return;   // every thread of both CTAs
  // testing: 1 = the first stage's barrier waits for an arrival that nobody makes; the first producer gives up
  // before it has published a tile (2) or loaded one (3), so that the other CTA's roles, or its copies, are left alone
  const int stall = C.stall ? 1 + blockIdx.x / 2 % 3 : 0;
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        tc::mbar_init(full(s), s == 0 && stall == 1 ? 2 : 1);
        tc::mbar_init(empty(s), 1);
      }
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(tfull(a), 1);
        tc::mbar_init(tempty(a), 2 * kEpiWarps);   // one arrival for each epilogue warp of the pair
      }
      tc::mbar_init(done, 1);
      for (int i = 0; i < kQueue; ++i) s_queue[i] = 0;
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
  Tiles<kN> T(C);
  // The leader's first producer takes tiles and publishes each, or kNoTile at
  // the end, as an entry of a queue in both CTAs; the other roles read it there.
  // No role is kQueue tiles behind: two accumulators and kStages stages at most.
  auto publish = [&](int seq, int t) {
    const unsigned long long v = (unsigned long long)(unsigned)(seq + 1) << 32 | (unsigned)t;
    *(volatile unsigned long long*)&s_queue[seq % kQueue] = v;
    tc::st_peer_u64(tc::map_peer(tc::smem_u32(&s_queue[seq % kQueue]), 1), v);
  };
  auto read = [&](int seq) {   // kAborted if it does not come
    volatile unsigned long long* slot = &s_queue[seq % kQueue];
    const uint64_t t0 = tc::globaltimer();
    while (true) {
      const unsigned long long v = *slot;
      if ((v >> 32) == (unsigned)(seq + 1)) return (int)(unsigned)v;
      if (s_abort || tc::globaltimer() - t0 > C.limit) return (int)kAborted;
    }
  };
  // the counter of the step before a tile's, and what it has to reach
  auto before = [&]() { return C.written + (int64_t)(T.p - 1) * C.batch + T.matrix; };
  auto need = [&]() { return T.tiles(T.p - 1) * 2 * kEpiWarps; };

  uint32_t filled = 0, fill_par = 0;   // a producer's: stages filled, and the parity of each one's latest
  if (warp == 0 || warp == kSecondProducer) {
    // ------------------------------------------------------------ TMA producers (both CTAs)
    const bool second = warp == kSecondProducer;
    if (tc::elect_one()) {
      int stage = 0, seen_p = 0, seen_m = -1;   // a step and matrix whose operands are known to be written
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t to = second ? sB : sA;
      const bool takes = rank == 0 && !second;
      for (int seq = 0; ok; ++seq) {
        int t;
        if (takes && stall == 2) {
          ok = false;
          break;
        }
        if (takes) {
          // not ahead of time: while it waited here another CTA could have started it
          t = atomicAdd(C.next, 1);
          if (!T.seek(t)) t = kNoTile;
          publish(seq, t);
        } else {
          t = read(seq);
          if (t >= 0) T.seek(t);
        }
        ok = t != kAborted && !(takes && stall == 3);
        if (t < 0 || !ok) break;
        if (T.p > 0 && (T.p != seen_p || T.matrix != seen_m)) {
          ok = wait_written(before(), need(), &s_abort, C.limit);
          if (!ok) break;
          seen_p = T.p;
          seen_m = T.matrix;
        }
        const Step& S = C.step[T.p];
        const bool mn = second && S.mn();
        // b's part of a tile of 128 columns is 64 rows, too
        const CUtensorMap* map = mn || (second && kN == 128) ? &C.across[S.b] : &C.along[second ? S.b : S.a];
        // b's columns are split evenly between the CTAs
        const int r = second ? T.n0 + rank * (T.mma_n() / 2) : T.m0 + rank * kBM;
        const int nk = (T.k() + kBK - 1) / kBK;
        for (int kb = 0; kb < nk; ++kb) {
          if (!tc::mbar_wait(empty(stage), phase ^ 1u, &s_abort, C.limit)) {
            ok = false;
            break;
          }
          if (rank == 0 && !second) tc::mbar_arrive_expect_tx(full(stage), 2 * (kOperand + kOperandB));
          const uint32_t at = to + stage * (second ? kOperandB : kOperand);
          auto load = [&](uint32_t dst, int c0, int c1) {
            tc::tma_load_3d_pair(dst, map, tc::map_peer(full(stage), 0), c0, c1, T.matrix);
          };
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            const int k = kb * kBK + u * kBox;
            if (mn) {
              load(at + u * kBlockB, r, k);
              if (kN == 256) load(at + u * kBlockB + kHalf, r + 64, k);
            } else {
              load(at + u * (second ? kBlockB : kBlock), k, r);
            }
          }
          filled |= 1u << stage;
          fill_par = (fill_par & ~(1u << stage)) | (phase << stage);
          advance<kStages>(stage, phase);
        }
      }
      if (!ok) give_up(C.err, &s_abort);
      tc::st_peer_u64(tc::map_peer(tc::smem_u32(&s_copies[rank * 2 + second]), 0),
                      (unsigned long long)fill_par << 32 | filled);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (rank == 0 && tc::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;   // ready: the stage at hand was seen full
      const uint64_t a0 = tc::sdesc_k128(sA);
      for (int seq = 0; ok; ++seq) {
        const int t = read(seq);
        ok = t != kAborted;
        if (t < 0) break;
        T.seek(t);
        const bool mn = C.step[T.p].mn();
        const uint64_t b0 = mn ? sdesc_mn128(sB) : tc::sdesc_k128(sB);
        const uint32_t as = kStepK >> 4, bs = (mn ? kStepMN : kStepK) >> 4;
        const uint32_t idesc = idesc_f16_f32(kRows, T.mma_n()) | (mn ? kMajorB : 0u);
        const int k = T.k(), nk = (k + kBK - 1) / kBK;
        if (!tc::mbar_wait(tempty(acc), acc_phase ^ 1u, &s_abort, C.limit)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t dst = tmem + (uint32_t)(acc * kN);
#pragma unroll 1
        for (int kb = 0; kb < nk; ++kb) {
          if (!ready && !tc::mbar_wait(full(stage), phase, &s_abort, C.limit)) {
            ok = false;
            break;
          }
          const int here = stage, ng = min(kBK / kGroup, (k - kb * kBK + kGroup - 1) / kGroup);
          advance<kStages>(stage, phase);
          // looked at under the MMAs still running (the wait itself costs 200 cycles)
          ready = tc::mbar_test_wait(full(stage), phase);
          const uint64_t a = a0 + (uint32_t)(here * (kOperand >> 4)), b = b0 + (uint32_t)(here * (kOperandB >> 4));
#pragma unroll
          for (int g = 0; g < kBK / kGroup; ++g) {
            if (g < ng) {
              const uint32_t sub = g / (kBox / kGroup), in = g % (kBox / kGroup);
              tc::mma_bf16_pair(dst, a + sub * (kBlock >> 4) + in * as, b + sub * (kBlockB >> 4) + in * bs, idesc, g || kb);
            }
          }
          commit(empty(here));
        }
        if (!ok) break;
        commit(tfull(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) give_up(C.err, &s_abort);
      commit(done);   // both CTAs learn when every MMA has finished
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;   // TMEM lanes 32 q .. 32 q + 31 belong to this warp
    const uint32_t buf = sOut + (warp - 2) * kStoreBytes;
    uint8_t* mine = smem_raw + (buf - tc::smem_u32(smem_raw));
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int seq = 0;; ++seq) {
      const int t = __shfl_sync(0xffffffffu, lane == 0 ? read(seq) : 0, 0);
      if (t == kAborted) give_up(C.err, &s_abort);
      if (t < 0) break;
      T.seek(t);
      const Step& S = C.step[T.p];
      const int cols = T.cols(), row0 = T.m0 + rank * kBM + q * 32, row = row0 + lane;
      const bool mirror = !S.wide() && T.n0 >= T.m0 + kRows;
      float alpha = S.alpha;
      if (S.opens) {
        const float by = C.scale[T.matrix].correction;
        alpha *= S.opens == 2 ? by * by : by;
      }
      const __half* add = S.add >= 0 && row < C.s
                              ? C.buf[S.add] + T.matrix * C.square_plane + row * C.square : nullptr;
      // 32 elements of the addend; rows are padded to 8: a vector that starts inside the row lies inside it
      auto fetch = [&](int col, uint4* v) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          v[g] = add && col + g * 8 < cols ? __ldcg(reinterpret_cast<const uint4*>(add + col + g * 8))
                                           : make_uint4(0u, 0u, 0u, 0u);
      };
      uint4 ahead[4];
      const int first_col = T.n0 + half * kChunks * 64;
      bool ok = true;
      if (S.add >= 0) {
        ok = wait_written(before(), need(), &s_abort, C.limit);   // long since: the operands are
        fetch(first_col, ahead);
      }
      ok = ok && tc::mbar_wait(tfull(acc), acc_phase, &s_abort, C.limit);
      if (!__all_sync(0xffffffffu, ok)) {
        give_up(C.err, &s_abort);
        break;
      }
      tc::tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kN + half * kChunks * 64);
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        const int col = first_col + c * 64;
        uint32_t packed[2][16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tc::tmem_ld_32x32b_x32(tbase + c * 64 + h * 32, r);
          if (S.add < 0) {
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __half2 f = __floats2half2_rn(alpha * __uint_as_float(r[2 * j]), alpha * __uint_as_float(r[2 * j + 1]));
              packed[h][j] = *reinterpret_cast<const uint32_t*>(&f);
            }
            continue;
          }
          uint4 more[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) more[g] = ahead[g];
          if (h == 0 || c + 1 < kChunks) fetch(col + (h + 1) * 32, ahead);
          tc::tmem_wait_ld();
          const int diagonal = row - col - h * 32;   // the column of diag I, if it is one of these
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float2 m = __half22float2(reinterpret_cast<const __half2*>(more)[j]);
            const float x = fmaf(S.beta, m.x, S.alpha * __uint_as_float(r[2 * j])) + (diagonal == 2 * j ? S.diag : 0.f);
            const float y =
                fmaf(S.beta, m.y, S.alpha * __uint_as_float(r[2 * j + 1])) + (diagonal == 2 * j + 1 ? S.diag : 0.f);
            const __half2 f = __floats2half2_rn(x, y);
            packed[h][j] = *reinterpret_cast<const uint32_t*>(&f);
          }
        }
        if (c == kChunks - 1) {   // tensor memory has been read
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (rank == 0) tc::mbar_arrive(tempty(acc));
            else tc::mbar_arrive_remote_relaxed(tc::map_peer(tempty(acc), 0));
          }
        }
        if (row0 >= C.s || col >= cols) continue;
        // The tile leaves through shared memory by TMA, which writes what lies
        // inside the matrix; stored by its threads, a row each and the mirrored
        // elements one by one, a short product's tile took longer than its MMAs.
        if (T.p == C.steps - 1) {
          // the result goes straight to the tensor
          const Segment& D = segment_of(M, T.matrix);
          finish<kN == 256>(M, D, (int64_t)(T.matrix - D.first) * D.rows * D.cols, mine, packed, row0, col, lane);
          continue;
        }
        if (lane == 0) tc::bulk_wait_read();   // the buffer's previous store has been read
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)   // 16 bytes at the place that the 128-byte swizzle gives them
          *reinterpret_cast<uint4*>(mine + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(packed[j >> 2][j % 4 * 4], packed[j >> 2][j % 4 * 4 + 1], packed[j >> 2][j % 4 * 4 + 2],
                         packed[j >> 2][j % 4 * 4 + 3]);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::tma_store_3d(&C.store[S.out], buf, col, row0, T.matrix);
        if (mirror) {
          if (lane == 0) tc::bulk_wait_read();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 64; ++j)
            reinterpret_cast<uint16_t*>(mine)[j * 32 + lane] = (uint16_t)(packed[j >> 5][(j & 31) >> 1] >> (16 * (j & 1)));
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::tma_store_3d(&C.mirror[S.out], buf, row0, col, T.matrix);
        }
      }
      if (lane == 0 && T.p < C.steps - 1) {
        tc::bulk_wait_all();   // written, and ...
        asm volatile("fence.proxy.async.global;" ::: "memory");
        // ... before the count
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(C.written + (int64_t)T.p * C.batch + T.matrix)
                     : "memory");
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) tc::bulk_wait_all();
  }
  tc::tc_fence_before();
  __syncthreads();
  // every MMA has finished before the CTAs part
  if (warp == 1) {
    if (lane == 0 && !tc::mbar_wait(done, 0, nullptr, kWaitNs)) set_error(C.err, kDevTimeout);
    __syncwarp();
  }
  if (threadIdx.x < 2) tc::st_peer_u32(tc::map_peer(tc::smem_u32(&s_gave_up[rank]), threadIdx.x), (uint32_t)s_abort);
  __syncwarp();                     // the cluster's barrier takes whole warps
  tc::cluster_sync();               // neither CTA leaves while the other may still signal it
  if (s_gave_up[0] | s_gave_up[1]) {
    // After an abort every copy lands before either CTA leaves.  Both CTAs' are
    // counted by the leader's stage barriers; where not all four producers have
    // filled a stage, what is missing is made up for here.
    if (rank == 0 && threadIdx.x == 0)
      for (int s = 0; s < kStages; ++s) {
        const uint32_t parity = tc::mbar_test_wait(full(s), 0) ? 1 : 0;   // of the phase that is not complete
        uint32_t bytes = 0;
        bool armed = false;
        for (int i = 0; i < 4; ++i)
          if ((s_copies[i] >> s & 1) && (s_copies[i] >> (32 + s) & 1) == parity) {
            bytes += i & 1 ? kOperandB : kOperand;
            armed |= i == 0;
          }
        if (!bytes) continue;
        if (!armed) tc::mbar_arrive_expect_tx(full(s), bytes);
        else if (bytes < 2 * (kOperand + kOperandB)) tc::mbar_complete_tx(full(s), 2 * (kOperand + kOperandB) - bytes);
        if (!tc::mbar_wait(full(s), parity, nullptr, kWaitNs)) set_error(C.err, kDevTimeout);
      }
    __syncwarp();
    tc::cluster_sync();
  }
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The steps of `iterations`; the last one's result goes to the tensor.  In pairs:
// with B1 and A1 = (B1 A) B1 the next A without X, and X <- (B2 B1) X once for
// two iterations, three more products of s x s for one X X^T and one B X less.
void plan_steps(Chain& C, int iterations, bool pairs) {
  const float back = 1.f / kHeld;   // what is held is 2^12 times the value: a product of two comes out 2^24 times
  Buffer X = kX, Y = kY;
  bool X0 = true;   // X is the first
  int n = 0;
  auto put = [&](Buffer a, Buffer b, Buffer out) {
    const int8_t opens = (int8_t)((a == X && X0) + (b == X && X0));
    C.step[n++] = Step{a, b, out, kNone, a == b && a <= kY, opens, back, 0.f, 0.f};
  };
  auto polynomial = [&](Buffer out) { C.step[n++] = Step{kG, kG, out, kG, false, 0, kC * back, kB, kA * kHeld}; };
  for (int i = 0; i < iterations;) {
    put(X, X, kG);
    polynomial(kP);
    Buffer apply = kP;
    if (pairs && i + 2 <= iterations) {
      put(kP, kG, kQ);
      put(kQ, kP, kG);
      polynomial(kQ);
      put(kQ, kP, kG);
      apply = kG;
      ++i;
    }
    put(apply, X, Y);
    const Buffer t = X;
    X = Y;
    Y = t;
    X0 = false;
    ++i;
  }
  C.steps = n;
}

template <int kN>
cudaError_t launch_chain(Chain& C, const Matrices& M, int64_t tiles, cudaStream_t st) {
  const int64_t most = sm_count() / 2, pairs = tiles < most ? tiles : most;
  const int64_t stages = (C.L + kBK - 1) / kBK;
  C.limit = kWaitNs + (uint64_t)((tiles / pairs + 2) * stages) * kStageNs;
  auto kern = chain_kernel<kN>;
  const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (r != cudaSuccess) return r;
  return launch_kernel(kern, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmem, st, 2, C, M);
}

// ---------------------------------------------------------------- before the products

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

__device__ __forceinline__ void add_square(Squares& q, float u) {
  const float b = u * kDown, s = u * kUp;
  q.mid = fmaf(u, u, q.mid);
  q.big = fmaf(b, b, q.big);
  q.small = fmaf(s, s, q.small);
}

// The two factors that take u to X as it is held: a power of two first, so that
// no product overflows or vanishes on the way.
__device__ __forceinline__ float2 factors_of(const Squares& q) {
  if (isinf(q.mid)) return isinf(q.big) ? make_float2(NAN, NAN) : make_float2(kDown, kHeld / sqrtf(q.big));
  // a sum above 1e-20 has no share worth mentioning of squares that vanished
  if (!(q.mid <= 1e-20f)) return make_float2(1.f, kHeld / sqrtf(q.mid));   // a NaN too
  return q.small > 0.f ? make_float2(kUp, kHeld / sqrtf(q.small)) : make_float2(0.f, 0.f);
}
// The sum over a block's warps, for thread 0.
__device__ __forceinline__ Squares block_sum(Squares q, Squares* s_w) {
  q = warp_sum(q);
  if (threadIdx.x % 32 == 0) s_w[threadIdx.x / 32] = q;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int w = 1; w < (int)blockDim.x / 32; ++w) {
      q.mid += s_w[w].mid;
      q.big += s_w[w].big;
      q.small += s_w[w].small;
    }
  return q;
}

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
    for (int x = 0; x < 4; ++x)
      if (x < left) add_square(q, u[x]);
  }
  q = block_sum(q, s_w);
  if (threadIdx.x == 0) part[blockIdx.x] = q;
}

// One block for each matrix: its counters to zero, and X's factors.  guess: those
// with which X has been written already; it stays if they are off by a factor
// of 2 at most.
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ Matrices M, const Squares* __restrict__ part,
                                                   const float2* __restrict__ guess, Scale* __restrict__ scale,
                                                   int* __restrict__ written, int steps, int* __restrict__ next) {
  __shared__ Squares s_w[8];
  pdl_enter();
  if (M.skip && *M.skip) return;
  for (int i = threadIdx.x; i < steps; i += 256) written[(int64_t)i * gridDim.x + blockIdx.x] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *next = 0;
  Squares q = {0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = threadIdx.x; i < M.parts; i += 256) {
    const Squares p = part[(int64_t)blockIdx.x * M.parts + i];
    q.mid += p.mid;
    q.big += p.big;
    q.small += p.small;
  }
  q = block_sum(q, s_w);
  if (threadIdx.x == 0) {
    const float2 f = factors_of(q);
    Scale S = {f.x, f.y, 1.f, 1};
    if (guess) {
      const float2 g = guess[blockIdx.x];
      const float by = f.y / g.y;
      if (f.x == g.x && by >= 0.5f && by <= 2.f) S = {g.x, g.y, by, 0};
    }
    scale[blockIdx.x] = S;
  }
}

// A block's tile of 64 x 64 elements of a matrix: rows r0.., columns c0.. as it
// lies in the tensor; `flip`: X is its transpose.
struct Place {
  const Segment* S;
  int matrix, r0, c0;
  bool flip;
};
__device__ __forceinline__ Place place_of(const Matrices& M, int matrix, int t) {
  Place p;
  p.matrix = matrix;
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

// X = u / |u|, as it is held, its columns padded with zeros to the pitch, for the
// matrices whose X is not there yet; `blocks` blocks for each matrix.
template <typename T>
__global__ void __launch_bounds__(256)
build_kernel(const __grid_constant__ Matrices M, const Scale* __restrict__ factors, int blocks, __half* __restrict__ X) {
  __shared__ float tile[64][65];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const int matrix = blockIdx.x / blocks;
  const Scale f = factors[matrix];
  if (!f.build) return;
  for (int t = blockIdx.x % blocks; t < M.tiles_s * M.tiles_L; t += blocks) {
    const Place at = place_of(M, matrix, t);
    const Segment& S = *at.S;
    const int64_t base = (int64_t)(at.matrix - S.first) * S.rows * S.cols;
    const T* g = reinterpret_cast<const T*>(S.g) + base;
    const float* m = M.raw ? nullptr : S.m + base;
    const float scale = M.grad_scale ? *M.grad_scale : 1.f;
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
      for (int x = 0; x < 4; ++x) u[x] = u[x] * f.a * f.b;
      if (at.flip) {
#pragma unroll
        for (int x = 0; x < 4; ++x) tile[y + 16 * i][x4 + x] = u[x];
      } else if (r < M.s && c < M.pitch) {
        *reinterpret_cast<uint2*>(out + (int64_t)r * M.pitch + c) = pack_half4(u);
      }
    }
    if (!at.flip) continue;
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
    __syncthreads();
  }
}

// The same in one pass, with X's factors guessed: the update's size from 4096 of
// its elements, taken to a power of two.  The products with that X take the norm
// itself into account (in fp32: X is rounded once, as it would be), and where the
// guess is wrong by more than a factor of 2 X is built again.  With the factors
// known beforehand g and m are read once: 12 bytes an element instead of 18,
// where they are bf16 and fp32.  48 matrices of 1408 x 4096 0.47 ms (7.1 TB/s),
// where the two kernels above took 0.9.
constexpr int kSample = 4096;
template <typename T>
__global__ void __launch_bounds__(256) sample_kernel(const __grid_constant__ Matrices M, float2* __restrict__ guess) {
  __shared__ Squares s_w[8];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const Segment& S = segment_of(M, blockIdx.x);
  const int64_t n = (int64_t)S.rows * S.cols, base = (int64_t)(blockIdx.x - S.first) * n;
  const T* g = reinterpret_cast<const T*>(S.g) + base;
  const float* m = M.raw ? nullptr : S.m + base;
  const float scale = M.grad_scale ? *M.grad_scale : 1.f;
  const bool vg = aligned_to(g, 4 * sizeof(T)), vm = aligned_to(m, 16);
  const uint32_t stride = (uint32_t)(n / kSample);   // groups of four between two that are read
  Squares q = {0.f, 0.f, 0.f};
#pragma unroll
  for (int it = 0; it < kSample / 1024; ++it) {
    // one of each `stride` groups, another one every time
    const uint32_t j = it * 256 + threadIdx.x;
    const int64_t i = ((int64_t)j * stride + (uint32_t)(((uint64_t)(j * 2654435769u) * stride) >> 32)) * 4;
    float u[4], mm[4];
    load4(g + i, vg, 4, u);
    if (!M.raw) load4(m + i, vm, 4, mm);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (!M.raw) {
        const float gx = u[x] * scale, mx = fmaf(M.mu, mm[x], gx);
        u[x] = M.nesterov ? fmaf(M.mu, mx, gx) : mx;
      }
      add_square(q, u[x]);
    }
  }
  q = block_sum(q, s_w);
  if (threadIdx.x == 0) {
    const float by = (float)n / kSample;
    const float2 f = factors_of(Squares{q.mid * by, q.big * by, q.small * by});
    guess[blockIdx.x] = make_float2(f.x, __int_as_float((__float_as_int(f.y) + 0x400000) & 0xff800000));
  }
}

// A block has 64 rows of 128 columns of X; transposed through shared memory, a
// row's groups of four columns exchanged by the row's number.  What bounds it is
// HBM, with eight rows of a thread in flight, and the sums of squares that hardly
// ever count left out (with four rows and all sums 0.66 ms instead of 0.47).
template <typename T>
__global__ void __launch_bounds__(256, 3)
step_kernel(const __grid_constant__ Matrices M, const float2* __restrict__ guess, Squares* __restrict__ part,
            __half* __restrict__ X) {
  __shared__ Squares s_w[8];
  __shared__ __align__(16) float tile[64][128];
  pdl_enter();
  if (M.skip && *M.skip) return;
  const int matrix = blockIdx.x / M.parts, t = blockIdx.x % M.parts, across = (M.L + 127) / 128;
  const Segment& S = segment_of(M, matrix);
  const bool flip = S.rows > S.cols;
  const int a = t / across * 64, b = t % across * 128;   // in X
  const int64_t base = (int64_t)(matrix - S.first) * S.rows * S.cols;
  const T* g = reinterpret_cast<const T*>(S.g) + base;
  float* m = M.raw ? nullptr : S.m + base;
  const float scale = M.grad_scale ? *M.grad_scale : 1.f;
  const float2 f = guess[matrix];
  const bool vg = aligned_to(g, 4 * sizeof(T)) && S.cols % 4 == 0, vm = aligned_to(m, 16) && S.cols % 4 == 0;
  __half* out = X + (int64_t)matrix * M.plane;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // four columns of the tensor to a thread, every `by`-th row
  const int x4 = flip ? threadIdx.x % 16 * 4 : lane * 4, y = flip ? threadIdx.x / 16 : warp, by = flip ? 16 : 8;
  const int r0 = (flip ? b : a) + y, c = (flip ? a : b) + x4;
  Squares q = {0.f, 0.f, 0.f};
  const bool whole = vg && (M.raw || vm) && f.x == 1.f &&
                     (flip ? b + 128 <= S.rows && a + 64 <= S.cols : a + 64 <= S.rows && b + 128 <= S.cols);
  if (whole) {
    // all of it lies inside, and X takes one factor: eight rows in flight, and one sum of squares
    float u[8][4], mm[8][4];
    const int64_t o = (int64_t)r0 * S.cols + c, step = (int64_t)by * S.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      load4(g + o + i * step, true, 4, u[i]);
      if (!M.raw) load4(m + o + i * step, true, 4, mm[i]);
    }
    float mid = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!M.raw) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float gx = u[i][x] * scale;
          mm[i][x] = fmaf(M.mu, mm[i][x], gx);
          u[i][x] = M.nesterov ? fmaf(M.mu, mm[i][x], gx) : mm[i][x];
        }
        store4(m + o + i * step, true, 4, mm[i]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        mid = fmaf(u[i][x], u[i][x], mid);
        u[i][x] *= f.y;
      }
      if (flip) {
#pragma unroll
        for (int x = 0; x < 4; ++x) tile[x4 + x][(y + i * by) ^ (x4 & 28)] = u[i][x];
      } else {
        *reinterpret_cast<uint2*>(out + (int64_t)(r0 + i * by) * M.pitch + c) = pack_half4(u[i]);
      }
    }
    // The other two sums are this one times 2^-180 and 2^180, unless squares overflowed, or vanished and count.
    float sum = mid;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    q = Squares{mid, mid * kDown * kDown, mid * kUp * kUp};
    if (!(sum > 1e-30f && sum <= 3e38f)) {
      q = Squares{0.f, 0.f, 0.f};
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        float v[4], mv[4];
        load4(g + o + i * step, true, 4, v);
        if (!M.raw) load4(m + o + i * step, true, 4, mv);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!M.raw) v[x] = M.nesterov ? fmaf(M.mu, mv[x], v[x] * scale) : mv[x];
          add_square(q, v[x]);
        }
      }
    }
  }
#pragma unroll 1
  for (int i0 = 0; i0 < 8 && !whole; i0 += 4) {
    float u[4][4], mm[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + (i0 + i) * by, left = r < S.rows ? min(4, S.cols - c) : 0;
      const int64_t o = (int64_t)r * S.cols + c;
#pragma unroll
      for (int x = 0; x < 4; ++x) u[i][x] = mm[i][x] = 0.f;
      if (left > 0) {
        load4(g + o, vg, left, u[i]);
        if (!M.raw) load4(m + o, vm, left, mm[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + (i0 + i) * by, left = r < S.rows ? min(4, S.cols - c) : 0;
      if (!M.raw) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float gx = u[i][x] * scale;
          mm[i][x] = fmaf(M.mu, mm[i][x], gx);
          u[i][x] = M.nesterov ? fmaf(M.mu, mm[i][x], gx) : mm[i][x];
        }
        if (left > 0) store4(m + (int64_t)r * S.cols + c, vm, left, mm[i]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {   // zeros behind the row
        add_square(q, u[i][x]);
        u[i][x] = u[i][x] * f.x * f.y;
      }
      if (flip) {
#pragma unroll
        for (int x = 0; x < 4; ++x) tile[x4 + x][(y + (i0 + i) * by) ^ (x4 & 28)] = u[i][x];
      } else if (r < M.s && c < M.pitch) {
        *reinterpret_cast<uint2*>(out + (int64_t)r * M.pitch + c) = pack_half4(u[i]);
      }
    }
  }
  if (flip) {
    __syncthreads();
    const int to = b + lane * 4;
#pragma unroll 4
    for (int i = warp; i < 64; i += 8)
      if (a + i < M.s && to < M.pitch)
        *reinterpret_cast<uint2*>(out + (int64_t)(a + i) * M.pitch + to) =
            pack_half4(reinterpret_cast<const float*>(&tile[i][(lane * 4) ^ (i & 28)]));
  }
  q = block_sum(q, s_w);
  if (threadIdx.x == 0) part[blockIdx.x] = q;
}

// ---------------------------------------------------------------- small matrices

// Matrices with a short side of at most 128 and a long one of at most 4096 stay
// on chip: a cluster takes a matrix, each of its CTAs up to 512 columns of X,
// and the whole step is one launch.  X, A and B lie in shared memory as panels
// of 64 columns (128 rows of 128 bytes, 128-byte swizzle), which the MMAs read
// along the rows (X X^T, A A, and B) or across them (X in B X).  With several
// CTAs the partial sums of X X^T are added up in the CTAs' order through the
// cluster's shared memory, each CTA taking a share of the rows.
//
// What bounds it is the chain of products, each of which waits for the one
// before: 2.3 us an iteration for 64 x 96, 4.6 for 128 x 512 (of 18 and 44 us
// with five), 7 to 9 with several CTAs (128 x 4096: 67 us).
//
// With a short side of at most 16 an MMA is mostly padding: X stays in fp32, and
// the products are the CUDA cores', exact to fp32 (held in fp16 a vector is 1e-3
// off, a matrix of two rows up to 4e-3).  X X^T by warps, in blocks of 4 x 4
// elements whose sums over the lanes take 16 exchanges; B by a thread for each
// element; B X by a thread for each column, which it keeps in registers.  One
// iteration of 16 x 16 takes 1.8 us (MMAs 2.0), 16 x 512 3.5 (4.6), 16 x 4096
// 4.7 (8.8); 64 matrices of 16 x 4096 96 us with five (276).
constexpr int kSide = 128, kPanel = kSide * 128, kSlice = 512, kMostCtas = 8, kSmallThreads = 512;
// Short sides of at most kThinSide are left to the CUDA cores, in fp32.
constexpr int kThinSide = 16, kThinPitch = kSlice + 4, kThinSums = kSmallThreads / 2;
constexpr size_t kThinSmem =
    4 * (size_t)(kThinSide * kThinPitch + 2 * kMostCtas * kThinSums + kThinSide * (2 * kThinSide + 1));
constexpr size_t kSmallSmem = 1024 + (size_t)(kSlice / 64 + 6) * kPanel;

// Byte offset of elements (row, col) .. (col a multiple of 4) in panels.
__device__ __forceinline__ uint32_t panel_at(int row, int col) {
  const int b = col % 64 * 2;
  return (uint32_t)(col / 64 * kPanel + row * 128 + ((((b >> 4) ^ (row & 7)) << 4) | (b & 15)));
}

__device__ __forceinline__ float4 ld_peer_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <typename T, bool kThin>
__global__ void __launch_bounds__(kSmallThreads, kThin ? 2 : 1)
small_kernel(const __grid_constant__ Matrices M, int iterations, bool opens, int stall, int* err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[2];
  __shared__ Squares s_w[kSmallThreads / 32], s_part[kMostCtas];
  const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const X = smem_raw + (base - tc::smem_u32(smem_raw));   // panels of X, two of A, four of partial sums (two of B)
  uint8_t* const A = X + kSlice / 64 * kPanel;
  uint8_t* const B = A + 2 * kPanel;
  const uint32_t sX = base, sA = sX + kSlice / 64 * kPanel, sB = sA + 2 * kPanel, bar = tc::smem_u32(s_bar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, part = warp >> 2;   // TMEM lanes, and columns
  const int rank = (int)tc::cluster_ctarank();
  uint32_t ctas;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  // thin: X in fp32, two sets of every warp's sums of X X^T, B and A
  float* const thin_x = reinterpret_cast<float*>(smem_raw);
  float* const thin_sums = thin_x + kThinSide * kThinPitch;
  float* const thin_b = thin_sums + 2 * kMostCtas * kThinSums;
  float* const thin_a = thin_b + kThinSide * kThinSide;
  if (kThin) {
    for (int i = threadIdx.x; i < kThinSide * kThinPitch / 4; i += kSmallThreads)
      reinterpret_cast<float4*>(thin_x)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    if (warp == 0) {
      if (lane == 0) {
        tc::mbar_init(bar, 1 + stall);
        tc::mbar_init(bar + 8, 1);
        s_abort = 0;
        tc::fence_barrier_init();
      }
      __syncwarp();
      tc::tmem_alloc(tc::smem_u32(&s_tmem), 512);
      tc::tmem_relinquish();
    }
    for (int i = threadIdx.x; i < kSlice / 64 * kPanel / 16; i += kSmallThreads)
      reinterpret_cast<uint4*>(X)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::tc_fence_before();
  }
  __syncthreads();
  if (!kThin) tc::tc_fence_after();
  if (ctas > 1) tc::cluster_arrive();   // awaited before the first store to another CTA, or where there is none
  // A call's launches of this kernel have nothing to do with one another, nor
  // with the products of larger matrices before them: but for one that opens the
  // call they start beside what is before them, and end behind it.  (What was on
  // the stream before the call is complete: the call's first kernel waits for
  // that before it lets another start.  24 matrices of up to 2048 to a side:
  // 253 us one after another, of which 120 are one larger matrix'.)
  if (opens) pdl_wait();
  pdl_trigger();
  const uint32_t tmem = kThin ? 0 : s_tmem;
  const bool issuer = !kThin && warp == 0 && tc::elect_one();   // of every MMA, and of the commits that follow them
  const bool skip = M.skip && *M.skip;   // the same for every thread of the cluster

  const int matrix = blockIdx.x / ctas;
  const Segment& S = segment_of(M, matrix);
  const bool flip = S.rows > S.cols;
  const int s = flip ? S.cols : S.rows, L = flip ? S.rows : S.cols;
  const int c0 = rank * kSlice, w = max(0, min(kSlice, L - c0)), panels = (w + 63) / 64;
  const int64_t first = (int64_t)(matrix - S.first) * S.rows * S.cols;
  const T* g = reinterpret_cast<const T*>(S.g) + first;
  float* m = M.raw ? nullptr : S.m + first;
  const float scale = M.grad_scale ? *M.grad_scale : 1.f;
  // this CTA's part of the tensor, four elements of a row at a time
  const int r0 = flip ? c0 : 0, nr = flip ? w : s, t0 = flip ? 0 : c0, nc = flip ? s : w, vecs = (nc + 3) / 4;
  const bool even = S.cols % 4 == 0;
  // Lanes go along a row, `along` (a power of two) to a row; four rows of a
  // thread at a time: `load` starts their loads, `use` has them.  (What bounds
  // these passes is their instructions: with a division for each group of four a
  // matrix of 128 x 512 took 39 us for one iteration.)
  struct At {
    int64_t o;      // in the matrix
    int r, c, left;
  };
  // a transposed matrix: 8 lanes at most, since a row's elements are one column of X in shared memory, whose
  // rows share their banks
  const int most = flip ? 8 : 32, along = min(most, vecs > 16 ? 32 : vecs > 8 ? 16 : vecs > 4 ? 8 : vecs > 2 ? 4 : 2);
  const int rows = kSmallThreads / along;
  auto each = [&](auto load, auto use) {
    for (int v = threadIdx.x % along; v < vecs; v += along) {
      const int c = v * 4, left = min(4, nc - c);
      const int64_t o = (int64_t)r0 * S.cols + t0 + c;
      for (int i = threadIdx.x / along; i < nr; i += 4 * rows) {
        float a[4][4], b[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = i + u * rows;
          if (r < nr) load(At{o + (int64_t)r * S.cols, r, c, left}, a[u], b[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = i + u * rows;
          if (r < nr) use(At{o + (int64_t)r * S.cols, r, c, left}, a[u], b[u]);
        }
      }
    }
  };

  if (!skip) {
    // the momentum's step and the update's norm
    const bool vg = even && aligned_to(g, 4 * sizeof(T)), vm = even && aligned_to(m, 16);
    Squares sq = {0.f, 0.f, 0.f};
    auto load_u = [&](const At& p, float* u, float* mm) {
      load4(g + p.o, vg, p.left, u);
      if (!M.raw) load4(m + p.o, vm, p.left, mm);
    };
    each(load_u, [&](const At& p, float* u, float* mm) {
      if (!M.raw) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float gx = u[x] * scale;
          mm[x] = fmaf(M.mu, mm[x], gx);
          u[x] = M.nesterov ? fmaf(M.mu, mm[x], gx) : mm[x];
        }
        store4(m + p.o, vm, p.left, mm);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x < p.left) add_square(sq, u[x]);
    });
    sq = block_sum(sq, s_w);
    __syncwarp();
    if (ctas > 1) tc::cluster_wait();
    if (threadIdx.x == 0) {
      for (uint32_t i = 0; i < ctas; ++i) {   // to every CTA of the cluster
        const uint32_t to = tc::map_peer(tc::smem_u32(&s_part[rank]), i);
        tc::st_peer_f32(to, sq.mid);
        tc::st_peer_f32(to + 4, sq.big);
        tc::st_peer_f32(to + 8, sq.small);
      }
    }
    __syncwarp();
    tc::cluster_sync();
    Squares all = s_part[0];
    for (uint32_t i = 1; i < ctas; ++i) {
      all.mid += s_part[i].mid;
      all.big += s_part[i].big;
      all.small += s_part[i].small;
    }
    const float2 f = factors_of(all);
    each(load_u, [&](const At& p, float* u, const float* mm) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (!M.raw) u[x] = M.nesterov ? fmaf(M.mu, mm[x], u[x] * scale) : mm[x];
        u[x] = x < p.left ? u[x] * f.x * f.y : 0.f;
      }
      if (kThin) {   // as it is, not times 2^12
#pragma unroll
        for (int x = 0; x < 4; ++x) u[x] *= 1.f / kHeld;
        if (flip) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (x < p.left) thin_x[(p.c + x) * kThinPitch + p.r] = u[x];
        } else {
          *reinterpret_cast<float4*>(thin_x + p.r * kThinPitch + p.c) = make_float4(u[0], u[1], u[2], u[3]);
        }
        return;
      }
      const uint2 h = pack_half4(u);
      if (flip) {
        const __half* e = reinterpret_cast<const __half*>(&h);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x < p.left) *reinterpret_cast<__half*>(X + panel_at(p.c + x, p.r & ~3) + (p.r & 3) * 2) = e[x];
      } else {
        *reinterpret_cast<uint2*>(X + panel_at(p.r, p.c)) = h;
      }
    });

    if constexpr (kThin) {
      // A = X X^T in blocks of 4 x 4 on and above the diagonal, each the work of `parts` warps, which share the
      // columns: this warp has every parts-th 32 columns of block (bi, bj).
      const int side = (s + 3) / 4, blocks = side * (side + 1) / 2, parts = kSmallThreads / 32 / blocks;
      const int mine = warp / blocks;
      int bi = 0, bj = warp % blocks;
      while (bj >= side - bi) bj -= side - bi++;
      bj += bi;
      __syncthreads();
      float x[kThinSide];   // this thread's column
#pragma unroll
      for (int n = 0; n < kThinSide; ++n) x[n] = thin_x[n * kThinPitch + threadIdx.x];
#pragma unroll 1
      for (int it = 0; it < iterations; ++it) {
        float* sums = thin_sums + (it & 1) * kMostCtas * kThinSums;
        if (mine < parts) {
          float v[16];
#pragma unroll
          for (int n = 0; n < 16; ++n) v[n] = 0.f;
#pragma unroll 2
          for (int c = mine * 32 + lane; c < w; c += parts * 32) {
            float e[4], o[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              e[n] = thin_x[(bi * 4 + n) * kThinPitch + c];
              o[n] = thin_x[(bj * 4 + n) * kThinPitch + c];
            }
#pragma unroll
            for (int n = 0; n < 16; ++n) v[n] = fmaf(e[n / 4], o[n % 4], v[n]);
          }
          // over the lanes: lanes 2 n and 2 n + 1 end with value n
#pragma unroll
          for (int half = 8; half > 0; half /= 2) {
            const bool up = lane & (2 * half);
#pragma unroll
            for (int n = 0; n < half; ++n) {
              const float give = up ? v[n] : v[n + half], keep = up ? v[n + half] : v[n];
              v[n] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * half);
            }
          }
          v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
          const uint32_t to = tc::smem_u32(sums + rank * kThinSums + warp * 16 + lane / 2);
          for (uint32_t r = lane & 1; r < ctas; r += 2) tc::st_peer_f32(tc::map_peer(to, r), v[0]);
        }
        __syncwarp();
        if (ctas > 1) tc::cluster_sync();
        else __syncthreads();
        const int i = threadIdx.x / kThinSide, j = threadIdx.x % kThinSide;   // of A and B, 256 threads
        if (i < kThinSide) {
          float v = 0.f;
          const int lo = min(i / 4, j / 4), hi = max(i / 4, j / 4);
          if (hi < side) {
            const int block = lo * side - lo * (lo - 1) / 2 + hi - lo;
            const int at = block * 16 + (i / 4 <= j / 4 ? i % 4 * 4 + j % 4 : j % 4 * 4 + i % 4);
            for (uint32_t r = 0; r < ctas; ++r)
              for (int n = 0; n < parts; ++n) v += sums[r * kThinSums + n * blocks * 16 + at];
          }
          thin_a[i * (kThinSide + 1) + j] = v;
        }
        __syncthreads();
        // B = a I + b A + c A A
        if (i < kThinSide) {
          float v[2] = {0.f, 0.f};
#pragma unroll
          for (int n = 0; n < kThinSide; ++n)
            v[n & 1] = fmaf(thin_a[i * (kThinSide + 1) + n], thin_a[n * (kThinSide + 1) + j], v[n & 1]);
          thin_b[i * kThinSide + j] =
              kC * (v[0] + v[1]) + kB * thin_a[i * (kThinSide + 1) + j] + (i == j ? kA : 0.f);
        }
        __syncthreads();
        // X = B X: a thread for a column
        if ((int)threadIdx.x < w) {
          float y[kThinSide];
#pragma unroll
          for (int r = 0; r < kThinSide; ++r) {
            y[r] = 0.f;
            if (r >= s) continue;
#pragma unroll
            for (int n = 0; n < kThinSide; n += 4) {
              const float4 e = *reinterpret_cast<const float4*>(thin_b + r * kThinSide + n);
              y[r] = fmaf(e.x, x[n], fmaf(e.y, x[n + 1], fmaf(e.z, x[n + 2], fmaf(e.w, x[n + 3], y[r]))));
            }
            thin_x[r * kThinPitch + threadIdx.x] = y[r];
          }
#pragma unroll
          for (int r = 0; r < kThinSide; ++r) x[r] = y[r];
        }
        __syncthreads();
      }
    } else {
      uint32_t phase = 0;
      // What the threads wrote to shared memory is there for the MMAs that `issue` starts; returns when they are done.
      // On an expired wait every CTA of the cluster is told: no more MMAs are waited for, and what follows is computed
      // on whatever is there, up to the barriers that all have to meet.
      auto products = [&](auto issue) {
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncthreads();
        if (issuer) {
          tc::tc_fence_after();
          issue();
          tc::tc_commit(bar);
        }
        __syncwarp();
        if (!tc::mbar_wait(bar, phase, &s_abort, kWaitNs)) {
          set_error(err, kDevTimeout);
          for (uint32_t i = 0; i < ctas; ++i) tc::st_peer_u32(tc::map_peer(tc::smem_u32(&s_abort), i), 1u);
        }
        phase ^= 1u;
        __syncwarp();
        tc::tc_fence_after();
      };
      const int row = q * 32 + lane;
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
      // 32 values of this thread's row to columns col .. of panels
      auto keep32 = [&](uint8_t* to, int col, const float* v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 u;
          __half2* h = reinterpret_cast<__half2*>(&u);
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = __floats2half2_rn(v[j * 8 + 2 * x], v[j * 8 + 2 * x + 1]);
          *reinterpret_cast<uint4*>(to + panel_at(row, col + j * 8)) = u;
        }
      };
      constexpr float back = 1.f / kHeld;
#pragma unroll 1
      for (int it = 0; it < iterations; ++it) {
        // A = X X^T
        products([&]() {
          const int steps = (w + 15) / 16;
          for (int k = 0; k < steps; ++k) {
            const uint64_t d = tc::sdesc_k128(sX + k / 4 * kPanel) + (uint32_t)(k % 4 * 2);
            tc::mma_bf16(tmem, d, d, idesc_f16_f32(kSide, kSide), k > 0);
          }
        });
        uint32_t r[32];
        tc::tmem_ld_32x32b_x32(lanes + part * 32, r);
        tc::tmem_wait_ld();
        if (ctas == 1) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = back * __uint_as_float(r[j]);
          keep32(A, part * 32, v);
        } else {
          // partial sums: 128 rows of 128 fp32, 16 bytes of a row exchanged by the row's number
          float4* sums = reinterpret_cast<float4*>(B);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 v = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                         __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
            sums[row * 32 + ((part * 8 + j) ^ (row & 31))] = w > 0 ? v : make_float4(0.f, 0.f, 0.f, 0.f);
          }
          tc::tc_fence_before();
          __syncthreads();
          tc::cluster_sync();
          // rows rank * share ..: every CTA's sums of four elements added up, for every CTA
          const int share = kSide / (int)ctas;
          for (int i = threadIdx.x; i < share * 32; i += kSmallThreads) {
            const int rr = rank * share + i / 32, j = i % 32;
            const uint32_t from = sB + (uint32_t)(rr * 32 + (j ^ (rr & 31))) * 16, to = sA + panel_at(rr, j * 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (uint32_t k = 0; k < ctas; ++k) {
              const float4 x = ld_peer_f32x4(tc::map_peer(from, k));
              v.x += x.x;
              v.y += x.y;
              v.z += x.z;
              v.w += x.w;
            }
            const float e[4] = {v.x * back, v.y * back, v.z * back, v.w * back};
            const uint2 h = pack_half4(e);
            for (uint32_t k = 0; k < ctas; ++k)
              tc::st_peer_u64(tc::map_peer(to, k), (unsigned long long)h.y << 32 | h.x);
          }
          asm volatile("fence.proxy.async;" ::: "memory");
          tc::cluster_sync();
        }
        // B = a I + b A + c A A
        products([&]() {
          for (int k = 0; k < kSide / 16; ++k) {
            const uint64_t d = tc::sdesc_k128(sA + k / 4 * kPanel) + (uint32_t)(k % 4 * 2);
            tc::mma_bf16(tmem, d, d, idesc_f16_f32(kSide, kSide), k > 0);
          }
        });
        {
          const int col = part * 32;
          tc::tmem_ld_32x32b_x32(lanes + col, r);
          tc::tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 u = *reinterpret_cast<const uint4*>(A + panel_at(row, col + j * 8));
            const __half2* e = reinterpret_cast<const __half2*>(&u);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float2 a = __half22float2(e[x]);
              const int i = j * 8 + 2 * x;
              v[i] = fmaf(kB, a.x, kC * back * __uint_as_float(r[i])) + (row == col + i ? kA * kHeld : 0.f);
              v[i + 1] = fmaf(kB, a.y, kC * back * __uint_as_float(r[i + 1])) + (row == col + i + 1 ? kA * kHeld : 0.f);
            }
          }
          keep32(B, col, v);
        }
        // X = B X
        products([&]() {
          for (int n = 0; n < panels; n += 4) {
            const uint32_t idesc = idesc_f16_f32(kSide, min(4, panels - n) * 64) | kMajorB;
            for (int k = 0; k < kSide / 16; ++k) {
              const uint64_t a = tc::sdesc_k128(sB + k / 4 * kPanel) + (uint32_t)(k % 4 * 2);
              const uint64_t b = (tc::sdesc_k128(sX + n * kPanel) | ((uint64_t)(kPanel >> 4) << 16)) + (uint32_t)(k * (2048 >> 4));
              tc::mma_bf16(tmem + n * 64, a, b, idesc, k > 0);
            }
          }
        });
#pragma unroll 1
        for (int c = part; c < panels * 2; c += 4) {
          tc::tmem_ld_32x32b_x32(lanes + c * 32, r);
          tc::tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = back * __uint_as_float(r[j]);
          keep32(X, c * 32, v);
        }
      }
      tc::tc_fence_before();
      __syncthreads();
    }
    // p = p keep - step O, and its bf16 copy; raw: out = O.  Not after an expired wait of this CTA, or of another
    // one before the last sums of X X^T, for which the cluster met.
    const bool whole = kThin || !*(volatile int*)&s_abort;
    if (whole)
      each([&](const At& a, float* p, float*) { get4(M, S, first + a.o, even, a.left, p); },
           [&](const At& a, const float* p, float* v) {
             constexpr float back = 1.f / kHeld;
             if (kThin) {
#pragma unroll
               for (int x = 0; x < 4; ++x)
                 v[x] = x < a.left ? thin_x[flip ? (a.c + x) * kThinPitch + a.r : a.r * kThinPitch + a.c + x] : 0.f;
             } else if (flip) {
#pragma unroll
               for (int x = 0; x < 4; ++x)
                 v[x] = x < a.left
                            ? __half2float(*reinterpret_cast<const __half*>(X + panel_at(a.c + x, a.r & ~3) + (a.r & 3) * 2)) * back
                            : 0.f;
             } else {
               const uint2 u = *reinterpret_cast<const uint2*>(X + panel_at(a.r, a.c));
               const __half2* h = reinterpret_cast<const __half2*>(&u);
               const float2 x = __half22float2(h[0]), y = __half22float2(h[1]);
               v[0] = x.x * back;
               v[1] = x.y * back;
               v[2] = y.x * back;
               v[3] = y.y * back;
             }
             put4(M, S, first + a.o, even, a.left, p, v);
           });
  } else if (ctas > 1) {
    tc::cluster_wait();
  }
  if (!opens) pdl_wait();
  __syncwarp();
  if (ctas > 1) tc::cluster_sync();   // no CTA leaves while another may still read its shared memory
  if (!kThin && warp == 0) {
    // after an expired wait, which may have been the other CTAs', MMAs may still run
    if (issuer && *(volatile int*)&s_abort) {
      tc::tc_commit(bar + 8);
      if (!tc::mbar_wait(bar + 8, 0, nullptr, kWaitNs)) set_error(err, kDevTimeout);
    }
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- the order of it all

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Matrices of s x L (s <= L) that run together, and their buffers.
constexpr size_t kMostBytes = (size_t)4 << 30;   // a larger batch runs in parts of this size
struct Sizes {
  int s, L, parts, tiles;   // partial sums of a matrix by the element, and by the tile
  int64_t pitch, square;   // of X, and of A and B
  Sizes(int rows, int cols) {
    s = rows < cols ? rows : cols;
    L = rows < cols ? cols : rows;
    pitch = round8(L);
    square = round8(s);
    parts = (int)(((int64_t)s * L + kPart - 1) / kPart);
    tiles = (s + 63) / 64 * ((L + 127) / 128);
  }
  size_t x() const { return (size_t)s * pitch * 2; }
  size_t a() const { return (size_t)s * square * 2; }
  size_t bytes(int64_t n) const {   // X and its successor, three short matrices, counters, sums, factors
    return 2 * round256(n * x()) + 3 * round256(n * a()) + 256 + round256(n * kMaxSteps * sizeof(int)) +
           round256(n * tiles * sizeof(Squares)) + round256(n * sizeof(Scale)) + round256(n * sizeof(float2));
  }
  int64_t most() const {
    int64_t n = (int64_t)(kMostBytes /
                          (2 * x() + 3 * a() + kMaxSteps * sizeof(int) + tiles * sizeof(Squares) + sizeof(Scale) + sizeof(float2)));
    const int64_t blocks = (int64_t)((s + 63) / 64) * ((L + 63) / 64);    // of X's kernels, for a matrix
    const int64_t tiles = (int64_t)((s + 127) / 128) * ((L + 127) / 128);   // of a step, at most
    const int64_t grid = ((int64_t)1 << 30) / blocks, numbers = ((int64_t)1 << 30) / (tiles * kMaxSteps);
    if (n > grid) n = grid;
    if (n > numbers) n = numbers;
    return n < 1 ? 1 : n;
  }
};

bool empty(const moe_muon_tensor& t) { return t.batch == 0 || t.rows == 0 || t.cols == 0; }
// CTAs of the cluster that a small matrix takes, 0 for another.
int small_ctas(const moe_muon_tensor& t) {
  const int s = t.rows < t.cols ? t.rows : t.cols, L = t.rows < t.cols ? t.cols : t.rows;
  if (s > kSide || L > kMostCtas * kSlice) return 0;
  int n = 1;
  while (n * kSlice < L) n *= 2;
  return n;
}
bool large(const moe_muon_tensor& t) { return !empty(t) && !small_ctas(t); }
bool alike(const moe_muon_tensor& a, const moe_muon_tensor& b) {
  return (a.rows == b.rows && a.cols == b.cols) || (a.rows == b.cols && a.cols == b.rows);
}
// Whether tensor i is the first large one of its size.
bool leads(const moe_muon_tensor* t, int i) {
  if (!large(t[i])) return false;
  for (int j = 0; j < i; ++j)
    if (large(t[j]) && alike(t[i], t[j])) return false;
  return true;
}

cudaError_t run_matrices(Matrices& M, const Sizes& z, int n, bool grad_bf16, int iterations, bool beside, bool stall,
                         char* ws, cudaStream_t st) {
  int* err = (int*)ws;
  char* at = ws + 256;
  auto take = [&](size_t bytes) {
    char* p = at;
    at += round256(bytes);
    return p;
  };
  Chain C = {};
  for (int i = 0; i < kBuffers; ++i) C.buf[i] = (__half*)take(n * (i <= kY ? z.x() : z.a()));
  C.next = (int*)take(256);
  C.written = (int*)take((size_t)n * kMaxSteps * sizeof(int));
  Squares* part = (Squares*)take((size_t)n * z.tiles * sizeof(Squares));
  Scale* scale = (Scale*)take((size_t)n * sizeof(Scale));
  float2* guess = (float2*)take((size_t)n * sizeof(float2));
  C.scale = scale;
  C.s = z.s;
  C.L = z.L;
  C.batch = n;
  C.pitch = z.pitch;
  C.plane = z.s * z.pitch;
  C.square = z.square;
  C.square_plane = z.s * z.square;
  C.skip = M.skip;
  C.err = err;
  C.beside = beside;
  C.stall = stall;
  for (int i = 0; i < kBuffers; ++i) {
    const bool x = i <= kY;
    if (!tma_map_16bit_3d(&C.along[i], C.buf[i], n, z.s, x ? z.L : z.s, x ? z.pitch : z.square,
                          x ? C.plane : C.square_plane, kBM) ||
        !tma_map_16bit_3d(&C.store[i], C.buf[i], n, z.s, x ? z.L : z.s, x ? z.pitch : z.square,
                          x ? C.plane : C.square_plane, 32) ||
        !tma_map_16bit_3d(&C.across[i], C.buf[i], n, z.s, x ? z.L : z.s, x ? z.pitch : z.square,
                          x ? C.plane : C.square_plane, kBox) ||
        (!x && !tma_map_16bit_3d(&C.mirror[i], C.buf[i], n, z.s, z.s, z.square, C.square_plane, 64, 32)))
      return cudaErrorNotSupported;
  }
  // Tiles of 256 or of 128 columns, whichever take less time by their number: 64
  // elements of the reduction take 600 cycles with 256 columns and 420 with 128
  // (half of the work, but 24 KB for each SM instead of 32, and L2 gives an SM 64
  // bytes a cycle), and a step's start with the epilogue of its last tile 12000
  // and 9000.
  auto tiles_of = [&](int cols, bool wide) {
    const int64_t mt = (z.s + kRows - 1) / kRows, nt = (z.s + cols - 1) / cols, nL = (z.L + cols - 1) / cols;
    return n * (wide ? mt * nL : mt * nt - kRows / cols * (mt * (mt - 1) / 2));
  };
  const int64_t most = sm_count() / 2;
  auto cost = [&](int cols, int64_t stage, int64_t start) {
    const int64_t a = (z.L + kBox - 1) / kBox, b = (z.s + kBox - 1) / kBox;
    const int64_t wide = (tiles_of(cols, true) + most - 1) / most, shorts = (tiles_of(cols, false) + most - 1) / most;
    return (shorts * (a + b) + wide * b) * stage + 3 * start;
  };
  const bool broad = cost(256, 600, 12000) <= cost(128, 420, 9000);
  // Two iterations at a time where the products with X are longer by enough and
  // the short ones fill the SMs.
  const bool pairs = 4 * (int64_t)z.L >= 5 * (int64_t)z.s && tiles_of(256, false) >= most;
  plan_steps(C, iterations, pairs);
  // X with guessed factors where that saves more than its two launches cost (8
  // matrices of 1024 x 1024 94 -> 87 us, 4 of them 60 -> 58, 6 of 1704 x 904 119
  // -> 122) and rows start on four elements (6 of 1700 x 901: 131 -> 144).
  bool guessed = (int64_t)n * z.s * z.L >= 1 << 23;
  for (int i = 0; i < M.n; ++i) guessed = guessed && M.seg[i].cols % 4 == 0;
  M.parts = guessed ? z.tiles : z.parts;
  // blocks for a matrix' X: all it takes, or a few that find it written
  const int per = M.tiles_s * M.tiles_L;
  const int blocks = guessed ? std::max(1, std::min(per, 8 * sm_count() / n)) : per;
  const dim3 sums((unsigned)((int64_t)n * M.parts)), one((unsigned)n), threads(256);
  cudaError_t e = cudaSuccess;
  if (guessed) {
    e = grad_bf16 ? launch_kernel(sample_kernel<bf16>, one, threads, 0, st, 1, M, guess)
                  : launch_kernel(sample_kernel<float>, one, threads, 0, st, 1, M, guess);
    if (e == cudaSuccess)
      e = grad_bf16 ? launch_kernel(step_kernel<bf16>, sums, threads, 0, st, 1, M, guess, part, C.buf[kX])
                    : launch_kernel(step_kernel<float>, sums, threads, 0, st, 1, M, guess, part, C.buf[kX]);
  } else {
    e = grad_bf16 ? launch_kernel(momentum_kernel<bf16>, sums, threads, 0, st, 1, M, part)
                  : launch_kernel(momentum_kernel<float>, sums, threads, 0, st, 1, M, part);
  }
  if (e == cudaSuccess)
    e = launch_kernel(norm_kernel, one, threads, 0, st, 1, M, part, guessed ? guess : nullptr, scale, C.written, C.steps,
                      C.next);
  const dim3 builds((unsigned)((int64_t)n * blocks));
  if (e == cudaSuccess)
    e = grad_bf16 ? launch_kernel(build_kernel<bf16>, builds, threads, 0, st, 1, M, scale, blocks, C.buf[kX])
                  : launch_kernel(build_kernel<float>, builds, threads, 0, st, 1, M, scale, blocks, C.buf[kX]);
  if (e != cudaSuccess) return e;
  return broad ? launch_chain<256>(C, M, tiles_of(256, true), st) : launch_chain<128>(C, M, tiles_of(128, true), st);
}

}  // namespace

size_t orthogonal_workspace(const moe_muon_tensor* tensors, int count) {
  size_t most = 0;
  for (int i = 0; i < count; ++i) {
    if (!leads(tensors, i)) continue;
    const Sizes z(tensors[i].rows, tensors[i].cols);
    int64_t n = 0;
    for (int j = i; j < count; ++j)
      if (large(tensors[j]) && alike(tensors[i], tensors[j])) n += tensors[j].batch;
    const int64_t cap = z.most();
    const size_t bytes = z.bytes(n < cap ? n : cap);
    if (bytes > most) most = bytes;
  }
  return 256 + most;
}

// What the kernels are told of matrices b .. b + n of a tensor.
static Segment segment(const moe_muon_tensor& t, int64_t b, int64_t n, int held, int grad_dtype,
                       const moe_muon_params& h, const OrthogonalRaw* raw) {
  const int64_t at = b * t.rows * t.cols;
  Segment S = {};
  S.rows = t.rows;
  S.cols = t.cols;
  S.first = held;
  if (raw) {
    S.g = (const char*)raw->x + at * (raw->x_dtype == MOE_BF16 ? 2 : 4);
    S.out = (char*)raw->out + at * (raw->out_dtype == MOE_BF16 ? 2 : 4);
  } else {
    S.p = t.p + at;
    S.p16 = t.p_bf16 ? (bf16*)t.p_bf16 + at : nullptr;
    S.g = (const char*)t.grad + at * (grad_dtype == MOE_BF16 ? 2 : 4);
    S.m = t.m + at;
    S.keep = (float)(1.0 - h.lr * t.weight_decay);
    S.step = (float)(h.lr * t.scale);
  }
  return S;
}

cudaError_t launch_orthogonal(const moe_muon_tensor* tensors, int count, int grad_dtype, const moe_muon_params& h,
                              const OrthogonalRaw* raw, const float* grad_scale, const int32_t* skip, bool stall,
                              void* ws, cudaStream_t st) {
  Matrices M = {};
  M.mu = (float)h.momentum;
  M.nesterov = h.nesterov != 0;
  M.raw = raw != nullptr;
  M.out_dtype = raw ? raw->out_dtype : MOE_F32;
  M.grad_scale = grad_scale;
  M.skip = skip;
  int held = 0;   // matrices in M
  // Collects the matrices of the tensors that `which` names, from tensor i on,
  // and has `run` run `most` of them at a time; it is told which time is the last.
  auto collect = [&](int i, int64_t most, auto which, auto run) {
    M.n = held = 0;
    for (int j = i; j < count; ++j) {
      const moe_muon_tensor& t = tensors[j];
      if (!which(t)) continue;
      for (int64_t b = 0; b < t.batch;) {
        if (held == most || M.n == kSegments) {
          const cudaError_t e = run(false);
          if (e != cudaSuccess) return e;
          M.n = held = 0;
        }
        const int64_t n = t.batch - b < most - held ? t.batch - b : most - held;
        M.seg[M.n++] = segment(t, b, n, held, grad_dtype, h, raw);
        held += (int)n;
        b += n;
      }
    }
    return held ? run(true) : cudaSuccess;
  };
  bool opens = true;   // the call with its next launch
  // the last size before the small matrices: those start beside its products
  int last = -1;
  if (std::any_of(tensors, tensors + count, [](const moe_muon_tensor& t) { return !empty(t) && small_ctas(t); }))
    for (int i = 0; i < count; ++i)
      if (leads(tensors, i)) last = i;
  for (int i = 0; i < count; ++i) {
    if (!leads(tensors, i)) continue;
    const Sizes z(tensors[i].rows, tensors[i].cols);
    M.s = z.s;
    M.L = z.L;
    M.pitch = z.pitch;
    M.plane = z.s * z.pitch;
    M.tiles_s = (z.s + 63) / 64;
    M.tiles_L = (z.L + 63) / 64;
    opens = false;
    const cudaError_t e = collect(
        i, z.most(), [&](const moe_muon_tensor& t) { return large(t) && alike(tensors[i], t); },
        [&](bool ends) {
          return run_matrices(M, z, held, grad_dtype == MOE_BF16, h.iterations, i == last && ends, stall, (char*)ws, st);
        });
    if (e != cudaSuccess) return e;
  }
  for (int n = 0; n < 8; ++n) {   // the longest first
    const int ctas = kMostCtas >> (n % 4);
    const bool thin = n >= 4;
    const cudaError_t e = collect(
        0, 1 << 24,
        [&](const moe_muon_tensor& t) {
          return !empty(t) && small_ctas(t) == ctas && (t.rows <= kThinSide || t.cols <= kThinSide) == thin;
        },
        [&](bool) {
          auto kern = grad_dtype == MOE_BF16 ? thin ? small_kernel<bf16, true> : small_kernel<bf16, false>
                                             : thin ? small_kernel<float, true> : small_kernel<float, false>;
          const size_t smem = thin ? kThinSmem : kSmallSmem;
          const cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
          if (r != cudaSuccess) return r;
          const bool now = opens;
          opens = false;
          return launch_kernel(kern, dim3((unsigned)(held * ctas)), dim3(kSmallThreads), smem, st, (unsigned)ctas, M,
                               (int)h.iterations, now, stall ? 1 : 0, (int*)ws);
        });
    if (e != cudaSuccess) return e;
  }
  static_assert(kMostCtas == 8, "one, two, four or eight CTAs");
  return cudaSuccess;
}

}  // namespace moe
