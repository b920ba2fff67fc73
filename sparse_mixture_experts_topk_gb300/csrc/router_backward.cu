// The load-balancing loss over the tokens that count, and the router's
// gradient (Qwen2-MoE code walkthrough, jsqmd.com, sections 3.1 and 3.3).
//
//   p = softmax(l / tau),  w = p[ids] / sum_j p[ids_j] = softmax(l[ids] / tau)
//   loss = E sum_e f_e P_e,  f_e = count_e / (n K),  P_e = sum_t p[t, e] / n
// over the n tokens that the mask keeps.  Backwards, with c_e = dloss E f_e / n
// the loss' derivative by p[t, e] (the counts have none):
//   dl[t, e] = 1/tau ( sum_{ids_j = e} w_j (dw_j - <w, dw>) + p_e (c_e - <p, c>) )
//   dWg = dl^T x,  dbias = sum_t dl,  dx = dl Wg
//
// A group of 8 or 16 lanes takes a token, each lane 4 experts at a time,
// so that a token's scores are one vector load a lane and every sum over them
// stays in the group.  What is summed over tokens leaves a block as one row of
// partial sums; the rows are added in their order, so results are
// deterministic.
//
// Long batches of many experts are bound by HBM and by the issue slots, half of
// which are taken (131072 tokens of 256 experts, 138 MB: 26 us, with the sums
// 31), short ones by the launches (8192 padded tokens of 32 experts: 5.3 us
// replayed from a graph, 64 tokens, which one block has, 2.1; called, 7.6 and 5.3,
// the host's time).
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

constexpr float kLog2E = 1.44269504088896341f;

// 2^x, within 2^-22 relative; zero for -infinity and where it would be subnormal.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Lanes for a token and experts for a lane, by the number of experts: few lanes
// with many experts, since a sum over a group's lanes costs the same for any
// number of groups in a warp (131072 tokens of 256 experts: 32 lanes 34 us, 16
// lanes 31).
template <int kLanes, int kVecs>
struct Group {
  static constexpr int kTokens = kThreads / kLanes;   // at a time in a block
  static constexpr int kN = 4 * kVecs;
  static constexpr int kAhead = kN > 8 ? 1 : 2;   // tokens of a group in flight together
  // expert i of this lane
  __device__ static int expert(int lane, int i) { return (i / 4) * kLanes * 4 + lane * 4 + i % 4; }
  __device__ static float sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ static float max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
  // This lane's scores of a token, -infinity past the last expert.
  __device__ static void load(const float* __restrict__ row, int lane, int E, bool live, float* l) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int e = expert(lane, 4 * v);
      if (E % 4 == 0) {
        const float4 q = live && e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        l[4 * v] = q.x;
        l[4 * v + 1] = q.y;
        l[4 * v + 2] = q.z;
        l[4 * v + 3] = q.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[4 * v + i] = live && e + i < E ? row[e + i] : 0.f;
      }
    }
    if (E == kLanes * kN) return;
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (expert(lane, i) >= E) l[i] = -INFINITY;
  }
  // The group's exponentials of scores / tau, less the largest, in place;
  // returns 1 / their sum.  scale: log2(e) / tau.  A NaN among the scores makes
  // all of it NaN.
  __device__ static float exponentials(float* l, float scale) {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) top = fmaxf(top, l[i]);
    top = max(top);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      l[i] = exp2_fast((l[i] - top) * scale);
      s += l[i];
    }
    return __fdividef(1.f, sum(s));
  }
};

// The groups' sums over a block's tokens, added in order: thread e has expert e's.
template <typename G>
__device__ __forceinline__ float block_sums(const float* acc, float* s, int lane, int group, int E) {
  constexpr int kWidth = G::kN * (kThreads / G::kTokens);
#pragma unroll
  for (int i = 0; i < G::kN; ++i) s[group * kWidth + G::expert(lane, i)] = acc[i];
  __syncthreads();
  float v = 0.f;
  if ((int)threadIdx.x < E)
    for (int g = 0; g < G::kTokens; ++g) v += s[g * kWidth + threadIdx.x];
  return v;
}

// a + b, and what its rounding lost added to `low` (exact: Knuth's two-sum).
// The loss' sums are held as such pairs: GB300 does few fp64 operations a
// cycle, and one block of them took 10 us for 256 experts.
__device__ __forceinline__ float two_sum(float a, float b, float* low) {
  const float s = a + b, t = s - a;
  *low += (a - (s - t)) + (b - t);
  return s;
}

// A block's row of partial sums and counts; kOne: of the only block, the loss.
template <int kLanes, int kVecs, bool kOne>
__global__ void __launch_bounds__(kThreads)
balance_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask,
               int64_t T, int E, int K, float inv_tau, float* __restrict__ part_p, int32_t* __restrict__ part_c,
               BalanceOut o, int* err) {
  using G = Group<kLanes, kVecs>;
  __shared__ float s_p[kThreads * 4 * kVecs];
  __shared__ int s_count[257];
  for (int i = threadIdx.x; i <= E; i += kThreads) s_count[i] = 0;
  __syncthreads();
  pdl_enter();
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  float acc[G::kN] = {};
  int n = 0;
  constexpr int kAhead = G::kAhead;
  const int64_t stride = (int64_t)gridDim.x * G::kTokens;
  for (int64_t t0 = (int64_t)blockIdx.x * G::kTokens; t0 < T; t0 += kAhead * stride) {
    float l[kAhead][G::kN];
    bool live[kAhead];
    int id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t t = t0 + u * stride + group;
      live[u] = t < T && (!mask || mask[t]);
      id[u] = t < T && lane < K ? ids[t * K + lane] : -1;
      G::load(logits + t * E, lane, E, t < T, l[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const float inv = G::exponentials(l[u], inv_tau * kLog2E);
      if (live[u]) {
#pragma unroll
        for (int i = 0; i < G::kN; ++i) acc[i] = fmaf(l[u][i], inv, acc[i]);
        ++n;
        if (id[u] >= 0 && id[u] < E) atomicAdd(&s_count[id[u]], 1);
        else if (id[u] != -1) set_error(err, kDevBadIndex);
      }
    }
  }
  if (lane == 0 && n) atomicAdd(&s_count[E], n);
  const int e = threadIdx.x;
  const float sum = block_sums<G>(acc, s_p, lane, group, E);   // its barrier ends the counting too
  if (!kOne) {
    if (e < E) part_p[(int64_t)blockIdx.x * E + e] = sum;
    for (int i = e; i <= E; i += kThreads) part_c[(int64_t)blockIdx.x * (E + 1) + i] = s_count[i];
    return;
  }
  // the results as balance_finish_kernel has them
  const int tokens = s_count[E];
  const float total = (float)tokens;
  if (e < E) {
    if (o.psum) o.psum[e] = sum;
    if (o.count) o.count[e] = s_count[e];
  }
  float v = e < E && tokens ? (float)s_count[e] / (total * (float)K) * (sum / total) : 0.f;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  __syncthreads();   // s_p has been read
  if (e % 32 == 0) s_p[e / 32] = v;
  __syncthreads();
  if (e == 0) {
    for (int i = 1; i < kThreads / 32; ++i) v += s_p[i];
    if (o.tokens) *o.tokens = tokens;
    if (o.loss) *o.loss = (float)E * v;
  }
}

// The partial rows added up, 32 experts to a block, and the loss from the
// blocks of the cluster (all of the grid).  (By the last blocks to arrive in
// the kernel before, which costs a fence and an atomic's round trip twice, a
// padded batch of 8192 tokens and 32 experts took 13 us; so it takes 6.5.)
__global__ void __launch_bounds__(1024)
balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int rows, int E, int K,
                      BalanceOut o) {
  __shared__ float s_hi[32][33], s_lo[32][33], s_term[32], s_block[8];
  __shared__ int s_c[32][33], s_n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();
  tc::cluster_arrive();   // awaited before the store to the first block
  pdl_enter();
  float hi = 0.f, lo = 0.f;
  int c = 0, n = 0;
  if (e < E) {
#pragma unroll 8
    for (int r = warp; r < rows; r += 32) {
      hi = two_sum(hi, part_p[(int64_t)r * E + e], &lo);
      c += part_c[(int64_t)r * (E + 1) + e];
    }
  }
  for (int r = threadIdx.x; r < rows; r += 1024) n += part_c[(int64_t)r * (E + 1) + E];
  s_hi[warp][lane] = hi;
  s_lo[warp][lane] = lo;
  s_c[warp][lane] = c;
  if (n) atomicAdd(&s_n, n);
  __syncthreads();
  // warp w: expert w of the block's
  hi = s_hi[lane][warp];
  lo = s_lo[lane][warp];
  c = s_c[lane][warp];
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    lo += __shfl_xor_sync(0xffffffffu, lo, w);
    hi = two_sum(hi, __shfl_xor_sync(0xffffffffu, hi, w), &lo);
    c += __shfl_xor_sync(0xffffffffu, c, w);
  }
  const int mine = blockIdx.x * 32 + warp;
  const float total = (float)s_n, sum = hi + lo;
  if (lane == 0) {
    if (mine < E && o.psum) o.psum[mine] = sum;
    if (mine < E && o.count) o.count[mine] = c;
    // f_e P_e, each a share, in fp32
    s_term[warp] = mine < E && s_n ? (float)c / (total * (float)K) * (sum / total) : 0.f;
  }
  __syncthreads();
  tc::cluster_wait();
  if (warp == 0) {
    float v = s_term[lane], low = 0.f;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      low += __shfl_xor_sync(0xffffffffu, low, w);
      v = two_sum(v, __shfl_xor_sync(0xffffffffu, v, w), &low);
    }
    if (lane == 0) tc::st_peer_f32(tc::map_peer(tc::smem_u32(&s_block[blockIdx.x]), 0), v + low);
  }
  __syncwarp();
  tc::cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float v = 0.f, low = 0.f;
    for (int i = 0; i < (int)gridDim.x; ++i) v = two_sum(v, s_block[i], &low);
    if (o.tokens) *o.tokens = s_n;
    if (o.loss) *o.loss = (float)E * (v + low);
  }
}

// Four values as bf16 parts: v = high + middle + low, each rounded from what
// the ones before it leave (exactly, but for values below 2^-110).
__device__ __forceinline__ void split4(const float* v, uint2* parts) {
  float rest[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(rest[0], rest[1]), b = __floats2bfloat162_rn(rest[2], rest[3]);
    parts[k] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    const float2 fa = __bfloat1622float2(a), fb = __bfloat1622float2(b);
    rest[0] -= fa.x;
    rest[1] -= fa.y;
    rest[2] -= fb.x;
    rest[3] -= fb.y;
  }
}

// The scores' gradient, and its sum over each block's tokens.  It is written
// as [T, E] fp32 (dl) and as bf16 parts (panels), where these are not null.
// Panels are 64 columns wide and zero past the last expert: the high parts of
// all experts, the middle ones, the low ones; up to 32 experts: [high | middle],
// [low | 0].  alive (or null): for the tokens of each step of a block, whether
// one counts, up to a multiple of 128 tokens.
template <int kLanes, int kVecs>
__global__ void __launch_bounds__(kThreads)
dlogits_kernel(RouterBackward b, int64_t T, int E, int K, float inv_tau, float* __restrict__ dl,
               bf16* __restrict__ panels, int panel_cols, uint8_t* __restrict__ alive,
               float* __restrict__ part_b, int* err) {
  using G = Group<kLanes, kVecs>;
  __shared__ float s_b[kThreads * 4 * kVecs];
  pdl_enter();
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  float c[G::kN], acc[G::kN] = {};
  if (b.dloss) {
    const float n = (float)*b.tokens, f = n > 0.f ? *b.dloss / n * ((float)E / (n * (float)K)) : 0.f;
    // sum_e p_e = 1: any constant may be taken off the counts.  Their mean, to an
    // integer: what is left of nearly equal ones has all its bits.
    const int mean = __float2int_rn(n * ((float)K / (float)E));
#pragma unroll
    for (int i = 0; i < G::kN; ++i) {
      const int e = G::expert(lane, i);
      c[i] = e < E ? f * (float)(b.count[e] - mean) : 0.f;
    }
  }
  const int64_t end = alive ? (T + 127) / 128 * 128 : T;
  for (int64_t t0 = (int64_t)blockIdx.x * G::kTokens; t0 < end; t0 += (int64_t)gridDim.x * G::kTokens) {
    const int64_t t = t0 + group;
    const bool live = t < T && (!b.mask || b.mask[t]);
    if (alive) {
      const int any = __syncthreads_or(live);
      if (threadIdx.x == 0) alive[t0 / G::kTokens] = any != 0;
    }
    // lane j has choice j; what is loaded for a token that does not count is not used
    const bool mine = b.dw && t < T && lane < K;
    int id = mine ? b.ids[t * K + lane] : -1;
    float g = mine ? b.dw[t * K + lane] : 0.f;
    float d[G::kN] = {};
    if (b.dloss) {
      float p[G::kN], dot = 0.f;
      G::load(b.logits + t * E, lane, E, t < T, p);
      const float inv = G::exponentials(p, inv_tau * kLog2E);
#pragma unroll
      for (int i = 0; i < G::kN; ++i) dot = fmaf(p[i], c[i], dot);
      dot = G::sum(dot) * inv;
#pragma unroll
      for (int i = 0; i < G::kN; ++i) d[i] = p[i] * inv * (c[i] - dot);
    }
    if (b.dw) {
      float z = -INFINITY;
      if (live && id >= 0 && id < E) {
        z = b.logits[t * E + id];
      } else {
        if (live && id != -1) set_error(err, kDevBadIndex);
        id = -1;
        g = 0.f;
      }
      const float top = G::max(z), x = id >= 0 ? exp2_fast((z - top) * (inv_tau * kLog2E)) : 0.f, s = G::sum(x);
      const float w = s != 0.f ? x / s : 0.f, dot = G::sum(w * g), v = w * (g - dot);
      for (int j = 0; j < K; ++j) {
        const int e = __shfl_sync(0xffffffffu, id, j, kLanes);
        const float vj = __shfl_sync(0xffffffffu, v, j, kLanes);
#pragma unroll
        for (int i = 0; i < G::kN; ++i)
          if (G::expert(lane, i) == e) d[i] += vj;
      }
    }
#pragma unroll
    for (int i = 0; i < G::kN; ++i) {
      d[i] = live ? d[i] * inv_tau : 0.f;
      acc[i] += d[i];
    }
    if (t < T && panels) {
      bf16* row = panels + t * panel_cols;
      const bool packed = E <= 32;
      const int width = packed ? 32 : panel_cols / 3;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int e = G::expert(lane, 4 * v);
        uint2 parts[3];
        split4(d + 4 * v, parts);
        if (e < width) {
#pragma unroll
          for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2*>(row + k * width + e) = parts[k];
          if (packed) *reinterpret_cast<uint2*>(row + 96 + e) = make_uint2(0u, 0u);
        }
      }
    }
    if (t < T && dl) {
      float* row = dl + t * E;
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const int e = G::expert(lane, 4 * v);
        if (E % 4 == 0) {
          if (e < E) *reinterpret_cast<float4*>(row + e) = make_float4(d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < E) row[e + i] = d[4 * v + i];
        }
      }
    }
  }
  if (b.dbias) {
    const float sum = block_sums<G>(acc, s_b, lane, group, E);
    if ((int)threadIdx.x < E) part_b[(int64_t)blockIdx.x * E + threadIdx.x] = sum;
  }
}

// The gate's products on CUDA cores, each of a launch's blocks for one of them:
//   dx: 16 tokens, a thread a column
//   dWg: partial sums over a share of the tokens, 16 experts, a thread a column
//   (a masked token's x is not read: it may hold anything)
//   dbias: the last block, the rows of partial sums in order
constexpr int kTokTile = 16, kExpTile = 16, kTokStep = 32;
struct SimtBlocks {
  int cols;             // blocks of 128 columns
  int64_t dx;           // blocks of dx
  int groups, splits;   // of dWg: of experts and of tokens
  int64_t dwg;
};

template <typename T>
__global__ void __launch_bounds__(128)
products_simt_kernel(RouterBackward b, SimtBlocks n, const float* __restrict__ dl, int64_t Tn, int E, int H,
                     float* __restrict__ part_w, const float* __restrict__ part_b, int rows_b) {
  __shared__ float s_dl[256 * kTokTile];
  pdl_enter();
  int64_t i = blockIdx.x;
  if (i < n.dx) {
    const T* Wg = reinterpret_cast<const T*>(b.Wg);
    T* dx = reinterpret_cast<T*>(b.dx);
    const int64_t t0 = i / n.cols * kTokTile;
    for (int k = threadIdx.x; k < E * kTokTile; k += 128) {
      const int tt = k / E, e = k % E;
      s_dl[e * kTokTile + tt] = t0 + tt < Tn ? dl[(t0 + tt) * E + e] : 0.f;
    }
    __syncthreads();
    const int h = (int)(i % n.cols) * 128 + threadIdx.x;
    if (h >= H) return;
    float acc[kTokTile] = {};
#pragma unroll 4
    for (int e = 0; e < E; ++e) {
      const float w = to_f32(Wg[(int64_t)e * H + h]);
#pragma unroll
      for (int k = 0; k < kTokTile; ++k) acc[k] = fmaf(s_dl[e * kTokTile + k], w, acc[k]);
    }
#pragma unroll
    for (int k = 0; k < kTokTile; ++k)
      if (t0 + k < Tn) dx[(t0 + k) * H + h] = from_f32<T>(acc[k]);
  } else if ((i -= n.dx) < n.dwg) {
    const T* x = reinterpret_cast<const T*>(b.x);
    const int h = (int)(i % n.cols) * 128 + threadIdx.x, e0 = (int)(i / n.cols % n.groups) * kExpTile;
    const int64_t split = i / n.cols / n.groups, a = Tn * split / n.splits, z = Tn * (split + 1) / n.splits;
    float acc[kExpTile] = {};
    for (int64_t t0 = a; t0 < z; t0 += kTokStep) {
      __syncthreads();
      for (int k = threadIdx.x; k < kTokStep * kExpTile; k += 128) {
        const int tt = k / kExpTile, e = e0 + k % kExpTile;
        s_dl[k] = t0 + tt < z && e < E ? dl[(t0 + tt) * E + e] : 0.f;
      }
      __syncthreads();
      if (h < H) {
        const int left = (int)(z - t0 < kTokStep ? z - t0 : kTokStep);
#pragma unroll 8
        for (int tt = 0; tt < left; ++tt) {
          const float v = !b.mask || b.mask[t0 + tt] ? to_f32(x[(t0 + tt) * H + h]) : 0.f;
#pragma unroll
          for (int k = 0; k < kExpTile; ++k) acc[k] = fmaf(s_dl[tt * kExpTile + k], v, acc[k]);
        }
      }
    }
    if (h < H)
#pragma unroll
      for (int k = 0; k < kExpTile; ++k)
        if (e0 + k < E) part_w[(split * E + e0 + k) * H + h] = acc[k];
  } else {
    for (int e = threadIdx.x; e < E; e += 128) {
      float v = 0.f;
#pragma unroll 8
      for (int r = 0; r < rows_b; ++r) v += part_b[(int64_t)r * E + e];
      b.dbias[e] = v;
    }
  }
}

// out[i] = the sum of `rows` rows of n, in order.
__global__ void __launch_bounds__(256)
row_sums_kernel(const float* __restrict__ part, int64_t rows, int64_t n, float* __restrict__ out) {
  pdl_enter();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
#pragma unroll 8
  for (int64_t r = 0; r < rows; ++r) v += part[r * n + i];
  out[i] = v;
}

int simt_splits(const Shape& s) {
  const int64_t blocks = (int64_t)((s.H + 127) / 128) * ((s.E + kExpTile - 1) / kExpTile);
  const int64_t want = (2 * (int64_t)sm_count() + blocks - 1) / blocks, most = (s.T + 63) / 64;
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n);
}

template <typename T>
cudaError_t products_simt(const Shape& s, const RouterBackward& b, const float* dl, float* part_w, const float* part_b,
                          int rows_b, cudaStream_t st) {
  SimtBlocks n = {};
  n.cols = (s.H + 127) / 128;
  n.dx = b.dx ? (s.T + kTokTile - 1) / kTokTile * n.cols : 0;
  n.groups = (s.E + kExpTile - 1) / kExpTile;
  n.splits = simt_splits(s);
  n.dwg = b.dWg ? (int64_t)n.cols * n.groups * n.splits : 0;
  const int64_t blocks = n.dx + n.dwg + (b.dbias ? 1 : 0), size = (int64_t)s.E * s.H;
  if (blocks == 0) return cudaSuccess;
  if (blocks >= (int64_t)1 << 31) return cudaErrorNotSupported;
  cudaError_t e = launch_kernel(products_simt_kernel<T>, dim3((unsigned)blocks), dim3(128), 0, st, 1, b, n, dl, s.T, s.E,
                                s.H, n.splits > 1 ? part_w : b.dWg, part_b, rows_b);
  if (e == cudaSuccess && b.dWg && n.splits > 1)
    e = launch_kernel(row_sums_kernel, dim3((unsigned)((size + 255) / 256)), dim3(256), 0, st, 1, part_w,
                      (int64_t)n.splits, size, b.dWg);
  return e;
}

// Runs f with the lanes of a token and the vectors of a lane that E takes.
template <typename F>
cudaError_t by_experts(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  if (E <= 64) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
  if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
}

}  // namespace

// Blocks that walk over the tokens: `per_sm` an SM at most while a block has no
// more than 2^13 tokens, and no more than have `rounds` tokens for each group.
static int64_t token_blocks(const Shape& s, int per_sm, int rounds) {
  const int64_t tokens = kThreads / (s.E <= 64 ? 8 : 16);
  const int64_t want = (s.T + rounds * tokens - 1) / (rounds * tokens), cap = per_sm * (int64_t)sm_count();
  const int64_t least = (s.T + 8191) / 8192;
  int64_t n = want < cap ? want : cap;
  if (n < least) n = least;
  return n < 1 ? 1 : n;
}
int64_t balance_partials(const Shape& s) { return token_blocks(s, 4, s.E <= 128 ? 2 : 1); }
// The scores' gradient: five blocks of 256 threads fit an SM.
int64_t dlogits_partials(const Shape& s) { return token_blocks(s, 5, 1); }

bool router_gate_on_tensor_cores(const Shape& s) {
  return s.dtype == MOE_BF16 && !(s.flags & MOE_FLAG_SIMT_ROUTER);
}
size_t router_scratch_bytes(const Shape& s) {
  if (!router_gate_on_tensor_cores(s)) return (size_t)s.T * s.E * 4;
  return (size_t)s.T * gate_panel_cols(s.E) * 2 + (size_t)(s.T + 127) / 128 * 16;   // and a tile's flags
}
int64_t router_weight_partials(const Shape& s) {
  return router_gate_on_tensor_cores(s) ? gate_part_floats(s) : (int64_t)simt_splits(s) * s.E * s.H;
}

cudaError_t launch_balance(const Shape& s, const float* logits, const int32_t* ids, const uint8_t* mask,
                           const BalanceOut& o, float* part_p, int32_t* part_c, int* err, cudaStream_t st) {
  const int rows = (int)balance_partials(s);
  const cudaError_t e = by_experts(s.E, [&](auto lanes, auto vecs) {
    constexpr int kLanes = decltype(lanes)::value, kVecs = decltype(vecs)::value;
    return launch_kernel(rows == 1 ? balance_kernel<kLanes, kVecs, true> : balance_kernel<kLanes, kVecs, false>,
                         dim3((unsigned)rows), dim3(kThreads), 0, st, 1, logits, ids, mask, s.T, s.E, s.K, s.inv_tau,
                         part_p, part_c, o, err);
  });
  if (e != cudaSuccess || rows == 1) return e;
  const unsigned blocks = s.E <= 32 ? 1 : s.E <= 64 ? 2 : s.E <= 128 ? 4 : 8;
  return launch_kernel(balance_finish_kernel, dim3(blocks), dim3(1024), 0, st, blocks, part_p, part_c, rows, s.E, s.K,
                       o);
}

cudaError_t launch_router_backward(const Shape& s, const RouterBackward& b, void* dl, float* part_b, float* part_w,
                                   int* err, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (s.T == 0) {
    if (b.dWg) e = cudaMemsetAsync(b.dWg, 0, (size_t)s.E * s.H * 4, st);
    if (e == cudaSuccess && b.dbias) e = cudaMemsetAsync(b.dbias, 0, (size_t)s.E * 4, st);
    return e;
  }
  const bool tc = router_gate_on_tensor_cores(s), products = b.dx || b.dWg;
  float* out = b.dlogits || tc || !products ? b.dlogits : (float*)dl;
  bf16* panels = tc && products ? (bf16*)dl : nullptr;
  uint8_t* alive = panels && b.mask && gate_skips_tiles(s.E) ? (uint8_t*)(panels + s.T * gate_panel_cols(s.E)) : nullptr;
  const int64_t rows = dlogits_partials(s);
  e = by_experts(s.E, [&](auto lanes, auto vecs) {
    return launch_kernel(dlogits_kernel<decltype(lanes)::value, decltype(vecs)::value>, dim3((unsigned)rows),
                         dim3(kThreads), 0, st, 1, b, s.T, s.E, s.K, s.inv_tau, out, panels, gate_panel_cols(s.E),
                         alive, part_b, err);
  });
  if (e != cudaSuccess) return e;
  if (tc) return launch_gate_tc(s, b, panels, alive, part_w, part_b, (int)rows, err, st);
  return s.dtype == MOE_BF16 ? products_simt<bf16>(s, b, out, part_w, part_b, (int)rows, st)
                             : products_simt<float>(s, b, out, part_w, part_b, (int)rows, st);
}

}  // namespace moe
