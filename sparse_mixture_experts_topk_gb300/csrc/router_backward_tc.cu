// The gate's products of the router's gradient on the tensor cores: from the
// scores' gradient dl [T, E] (router_backward.cu)
//   dWg = dl^T x  [E, H],   dx = dl Wg  [T, H]
// in one pass over x and dx, which are what it has to read and write: the
// products themselves are E wide.
//
// dl comes in bf16 parts whose sum it is: high + middle for dx, and low too for
// dWg (24 bits: dl itself).  What dx leaves out, 2^-18 of each dl, is under half
// of its own rounding to 8 bits even where Wg's rows are nearly alike, so that
// most of the sum cancels (a token's dl add up to zero): rows of bf16 that differ
// do so by 2^-8 of their size (with the low part, too, 32768 tokens of 64 experts
// take 99.5 us instead of 98.2).  A part times a bf16 value is exact in the tensor cores' fp32 sums.  The parts of 64 experts
// are a panel of 64 columns; up to 32 experts high and middle share one.
//
// A CTA takes 128 columns of H (a chunk) and walks over tiles of 128 tokens:
//   D1 [128 columns, E]   += x^T dl   x read along its rows ("MN-major"), the panels too
//   D2 [128 tokens, 128]   = dl Wg    the panels K-major, Wg's columns in shared memory
// so the same panel in shared memory serves both.  The tensor cores' fp32 sums
// round towards zero, half a last place low each on average: over all of a
// CTA's tokens dWg would be 1e-4 small (32768 tokens).  So D1 starts anew every
// tile (every four above 128 experts), the small parts apart or first, and the
// epilogue adds it to sums in registers, which leave as partial ones at the
// CTA's end; a last kernel adds those of a chunk in order.  D2 is
// double-buffered and leaves through shared memory by TMA.
//
// CTA b has chunk b mod chunks and every splits-th tile, so that the CTAs
// running at one time read whole rows of the same few tiles, and padding at
// the sequences' ends is shared out.  (Dealt out chunk by chunk, evenly over
// all SMs, the prefill layer's products took 6 us more: pieces of 256 bytes of
// rows far apart.)
//
// Roles: warp 0 producer of x and Wg, warp 1 of the panels, warp 2 MMA issuer,
// warp 3 zeroes the rows of tokens that the mask leaves out (0 x NaN is NaN),
// warps 4-11 epilogue, two for a quarter of the TMEM lanes, each with half of
// the columns.  Every wait is bounded: on expiry the kernel records a timeout in
// the workspace's error word, drains what it has in flight, frees its tensor
// memory and returns.
//
// What bounds it is HBM up to 32 experts (32768 tokens, H = 4096: 86 us for
// 537 MB, 93 % of the copy rate; the prefill layer's 8192 tokens, H = 3584:
// 22 us for 118 MB), and from 64 on the MMA thread, 2500 of a tile's 2870 cycles
// with 64 experts.  These are this kernel's times; with 32768 tokens of 64, 128
// and 256 experts it takes 101, 183 and 328 us, and the call 109, 195 and 350.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kTok = 128, kCols = 128;        // tokens of a tile, columns of a chunk
constexpr int kHalf = kTok * 128;             // bytes of 64 columns of an x tile, and of a panel
constexpr int kXBytes = 2 * kHalf;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kStoreBytes = 32 * 128;         // an epilogue warp's 32 rows of 64 columns
constexpr int kOut = kEpiWarps * kStoreBytes;
constexpr int kMaxX = 3, kMaxPanels = 5;
constexpr int kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;

// How E experts are held: `groups` of 64 columns of D1; panels of a tile, `per`
// of them in a slot of the ring.  Up to 32 experts a slot holds a tile's two
// panels and one MMA takes both: its operand x is read from shared memory once
// for 128 columns instead of for 64 (the prefill layer's call 30.9 -> 28.9 us).
// For 64 experts the three panels in a slot leave room for two tiles of x only
// (the call on 32768 padded tokens, 102.7 us then, 104.7), so slots hold one.
struct Plan {
  int E, groups, panels;
  bool packed;      // up to 32 experts: panels [high | middle] and [low | 0]
  int per, nx, np;  // ring sizes: tiles of x, slots of panels
  int bufs;         // buffers of D1
  __host__ __device__ explicit Plan(int e)
      : E(e), groups((e + 63) / 64), panels(e <= 32 ? 2 : 3 * ((e + 63) / 64)), packed(e <= 32),
        per(e <= 32 ? 2 : 1), nx(e <= 128 ? 3 : 2),
        np(e <= 32 ? 2 : e <= 64 || (e > 128 && e <= 192) ? 5 : 4), bufs(e <= 128 ? 2 : 1) {}
  __host__ __device__ int wg_bytes() const { return groups * 2 * 64 * 128; }
  size_t smem() const { return 1024 + (size_t)wg_bytes() + nx * kXBytes + np * per * kHalf + kOut; }
};

struct Params {
  CUtensorMap x, wg, panel, dx;   // boxes of 128, 32, 128 and 32 rows
  const uint8_t* mask;
  const uint8_t* alive;   // whether tokens of a tile count; null: all are taken
  int64_t T;
  int tiles, chunks;
  int E, H;
  float* part;     // [CTAs (packed: twice), E, 128] or null: no dWg
  bool dx_on;
  int* err;
  int stall;       // testing: 1 = the first panels' barrier waits for an arrival that nobody makes
};

// A CTA's tiles: `first` and every step-th after it.  kFlags: bytes for a tile
// that say whether a token of it counts (0: all do); those of the next tile are
// on their way while one is worked on.
template <int kFlags>
struct Walk {
  int tile, step, tiles, n;   // n: tiles before this one
  const uint8_t* alive;
  bool live, ahead;
  __device__ Walk(int first, int every, int count, const uint8_t* flags)
      : tile(first), step(every), tiles(count), n(0), alive(flags) {
    live = read(tile);
    ahead = read(tile + step);
  }
  __device__ bool read(int t) const {
    if (kFlags == 0 || !alive || t >= tiles) return true;
    const uint8_t* p = alive + (int64_t)t * kFlags;
    if (kFlags == 4) return __ldcg(reinterpret_cast<const unsigned*>(p)) != 0;
    const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
    return (v.x | v.y) != 0;
  }
  __device__ bool more() const { return tile < tiles; }
  __device__ void next() {
    tile += step;
    ++n;
    live = ahead;
    ahead = read(tile + step);
  }
  __device__ bool last() const { return tile + step >= tiles; }
  // whether a run of tiles is complete after this one
  __device__ bool ends(int run) const { return last() || (n + 1) % run == 0; }
};

struct Ring {
  int n, at;
  uint32_t phase;
  __device__ explicit Ring(int count) : n(count), at(0), phase(0) {}
  __device__ void next() {
    if (++at == n) {
      at = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ void give_up(int* err, volatile int* abort) {
  set_error(err, kDevTimeout);
  *abort = 1;
}

// Descriptor of an MN-major operand whose groups of 64 columns are `group` bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t group) {
  return tc::sdesc_k128(saddr) | ((uint64_t)(group >> 4) << 16);
}
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;

// kGroups: of 64 experts; kPacked: up to 32.
template <int kGroups, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1) gate_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ __align__(8) uint64_t s_bar[3 * kMaxX + 2 * kMaxPanels + 11];
  const Plan plan(P.E);
  const uint32_t sW = (tc::smem_u32(smem_raw) + 1023u) & ~1023u, sX = sW + plan.wg_bytes();
  const uint32_t sP = sX + plan.nx * kXBytes, sOut = sP + plan.np * plan.per * kHalf;
  const uint32_t bars = tc::smem_u32(s_bar);
  auto x_full = [&](int s) { return bars + 8 * s; };
  auto x_clean = [&](int s) { return bars + 8 * (kMaxX + s); };      // masked rows zeroed
  auto x_empty = [&](int s) { return bars + 8 * (2 * kMaxX + s); };
  auto p_full = [&](int s) { return bars + 8 * (3 * kMaxX + s); };
  auto p_empty = [&](int s) { return bars + 8 * (3 * kMaxX + kMaxPanels + s); };
  const uint32_t more = bars + 8 * (3 * kMaxX + 2 * kMaxPanels);
  const uint32_t w_full = more, done = more + 16;
  auto d1_full = [&](int a) { return more + 24 + 8 * a; };
  auto d1_empty = [&](int a) { return more + 40 + 8 * a; };
  auto d2_full = [&](int a) { return more + 56 + 8 * a; };
  auto d2_empty = [&](int a) { return more + 72 + 8 * a; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kMaxX; ++s) {
        tc::mbar_init(x_full(s), 1);
        tc::mbar_init(x_clean(s), 1);
        tc::mbar_init(x_empty(s), 1);
      }
      for (int s = 0; s < kMaxPanels; ++s) {
        tc::mbar_init(p_full(s), s == 0 ? 1 + P.stall : 1);
        tc::mbar_init(p_empty(s), 1);
      }
      tc::mbar_init(w_full, 1);
      for (int a = 0; a < 2; ++a) {
        tc::mbar_init(d1_full(a), 1);
        tc::mbar_init(d1_empty(a), kEpiWarps);
        tc::mbar_init(d2_full(a), 1);
        tc::mbar_init(d2_empty(a), kEpiWarps);
      }
      tc::mbar_init(done, 1);
      s_abort = 0;
      tc::fence_barrier_init();
      tc::fence_proxy_async_smem();
    }
  } else if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&s_tmem), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // What was on the stream before the call is complete: the kernel before
  // lets this one start only then.  x and Wg need no more, the rest waits for
  // that kernel.
  if (warp != 0 || P.alive) pdl_wait();
  // No early start for the sums behind it: beside this kernel they cost more
  // than their launch (the call on 32768 padded tokens 99.7 -> 98.3 us, on the
  // prefill layer 28.9 -> 28.1).
  const uint32_t tmem = s_tmem;
  const int chunk = blockIdx.x % P.chunks, h0 = chunk * kCols;
  const int first = blockIdx.x / P.chunks, splits = gridDim.x / P.chunks;
  const bool dwg = P.part != nullptr;
  constexpr int kRun = kGroups <= 2 ? 1 : 4;   // tiles that D1 sums
  // a tile none of whose tokens counts is not loaded; sums of several tiles take each
  constexpr int kPer = kPacked ? 2 : 1, kSlot = kPer * kHalf;
  constexpr int kD2 = 256;   // TMEM columns: D1 at 0 (and 128), D2 twice 128
  constexpr int kFlags = kRun > 1 ? 0 : kGroups == 2 ? 8 : 4;
  const uint8_t* alive = P.alive;
  // the producers' copies: stages filled and the parity of each one's latest
  uint32_t filled = 0, fill_par = 0;
  bool w_loaded = false;

  if (warp == 0) {
    // ------------------------------------------------------------ x and Wg
    if (tc::elect_one()) {
      Ring r(plan.nx);
      bool ok = true;
      if (P.dx_on) {
        tc::mbar_arrive_expect_tx(w_full, (uint32_t)plan.wg_bytes());
        for (int half = 0; half < 2; ++half)
          for (int e = 0; e < kGroups * 64; e += 32)
            tc::tma_load_2d(sW + half * kGroups * 64 * 128 + e * 128, &P.wg, w_full, h0 + half * 64, kPacked ? 0 : e);
        w_loaded = true;
      }
      for (Walk<kFlags> w(first, splits, P.tiles, alive); w.more() && ok; w.next()) {
        const int t0 = w.tile * kTok;
        if (!dwg || !w.live) continue;
        ok = tc::mbar_wait(x_empty(r.at), r.phase ^ 1u, &s_abort, kWaitNs);
        if (!ok) break;
        tc::mbar_arrive_expect_tx(x_full(r.at), kXBytes);
        tc::tma_load_2d(sX + r.at * kXBytes, &P.x, x_full(r.at), h0, t0);
        tc::tma_load_2d(sX + r.at * kXBytes + kHalf, &P.x, x_full(r.at), h0 + 64, t0);
        filled |= 1u << r.at;
        fill_par = (fill_par & ~(1u << r.at)) | (r.phase << r.at);
        r.next();
      }
      if (!ok) give_up(P.err, &s_abort);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ panels
    if (tc::elect_one()) {
      Ring r(plan.np);
      bool ok = true;
      for (Walk<kFlags> w(first, splits, P.tiles, alive); w.more() && ok; w.next()) {
        const int t0 = w.tile * kTok;
        for (int p = 0; p < plan.panels && w.live; p += kPer) {
          ok = tc::mbar_wait(p_empty(r.at), r.phase ^ 1u, &s_abort, kWaitNs);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(p_full(r.at), kSlot);
          // one by one, the low parts come first
          const int at = kPacked ? p : (2 - p / kGroups) * kGroups + p % kGroups;
          for (int u = 0; u < kPer; ++u)
            tc::tma_load_2d(sP + r.at * kSlot + u * kHalf, &P.panel, p_full(r.at), (at + u) * 64, t0);
          filled |= 1u << r.at;
          fill_par = (fill_par & ~(1u << r.at)) | (r.phase << r.at);
          r.next();
        }
      }
      if (!ok) give_up(P.err, &s_abort);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    // This thread's own latency counts: a wait takes 200 cycles even on a
    // barrier that is complete, so the next ones are looked at before MMAs are
    // issued, and the loops are unrolled (rolled ones took 6600 cycles a tile of
    // 64 experts where the MMAs take 1700).
    if (tc::elect_one()) {
      constexpr int kSlots = kPacked ? 1 : 3 * kGroups;   // of a tile
      constexpr uint32_t id1 = tc::idesc_bf16_f32(kCols, kPer * 64) | kMajorA | kMajorB;
      constexpr uint32_t id2 = tc::idesc_bf16_f32(kTok, kCols) | kMajorB;
      Ring x(plan.nx), p(plan.np), d1(plan.bufs), d2(2);
      const uint64_t x0 = sdesc_mn(sX, kHalf), p_mn = sdesc_mn(sP, kHalf), p_k = tc::sdesc_k128(sP);
      const uint64_t w0 = sdesc_mn(sW, kGroups * 64 * 128);
      const bool dx_on = P.dx_on, clean = P.mask != nullptr;
      auto x_bar = [&](int at) { return clean ? x_clean(at) : x_full(at); };
      bool begins = true;   // D1 with this tile
      bool ok = !dx_on || tc::mbar_wait(w_full, 0, &s_abort, kWaitNs);
      bool x_ready = false, p_ready = false, d1_ready = false;
#pragma unroll 1
      for (Walk<kFlags> w(first, splits, P.tiles, alive); w.more() && ok; w.next()) {
        const bool fresh = begins;
        begins = w.ends(kRun);
        if (!w.live) continue;
        if (dwg) {
          if (ok && fresh && !d1_ready) ok = tc::mbar_wait(d1_empty(d1.at), d1.phase ^ 1u, &s_abort, kWaitNs);
          if (ok && !x_ready) ok = tc::mbar_wait(x_bar(x.at), x.phase, &s_abort, kWaitNs);
        }
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t a1 = x0 + (uint32_t)(x.at * (kXBytes >> 4));
        const uint32_t to1 = tmem + d1.at * 128, to2 = tmem + kD2 + d2.at * kCols;
        const int x_at = x.at, d1_at = d1.at, d2_at = d2.at;
        const uint32_t d2_phase = d2.phase;
        if (dwg) {
          x.next();
          if (begins) d1.next();
        }
        if (dx_on) d2.next();
#pragma unroll
        for (int n = 0; n < kSlots; ++n) {
          if (!p_ready && !tc::mbar_wait(p_full(p.at), p.phase, &s_abort, kWaitNs)) {
            ok = false;
            break;
          }
          const int here = p.at, g = n % kGroups;
          p.next();
          p_ready = tc::mbar_test_wait(p_full(p.at), p.phase);
          if (n == kSlots - 1) {
            x_ready = dwg && tc::mbar_test_wait(x_bar(x.at), x.phase);
            d1_ready = dwg && begins && tc::mbar_test_wait(d1_empty(d1.at), d1.phase ^ 1u);
          }
          const uint32_t off = (uint32_t)(here * (kSlot >> 4));
          if (dwg) {
            const uint64_t b1 = p_mn + off;
            // the first panel of a group starts its sums
            const uint32_t on = n < kGroups && fresh ? 0u : 1u;
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)
              tc::mma_bf16(to1 + g * 64, a1 + k * (2048 >> 4), b1 + k * (2048 >> 4), id1, k ? 1u : on);
          }
          if (dx_on && n == 0) {   // D1's MMAs run while the epilogue empties D2
            if (!tc::mbar_wait(d2_empty(d2_at), d2_phase ^ 1u, &s_abort, kWaitNs)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
          }
          if (dx_on && (kPacked || n >= kGroups)) {   // high and middle parts
            const uint64_t a2 = p_k + off, b2 = w0 + (uint32_t)(g * (64 * 128 >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_bf16(to2, a2 + k * (32 >> 4), b2 + k * (2048 >> 4), id2, n > kGroups || k ? 1u : 0u);
          }
          tc::tc_commit(p_empty(here));
        }
        if (!ok) break;
        if (dwg) {
          tc::tc_commit(x_empty(x_at));
          if (begins) tc::tc_commit(d1_full(d1_at));
        }
        if (dx_on) {
          tc::tc_commit(d2_full(d2_at));
        }
      }
      if (!ok) give_up(P.err, &s_abort);
      tc::tc_commit(done);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ masked rows of x
    if (dwg && P.mask) {
      Ring x(plan.nx);
      // the mask's bytes of the next tile are on their way while this one's rows are zeroed
      uint8_t on[4];
      auto fetch = [&](int tile) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t t = (int64_t)tile * kTok + k * 32 + lane;
          on[k] = t < P.T ? P.mask[t] : 1;
        }
      };
      Walk<kFlags> w(first, splits, P.tiles, alive);
      fetch(w.tile);
      while (w.more()) {
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = __ballot_sync(0xffffffffu, !on[k]);
        const bool live = w.live;
        w.next();
        if (w.more()) fetch(w.tile);
        if (!live) continue;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(x_full(x.at), x.phase, &s_abort, kWaitNs))) {
          if (lane == 0) give_up(P.err, &s_abort);
          break;
        }
        if (out[0] | out[1] | out[2] | out[3]) {
          uint8_t* tile = smem_raw + (sX + x.at * kXBytes - tc::smem_u32(smem_raw));
          // 16 bytes a lane: a row of both halves at a time
          uint8_t* mine = tile + (lane >> 4 & 1) * kHalf + (lane & 7) * 16;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            // the lanes' bit 3 takes every other one of the rows
            for (uint32_t rest = out[k]; rest;) {
              const int r0 = __ffs(rest) - 1;
              rest &= rest - 1;
              const int r1 = rest ? __ffs(rest) - 1 : r0;
              rest &= rest - 1;
              *reinterpret_cast<uint4*>(mine + (k * 32 + (lane & 8 ? r1 : r0)) * 128) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(x_clean(x.at));
        x.next();
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;   // TMEM lanes 32 q .. 32 q + 31, columns
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t buf = sOut + (warp - 4) * kStoreBytes;
    uint8_t* row = smem_raw + (buf - tc::smem_u32(smem_raw)) + lane * 128;
    Ring d1(plan.bufs), d2(2);
    float sum[kGroups * 32] = {};   // of column half * 32 + j of each group: this thread's column of x
    bool ok = true;
    for (Walk<kFlags> w(first, splits, P.tiles, alive); w.more() && ok; w.next()) {
      if (P.dx_on) {
        const int64_t t0 = (int64_t)w.tile * kTok + q * 32;
        uint32_t r[2][32] = {};
        if (w.live) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(d2_full(d2.at), d2.phase, &s_abort, kWaitNs));
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t at = lanes + kD2 + d2.at * kCols + half * 64;
          tc::tmem_ld_32x32b_x32(at, r[0]);
          tc::tmem_ld_32x32b_x32(at + 32, r[1]);
          tc::tmem_wait_ld();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(d2_empty(d2.at));   // tensor memory has been read
          d2.next();
        }
        if (lane == 0) tc::bulk_wait_read();   // the last tile's store has read the buffer
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[k][j]);
#pragma unroll
          for (int j = 0; j < 4; ++j)   // 16 bytes at the place that the 128-byte swizzle gives them
            *reinterpret_cast<uint4*>(row + (((k * 4 + j) ^ (lane & 7)) << 4)) = Vec<bf16>::pack(v + j * 8);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && t0 < P.T && h0 + half * 64 < P.H)
          tc::tma_store_2d(&P.dx, buf, h0 + half * 64, (int)t0);
      }
      if (dwg && w.live && w.ends(kRun)) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(d1_full(d1.at), d1.phase, &s_abort, kWaitNs));
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          uint32_t r[32];
          tc::tmem_ld_32x32b_x32(lanes + d1.at * 128 + g * 64 + half * 32, r);
          tc::tmem_wait_ld();
          if (kPacked && half) {   // to the middle parts' sums the low ones'
            uint32_t m[32];
            tc::tmem_ld_32x32b_x32(lanes + d1.at * 128 + 64, m);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(m[j]));
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[g * 32 + j] += __uint_as_float(r[j]);
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(d1_empty(d1.at));
        d1.next();
      }
    }
    if (ok && dwg) {
      // up to 32 experts both halves have sums of the same experts: a row each
      const int64_t slot = ((int64_t)chunk * splits + first) * (kPacked ? 2 : 1) + (kPacked ? half : 0);
      float* out = P.part + slot * P.E * kCols + q * 32 + lane;
#pragma unroll
      for (int j = 0; j < kGroups * 32; ++j) {
        const int e = kPacked ? j : j / 32 * 64 + half * 32 + j % 32;
        if (e < P.E) out[(int64_t)e * kCols] = sum[j];
      }
    }
    if (!ok && lane == 0) give_up(P.err, &s_abort);
    if (lane == 0) tc::bulk_wait_all();
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (s_abort && (filled || w_loaded)) {   // the producing threads: every copy lands before the CTA leaves
    if (w_loaded) tc::mbar_wait(w_full, 0, nullptr, kWaitNs);
    for (int s = 0; s < (warp == 0 ? plan.nx : plan.np); ++s)
      if ((filled >> s) & 1u) tc::mbar_wait(warp == 0 ? x_full(s) : p_full(s), (fill_par >> s) & 1u, nullptr, kWaitNs);
  }
  if (warp == 1) {
    // and every MMA has finished before its memory is freed
    if (lane == 0 && !tc::mbar_wait(done, 0, nullptr, kWaitNs)) set_error(P.err, kDevTimeout);
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// dWg: a chunk's rows of partial sums in their order; the last blocks: the
// bias' gradient, the rows of partial sums in order.
__global__ void __launch_bounds__(256)
gate_sums_kernel(const float* __restrict__ part, int rows, int chunks, int E, int H,
                 float* __restrict__ dWg, const float* __restrict__ part_b, int rows_b, float* __restrict__ dbias) {
  pdl_enter();
  const int c = blockIdx.x;
  if (c < chunks) {
    const int e = blockIdx.y * 8 + threadIdx.x / 32, h = c * kCols + threadIdx.x % 32 * 4;
    if (e >= E || h >= H) return;   // H is a multiple of 8
    const float* p = part + ((int64_t)c * rows * E + e) * kCols + threadIdx.x % 32 * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = rows; k > 0; --k, p += (int64_t)E * kCols) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    *reinterpret_cast<float4*>(dWg + (int64_t)e * H + h) = s;
  } else {
    __shared__ float s_b[8][32];
    const int e = blockIdx.y * 32 + threadIdx.x % 32, g = threadIdx.x / 32;
    float v = 0.f;
    if (e < E && blockIdx.y * 32 < E)
#pragma unroll 8
      for (int r = g; r < rows_b; r += 8) v += part_b[(int64_t)r * E + e];
    s_b[g][threadIdx.x % 32] = v;
    __syncthreads();
    if (g == 0 && e < E) {
      for (int k = 1; k < 8; ++k) v += s_b[k][threadIdx.x];
      dbias[e] = v;
    }
  }
}

}  // namespace

// CTAs of a chunk.
static int64_t gate_splits(const Shape& s) {
  const int64_t n = sm_count() / ((s.H + kCols - 1) / kCols), tiles = (s.T + kTok - 1) / kTok, most = n < 1 ? 1 : n;
  return tiles < most ? (tiles < 1 ? 1 : tiles) : most;
}
int64_t gate_part_floats(const Shape& s) {
  const int64_t chunks = (s.H + kCols - 1) / kCols;
  return chunks * gate_splits(s) * (Plan(s.E).packed ? 2 : 1) * s.E * kCols;
}
int gate_panel_cols(int E) { return Plan(E).panels * 64; }
// Not where a sum goes over several tiles: there each of them is taken.
bool gate_skips_tiles(int E) { return E <= 128; }

cudaError_t launch_gate_tc(const Shape& s, const RouterBackward& b, const void* panels, const uint8_t* alive, float* part,
                           const float* part_b, int rows_b, int* err, cudaStream_t st) {
  const Plan plan(s.E);
  const int64_t tiles = (s.T + kTok - 1) / kTok, chunks = (s.H + kCols - 1) / kCols;
  const int splits = (int)gate_splits(s);
  cudaError_t e = cudaSuccess;
  if (b.dx || b.dWg) {
    Params P = {};
    const uint64_t T = (uint64_t)s.T, H = (uint64_t)s.H;
    if ((b.dWg && !tma_map_bf16(&P.x, b.x, T, H, kTok)) ||
        (b.dx && (!tma_map_bf16(&P.wg, b.Wg, (uint64_t)s.E, H, 32) || !tma_map_bf16(&P.dx, b.dx, T, H, 32))) ||
        !tma_map_bf16(&P.panel, panels, T, (uint64_t)plan.panels * 64, kTok))
      return cudaErrorNotSupported;
    P.mask = b.mask;
    P.alive = alive;
    P.T = s.T;
    P.tiles = (int)tiles;
    P.chunks = (int)chunks;
    P.E = s.E;
    P.H = s.H;
    P.part = b.dWg ? part : nullptr;
    P.dx_on = b.dx != nullptr;
    P.err = err;
    P.stall = (s.flags & MOE_FLAG_TEST_WAIT_TIMEOUT) ? 1 : 0;
    auto kern = plan.packed        ? gate_kernel<1, true>
                : plan.groups == 1 ? gate_kernel<1, false>
                : plan.groups == 2 ? gate_kernel<2, false>
                : plan.groups == 3 ? gate_kernel<3, false>
                                   : gate_kernel<4, false>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.smem());
    if (e != cudaSuccess) return e;
    e = launch_kernel(kern, dim3((unsigned)(splits * chunks)), dim3(kThreads), plan.smem(), st, 1, P);
  }
  if (e == cudaSuccess && (b.dWg || b.dbias)) {
    const int cols = b.dWg ? (int)chunks : 0;
    e = launch_kernel(gate_sums_kernel, dim3((unsigned)(cols + (b.dbias ? 1 : 0)), (unsigned)((s.E + 7) / 8)), dim3(256),
                      0, st, 1, part, splits * (plan.packed ? 2 : 1), cols, s.E, s.H, b.dWg, part_b, rows_b, b.dbias);
  }
  return e;
}

}  // namespace moe
