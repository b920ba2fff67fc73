// AdamW over many tensors in one launch, with the moments in 32 bits or in
// 8 bits with a scale for every 256 elements.
//
// For every element, with g = grad (times *grad_scale) in fp32 and step t:
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// 8-bit moments hold m and r = sqrt(v) (a square root halves v's exponent
// range) as e4m3 codes: with A the largest magnitude of the 256 elements of a
// block, code = e4m3(x (1 / A) 448) rounded to nearest even and scale = A / 448.
// A non-zero r keeps a non-zero code (at least 2^-9), so that no element's
// divisor falls to eps alone by rounding.  A block with A < 2^-100 is held as
// zeros.  A block with a NaN or an infinity gets that A as its scale and codes
// of 0 and NaN, so that all of it reads back as NaN: loud, not silently clipped.
//
// Every operation of the moments rounds by itself (no fused multiply-add), in
// the order written above, so that a code is a function of its inputs alone.
// The parameter's own update may fuse, and its quotient is the fast one (2
// units of the last place of an update that is itself a small part of p): with
// IEEE quotients the 8-bit step was bound by instructions, 1719 us for 587 M
// elements.  (A divisor is eps or at least 3e-23, the square root of the
// smallest fp32 number.)
//
// A warp takes one block of 256 elements: lane l holds elements 4 l .. 4 l + 3
// of both halves, so each load of the warp is contiguous; A is a warp maximum.
// The eight warps of a thread block take consecutive blocks, whose scales fill
// one 32-byte sector.  (Several blocks to a warp, one after the other, were
// slower by a third: 2.1 ms.  A grid that fits the GPU once, striding, took
// 647 us instead of 578 with moments in 32 bits.)
//
// Bound by memory: 28 bytes an element (moments in 32 bits, bf16 gradient, a
// bf16 copy of p) or 16 bytes and 16 / 256 of scales.  Measured: 578 us for
// 147 M elements (7.1 TB/s), in 8 bits 1545 us for 587 M (6.1 TB/s; two thirds
// of the issue slots are taken too).
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kBlock = MOE_ADAMW_BLOCK;   // elements that share a scale
constexpr int kWarps = 8;
constexpr int kPer = 8;                   // elements a lane holds
static_assert(kBlock == 32 * kPer, "a warp holds a block");
constexpr uint32_t kTinyBits = (127u - 100u) << 23;   // 2^-100
constexpr uint32_t kInfBits = 0x7f800000u;

// One tensor of a launch.
struct Slot {
  float* p;
  bf16* p16;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float keep;      // 1 - lr * weight decay
};

template <int kCap>
struct Slots {
  Slot s[kCap];
  uint32_t first[kCap];   // the number of blocks before a tensor's
  int count;
  uint32_t blocks;
};

struct Step {
  float beta1, one_minus_beta1, beta2, one_minus_beta2, inv_sqrt_c2, eps, lr_c1;
};

// Tensors a launch can take.  Its parameters travel with it, so that few
// tensors take a short list (40: 3 KB, 128: 9 KB, 400: 29 KB; a launch costs
// about 3 us more with the longest); they have to stay below 32764 bytes.
constexpr int kSmallCap = 40, kMiddleCap = 128, kLargeCap = 400;
static_assert(sizeof(Slots<kLargeCap>) + sizeof(Step) + 32 < 32764, "kernel parameters");

// Element 4 l + i of half h: the lane's value h * 4 + i.
template <bool kFull>
__device__ __forceinline__ int element(int lane, int c) {
  return (c >> 2) * 128 + lane * 4 + (c & 3);
}

// kPer elements of this lane from src (the block's first element), 0 past `left`.
template <bool kFull>
__device__ __forceinline__ void load(const float* src, int lane, int left, float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 f = *reinterpret_cast<const float4*>(src + h * 128 + lane * 4);
      v[h * 4] = f.x; v[h * 4 + 1] = f.y; v[h * 4 + 2] = f.z; v[h * 4 + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      v[c] = i < left ? src[i] : 0.f;
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void load(const bf16* src, int lane, int left, float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint2 u = *reinterpret_cast<const uint2*>(src + h * 128 + lane * 4);
      const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&u);
      const float2 lo = __bfloat1622float2(b[0]), hi = __bfloat1622float2(b[1]);
      v[h * 4] = lo.x; v[h * 4 + 1] = lo.y; v[h * 4 + 2] = hi.x; v[h * 4 + 3] = hi.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      v[c] = i < left ? __bfloat162float(src[i]) : 0.f;
    }
  }
}
// e4m3 codes, exact in half and in fp32
__device__ __forceinline__ float decode1(uint8_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}
template <bool kFull>
__device__ __forceinline__ void load(const uint8_t* src, int lane, int left, float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(src + h * 128 + lane * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        v[h * 4 + 2 * i] = f.x;
        v[h * 4 + 2 * i + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      v[c] = i < left ? decode1(src[i]) : 0.f;
    }
  }
}

template <bool kFull>
__device__ __forceinline__ void store(float* dst, int lane, int left, const float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(dst + h * 128 + lane * 4) =
          make_float4(v[h * 4], v[h * 4 + 1], v[h * 4 + 2], v[h * 4 + 3]);
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      if (i < left) dst[i] = v[c];
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void store(bf16* dst, int lane, int left, const float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 u;
      __nv_bfloat162* b = reinterpret_cast<__nv_bfloat162*>(&u);
      b[0] = __floats2bfloat162_rn(v[h * 4], v[h * 4 + 1]);
      b[1] = __floats2bfloat162_rn(v[h * 4 + 2], v[h * 4 + 3]);
      *reinterpret_cast<uint2*>(dst + h * 128 + lane * 4) = u;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      if (i < left) dst[i] = __float2bfloat16_rn(v[c]);
    }
  }
}
template <bool kFull>
__device__ __forceinline__ void store(uint8_t* dst, int lane, int left, const float* v) {
  if (kFull) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t u = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        u |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[h * 4 + 2 * i], v[h * 4 + 2 * i + 1]), __NV_SATFINITE,
                                                __NV_E4M3)
             << (16 * i);
      *reinterpret_cast<uint32_t*>(dst + h * 128 + lane * 4) = u;
    }
  } else {
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const int i = element<false>(lane, c);
      if (i < left) dst[i] = __nv_cvt_float_to_fp8(v[c], __NV_SATFINITE, __NV_E4M3);
    }
  }
}

// The largest magnitude of three; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The block's values as codes and its scale (lane 0 writes it).  Elements
// past the tensor's end are zeros and do not count.
template <bool kFull, bool kKeepNonZero>
__device__ __forceinline__ void encode(const float* x, uint8_t* codes, float* scale, int lane, int left) {
  float top = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; c += 2) top = max_abs(top, x[c], x[c + 1]);
  const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // as bits: NaN > infinity > finite
  const float A = __uint_as_float(bits);
  const bool finite = bits < kInfBits, big = bits >= kTinyBits && finite;
  const float inv = big ? __fmul_rn(__frcp_rn(A), 448.f) : 0.f;
  const float least = big ? 0.001953125f : 0.f;   // 2^-9, the smallest code
  float y[kPer];
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    y[c] = __fmul_rn(x[c], inv);
    if (kKeepNonZero && x[c] > 0.f) y[c] = fmaxf(y[c], least);
  }
  store<kFull>(codes, lane, left, y);
  if (lane == 0) *scale = big ? __fmul_rn(A, 1.0f / 448.0f) : (finite ? 0.f : A);
}

template <bool kFull, typename TG, bool kEight>
__device__ __forceinline__ void update_block(const Slot& s, uint32_t block, const Step& q, float grad_scale, int lane) {
  const int64_t at = (int64_t)block * kBlock;
  const int left = kFull ? kBlock : (int)min((int64_t)kBlock, s.n - at);
  float p[kPer], g[kPer], m[kPer], v[kPer];
  load<kFull>(s.p + at, lane, left, p);
  load<kFull>((const TG*)s.g + at, lane, left, g);
  if (kEight) {
    load<kFull>((const uint8_t*)s.m + at, lane, left, m);
    load<kFull>((const uint8_t*)s.v + at, lane, left, v);
    const float ms = s.m_scale[block], vs = s.v_scale[block];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      m[c] = __fmul_rn(m[c], ms);
      const float r = __fmul_rn(v[c], vs);
      v[c] = __fmul_rn(r, r);
    }
  } else {
    load<kFull>((const float*)s.m + at, lane, left, m);
    load<kFull>((const float*)s.v + at, lane, left, v);
  }
#pragma unroll
  for (int c = 0; c < kPer; ++c) {
    const float gc = __fmul_rn(g[c], grad_scale);
    m[c] = __fadd_rn(__fmul_rn(m[c], q.beta1), __fmul_rn(gc, q.one_minus_beta1));
    v[c] = __fadd_rn(__fmul_rn(v[c], q.beta2), __fmul_rn(__fmul_rn(gc, gc), q.one_minus_beta2));
    const float r = __fsqrt_rn(v[c]);
    p[c] = fmaf(p[c], s.keep, -q.lr_c1 * __fdividef(m[c], fmaf(r, q.inv_sqrt_c2, q.eps)));
    if (kEight) v[c] = r;
  }
  store<kFull>(s.p + at, lane, left, p);
  if (s.p16) store<kFull>(s.p16 + at, lane, left, p);
  if (kEight) {
    encode<kFull, false>(m, (uint8_t*)s.m + at, s.m_scale + block, lane, left);
    encode<kFull, true>(v, (uint8_t*)s.v + at, s.v_scale + block, lane, left);
  } else {
    store<kFull>((float*)s.m + at, lane, left, m);
    store<kFull>((float*)s.v + at, lane, left, v);
  }
}

template <int kCap, typename TG, bool kEight>
__global__ void __launch_bounds__(32 * kWarps)
adamw_kernel(const __grid_constant__ Slots<kCap> t, const __grid_constant__ Step q, const float* grad_scale,
             const int32_t* skip) {
  pdl_enter();
  if (skip && *skip != 0) return;
  const float gs = grad_scale ? *grad_scale : 1.0f;
  const int lane = threadIdx.x & 31;
  const uint32_t at = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (at >= t.blocks) return;
  int cur = 0, hi = t.count - 1;
  while (cur < hi) {   // the last tensor that starts at or before this block
    const int mid = (cur + hi + 1) >> 1;
    if (t.first[mid] <= at) cur = mid; else hi = mid - 1;
  }
  const Slot& s = t.s[cur];
  const uint32_t block = at - t.first[cur];
  // vector loads and stores need 16-byte aligned tensors and a whole block
  const uintptr_t all = (uintptr_t)s.p | (uintptr_t)s.p16 | (uintptr_t)s.g | (uintptr_t)s.m | (uintptr_t)s.v;
  if ((all & 15u) == 0 && ((int64_t)block + 1) * kBlock <= s.n)
    update_block<true, TG, kEight>(s, block, q, gs, lane);
  else
    update_block<false, TG, kEight>(s, block, q, gs, lane);
}

template <int kCap, typename TG, bool kEight>
cudaError_t run_adamw(const moe_adamw_tensor* tensors, int count, const Step& q, double lr, const float* grad_scale,
                      const int32_t* skip, cudaStream_t st) {
  int i = 0;
  while (i < count) {
    Slots<kCap> t;
    t.count = 0;
    uint64_t blocks = 0;
    for (; i < count && t.count < kCap; ++i) {
      const moe_adamw_tensor& x = tensors[i];
      if (x.n == 0) continue;
      const uint64_t nb = ((uint64_t)x.n + kBlock - 1) / kBlock;
      if (t.count > 0 && blocks + nb >= (1ull << 31)) break;   // block numbers stay in 32 bits
      Slot& s = t.s[t.count++];
      s.p = x.p;
      s.p16 = (bf16*)x.p_bf16;
      s.g = x.grad;
      s.m = x.m;
      s.v = x.v;
      s.m_scale = x.m_scale;
      s.v_scale = x.v_scale;
      s.n = x.n;
      t.first[t.count - 1] = (uint32_t)blocks;
      s.keep = (float)(1.0 - lr * (double)x.weight_decay);
      blocks += nb;
    }
    if (t.count == 0) break;
    t.blocks = (uint32_t)blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((blocks + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void* args[] = {&t, const_cast<Step*>(&q), &grad_scale, &skip};   // the list is copied once, by the launch
    const cudaError_t e = cudaLaunchKernelExC(&cfg, (const void*)adamw_kernel<kCap, TG, kEight>, args);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int kCap>
cudaError_t pick_adamw(const moe_adamw_tensor* tensors, int count, int grad_dtype, int state_bits, const Step& q,
                       double lr, const float* gs, const int32_t* skip, cudaStream_t st) {
  if (grad_dtype == MOE_BF16)
    return state_bits == 8 ? run_adamw<kCap, bf16, true>(tensors, count, q, lr, gs, skip, st)
                           : run_adamw<kCap, bf16, false>(tensors, count, q, lr, gs, skip, st);
  return state_bits == 8 ? run_adamw<kCap, float, true>(tensors, count, q, lr, gs, skip, st)
                         : run_adamw<kCap, float, false>(tensors, count, q, lr, gs, skip, st);
}

}  // namespace

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int count, int grad_dtype, int state_bits,
                         const moe_adamw_params& h, const float* grad_scale, const int32_t* skip, cudaStream_t st) {
  Step q;
  q.beta1 = (float)h.beta1;
  q.one_minus_beta1 = (float)(1.0 - h.beta1);
  q.beta2 = (float)h.beta2;
  q.one_minus_beta2 = (float)(1.0 - h.beta2);
  q.inv_sqrt_c2 = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)h.step)));
  q.eps = h.eps < 1e-30 ? 0.f : (float)h.eps;   // the fast quotient wants a divisor whose reciprocal is a normal number
  q.lr_c1 = (float)(h.lr / (1.0 - pow(h.beta1, (double)h.step)));
  auto pick = count <= kSmallCap ? pick_adamw<kSmallCap>
                                 : count <= kMiddleCap ? pick_adamw<kMiddleCap> : pick_adamw<kLargeCap>;
  return pick(tensors, count, grad_dtype, state_bits, q, h.lr, grad_scale, skip, st);
}

}  // namespace moe
