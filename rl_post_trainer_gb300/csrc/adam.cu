// adam.cu -- the optimizer step in front of the encode: global gradient norm,
// AdamW over a plan's tensors with FP32 or 8-bit moments, and the 8-bit
// moments' export. The formulas are those of include/pulse.h.
#include <cmath>

#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

constexpr uint32_t kMixA = 0xBB67AE85u;  // odd; the fraction of sqrt(3)
constexpr uint32_t kMixB = 0x9E3779B9u;  // odd; the fraction of the golden ratio

// Full-period 32-bit mixer: each xor-shift and each odd product is invertible.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= kMixA;
  x ^= x >> 15;
  x *= kMixB;
  x ^= x >> 16;
  return x;
}

__device__ __forceinline__ float load_grad(const AdamTensorDesc& d, uint64_t i) {
  if (d.grad_bf16) {
    const uint32_t b = static_cast<const uint16_t*>(d.g)[i];
    return __uint_as_float(b << 16);
  }
  return static_cast<const float*>(d.g)[i];
}

// Root and reciprocal are the hardware's, a unit or two off: the update carries that
// relative error, 2^-22, far under its own rounding against the weight. Rounded
// correctly, both cost the step 0.4 % on 1.54 billion parameters (5.62 against 5.59 ms),
// 3.5 % on 60 million at odd offsets (237 against 229 us) and 5 % on 1 million (4.7
// against 4.45 us); with 8-bit moments, which have no instructions to spare, 10 %.
// FULL_RANGE: arguments and results below 2^-126 count as they are, which costs FP32
// moments nothing. Without it they are 0: a second moment that small leaves eps alone in
// the divisor (8-bit moments: 3.41 ms so, 3.45 ms with the full range under the root).
template <bool FULL_RANGE>
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  if (FULL_RANGE)
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool FULL_RANGE>
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  if (FULL_RANGE)
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  else
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Moments and weight of one element. Products and sums of the moments are
// rounded one by one (no fused multiply-add), so that 8-bit codes made from
// them are the same wherever they are computed.
template <bool FULL_RANGE>
__device__ __forceinline__ void adam_element(const AdamLaunch& a, float alpha, float decay, float g,
                                             float& m, float& v, float& w) {
  m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_minus_beta1));
  v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
  const float den = fmaf(sqrt_approx<FULL_RANGE>(v), a.inv_sqrt_bc2, a.eps);
  w -= fmaf(decay, w, alpha * (m * rcp_approx<FULL_RANGE>(den)));
}

// 8 consecutive FP32 values, 32-byte aligned, in one access that leaves L1 alone.
struct F8 {
  float x[8];
};
__device__ __forceinline__ F8 ld_f8(const float* p) {
  F8 r;
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r.x[0]), "=f"(r.x[1]), "=f"(r.x[2]), "=f"(r.x[3]), "=f"(r.x[4]), "=f"(r.x[5]),
                 "=f"(r.x[6]), "=f"(r.x[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void st_f8(float* p, const F8& r) {
  asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(r.x[0]),
               "f"(r.x[1]), "f"(r.x[2]), "f"(r.x[3]), "f"(r.x[4]), "f"(r.x[5]), "f"(r.x[6]), "f"(r.x[7])
               : "memory");
}
// 8 consecutive gradients from element i on.
__device__ __forceinline__ F8 ld_grad8(const AdamTensorDesc& d, uint64_t i) {
  if (!d.grad_bf16) return ld_f8(static_cast<const float*>(d.g) + i);
  const uint4 b = ld_u4_no_l1(static_cast<const uint16_t*>(d.g) + i);
  F8 r;
  const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    r.x[2 * k] = __uint_as_float(u[k] << 16);
    r.x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
  }
  return r;
}

// Each element is read and written once, 26 bytes of traffic with BF16 gradients and
// 28 with FP32 ones, for 36 instructions: bound by memory (it issues in 25 % of its
// cycles). A thread takes one group of 8, whose four loads are all on their way
// before the first is used, and a tile is a CTA's 2,048 elements, so nothing loops.
// 1.54 billion parameters in a decoder's tensors with BF16 gradients: 5.60 ms, 7.17
// TB/s, where a plain copy moves 6.76 TB/s; two groups a thread 6.61 ms, tiles of
// 4,096 to 16,384 5.66 to 5.81 ms, 3 or 5 CTAs per SM 5.73 ms. Tensors whose buffers have no
// common offset go an element a thread, whose narrow accesses cost them half of that
// rate: 60 million parameters with BF16 gradients one element off take 447 us, 221 with all
// on their groups or all one element off.
constexpr int kAdam32Ctas = 4;  // CTAs per SM: 64 registers a thread
__global__ void __launch_bounds__(kAdamThreads, kAdam32Ctas)
    adam32_kernel(const __grid_constant__ AdamLaunch a) {
  stream_ready();
  const AdamTensorDesc d = a.tensors[a.tile_tensor[blockIdx.x]];
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  if (d.g == nullptr || !isfinite(scale)) return;
  const float alpha = a.alpha * d.lr_scale, decay = a.lr * d.lr_scale * d.weight_decay;
  const uint64_t tile = (blockIdx.x - d.tile_begin) * kAdam32Tile;
  const uint64_t n = d.n;
  float* pw = d.w;
  float* pm = static_cast<float*>(d.m);
  float* pv = static_cast<float*>(d.v);
  auto one = [&](uint64_t i) {
    float m = pm[i], v = pv[i], w = pw[i];
    adam_element<true>(a, alpha, decay, load_grad(d, i) * scale, m, v, w);
    pm[i] = m;
    pv[i] = v;
    pw[i] = w;
  };
  if (d.lead == kAdamNoGroups) {
    for (int j = threadIdx.x; j < kAdam32Tile && tile + j < n; j += kAdamThreads) one(tile + j);
    return;
  }
  // groups start `lead` elements in; the first tile takes the elements before them
  if (tile == 0 && threadIdx.x < d.lead && threadIdx.x < n) one(threadIdx.x);
  const uint64_t first = tile + d.lead + threadIdx.x * 8u;
  static_assert(kAdam32Tile == 8 * kAdamThreads, "one group a thread");
  if (first + 8 <= n) {
    F8 w = ld_f8(pw + first), m = ld_f8(pm + first), v = ld_f8(pv + first);
    const F8 g = ld_grad8(d, first);
#pragma unroll
    for (int k = 0; k < 8; ++k) adam_element<true>(a, alpha, decay, g.x[k] * scale, m.x[k], v.x[k], w.x[k]);
    st_f8(pw + first, w);
    st_f8(pm + first, m);
    st_f8(pv + first, v);
  } else {
    for (uint64_t k = first; k < n && k < first + 8; ++k) one(k);
  }
}

// ------------------------------------------------------------ 8-bit moments

// First FP32 exponent field of the codes, at the position of the code: the
// value of code c > 0 has the bits base + (c << 20).
__device__ __forceinline__ uint32_t m_base(uint32_t e) { return (e - 14u) << 23; }
__device__ __forceinline__ uint32_t v_base(uint32_t e) { return (e - 30u) << 23; }

// Exponent bytes of zeroed state are 0: every code there is 0 and reads as 0.
__device__ __forceinline__ float decode_m(uint32_t code, uint32_t e) {
  const uint32_t c = code & 0x7Fu;
  if (e == 0xFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((c ? m_base(e) + (c << 20) : 0u) | ((code & 0x80u) << 24));
}
__device__ __forceinline__ float decode_v(uint32_t code, uint32_t e) {
  if (e == 0xFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(code ? v_base(e) + (code << 20) : 0u);
}

__device__ __forceinline__ uint32_t block_key(uint32_t key, uint64_t block) {
  return mix32(key ^ mix32(uint32_t(block) ^ mix32(uint32_t(block >> 32))));
}

// Codes of one element from the new moments and the blocks' exponents.
__device__ __forceinline__ uint32_t encode_m(float m, uint32_t e, uint32_t r) {
  const uint32_t u = __float_as_uint(m), mag = u & 0x7FFFFFFFu;
  const int c = int((mag + (r << 4)) >> 20) - int(e - 14u) * 8;
  return uint32_t(min(max(c, 0), 127)) | ((u >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t encode_v(float v, uint32_t e, uint32_t r) {
  const uint32_t mag = __float_as_uint(v);
  const int c = int((mag + (r << 4)) >> 20) - int(e - 30u) * 8;
  return uint32_t(min(max(c, mag != 0u ? 1 : 0), 255));
}

// One block of 256 elements, any alignment and length: lane l takes elements
// l, l + 32, ...
__device__ __noinline__ void adam8_block_any(const AdamLaunch& a, const AdamTensorDesc* desc,
                                             float scale, float alpha, float decay,
                                             uint64_t block) {
  const AdamTensorDesc& d = *desc;
  uint8_t* pm = static_cast<uint8_t*>(d.m);
  uint8_t* pv = static_cast<uint8_t*>(d.v);
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t base = block * kAdamBlock;
  const uint32_t em = d.m_exp[block], ev = d.v_exp[block];
  float m[8], v[8];
  uint32_t mx = 0, vx = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint64_t i = base + lane + 32 * k;
    m[k] = v[k] = 0.0f;
    if (i < d.n) {
      float w = d.w[i];
      m[k] = decode_m(pm[i], em);
      v[k] = decode_v(pv[i], ev);
      adam_element<false>(a, alpha, decay, load_grad(d, i) * scale, m[k], v[k], w);
      d.w[i] = w;
    }
    mx = max(mx, __float_as_uint(m[k]) & 0x7FFFFFFFu);
    vx = max(vx, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  }
  // exponent field of the largest magnitude; 255 where one is not finite
  const uint32_t me = __reduce_max_sync(0xFFFFFFFFu, mx) >> 23;
  const uint32_t ve = __reduce_max_sync(0xFFFFFFFFu, vx) >> 23;
  const uint32_t me2 = min(max(me, 15u), 253u), ve2 = min(max(ve, 31u), 253u);
  const uint32_t key = block_key(a.key, d.block_begin + block);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t j = lane + 32 * k;
    const uint64_t i = base + j;
    if (i < d.n) {
      const uint32_t h = mix32(key + j * kMixB);
      pm[i] = uint8_t(me == 255u ? 0x7Fu : encode_m(m[k], me2, h >> 16));
      pv[i] = uint8_t(ve == 255u ? 0x7Fu : encode_v(v[k], ve2, h & 0xFFFFu));
    }
  }
  if (lane == 0) {
    d.m_exp[block] = uint8_t(me == 255u ? 0xFFu : me2);
    d.v_exp[block] = uint8_t(ve == 255u ? 0xFFu : ve2);
  }
}

// Two FP32 values in one register pair: products and sums of both with one
// instruction, each rounded to nearest.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The largest and smallest of three; NaN if one of them is (max) or never (min).
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Nonzero if one of the four bytes is zero.
__device__ __forceinline__ uint32_t zero_byte(uint32_t x) {
  return (x - 0x01010101u) & ~x & 0x80808080u;
}

// What the kernel keeps of a tensor, in registers.
struct Adam8Ptrs {
  float* w;
  const void* g;
  uint8_t* m;
  uint8_t* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  float scale, alpha, decay;
};

// A block's data, 8 consecutive elements a lane.
template <bool BF16>
struct Block8 {
  F8 w;
  float g[BF16 ? 4 : 8];  // BF16: pairs as they lie in memory
  uint2 m, v;
};

// ALIGNED: weights and gradients can be read in groups of 8 as well as the codes.
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void load_block8(Block8<BF16>& b, const Adam8Ptrs& p, uint64_t block) {
  const uint64_t i = block * kAdamBlock + (threadIdx.x & 31u) * 8u;
  b.m = ld_u2_no_l1(p.m + i);
  b.v = ld_u2_no_l1(p.v + i);
  if (!ALIGNED) {
#pragma unroll
    for (int k = 0; k < 8; ++k) b.w.x[k] = p.w[i + k];
#pragma unroll
    for (int k = 0; k < (BF16 ? 4 : 8); ++k) {
      if (BF16) {
        const uint16_t* g = static_cast<const uint16_t*>(p.g) + i + 2 * k;
        b.g[k] = __uint_as_float(g[0] | uint32_t(g[1]) << 16);
      } else {
        b.g[k] = static_cast<const float*>(p.g)[i + k];
      }
    }
    return;
  }
  b.w = ld_f8(p.w + i);
  if (BF16) {
    const uint4 u = ld_u4_no_l1(static_cast<const uint16_t*>(p.g) + i);
    b.g[0] = __uint_as_float(u.x), b.g[1] = __uint_as_float(u.y);
    b.g[2] = __uint_as_float(u.z), b.g[3] = __uint_as_float(u.w);
  } else {
    const F8 u = ld_f8(static_cast<const float*>(p.g) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) b.g[BF16 ? 0 : k] = u.x[k];
  }
}

template <bool BF16>
__device__ __forceinline__ uint64_t grad_pair(const Block8<BF16>& b, int pair) {
  if (BF16) {
    const uint32_t u = __float_as_uint(b.g[pair]);
    return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  return pack2(b.g[BF16 ? 0 : 2 * pair], b.g[BF16 ? 0 : 2 * pair + 1]);
}

// A whole block with 8 consecutive elements a lane; key: the block's; em and ev:
// its exponents, old and then new. The new exponents need the maxima of the whole
// block, so a block is a warp's: 256 values in its registers, read and written once.
// Instructions bound this kernel as much as memory does (53 an element, issued in 59 %
// of the cycles, next to 75 % of DRAM's), so the common case is kept short: two
// elements to an arithmetic instruction, codes converted by shifts; zero codes, zero
// second moments, and exponents at the ends of their range (infinities and NaN among
// them) take the general conversions, decided once per warp.
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void adam8_block_full(const AdamLaunch& a, const Adam8Ptrs& p,
                                                 uint64_t block, uint32_t key, Block8<BF16>& b,
                                                 uint32_t& em, uint32_t& ev) {
  const uint32_t lane = threadIdx.x & 31u;
  const uint64_t i = block * kAdamBlock + lane * 8u;
  float m[8], v[8];
  {
    const uint32_t mc[2] = {b.m.x & 0x7F7F7F7Fu, b.m.y & 0x7F7F7F7Fu};
    const uint32_t ms[2] = {b.m.x, b.m.y}, vc[2] = {b.v.x, b.v.y};
    const uint32_t zero = zero_byte(mc[0]) | zero_byte(mc[1]) | zero_byte(vc[0]) | zero_byte(vc[1]);
    if (__any_sync(0xFFFFFFFFu, zero != 0u) || em == 0xFFu || ev == 0xFFu) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = decode_m((ms[k / 4] >> (8 * (k % 4))) & 0xFFu, em);
        v[k] = decode_v((vc[k / 4] >> (8 * (k % 4))) & 0xFFu, ev);
      }
    } else {
      const uint32_t mb = m_base(em), vb = v_base(ev);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t c = __byte_perm(mc[k / 4], 0u, 0x4440u + k % 4);
        m[k] = __uint_as_float((c * 0x100000u + mb) | ((ms[k / 4] << (24 - 8 * (k % 4))) & 0x80000000u));
        v[k] = __uint_as_float(__byte_perm(vc[k / 4], 0u, 0x4440u + k % 4) * 0x100000u + vb);
      }
    }
  }
  float mx = 0.0f, vx = 0.0f, vn = __uint_as_float(0x7F800000u);
  // A sum is written as a fused a * 1 + b with the 1 from the launch arguments:
  // with add.rn.f32x2 the assembler fuses the products in front into it, and
  // the moments would not be rounded where the definition rounds them.
  const uint64_t one = pack2(a.one, a.one);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t g = mul2(grad_pair(b, k / 2), pack2(p.scale, p.scale));
    const uint64_t m2 = fma2(mul2(pack2(m[k], m[k + 1]), pack2(a.beta1, a.beta1)), one,
                             mul2(g, pack2(a.one_minus_beta1, a.one_minus_beta1)));
    const uint64_t v2 = fma2(mul2(pack2(v[k], v[k + 1]), pack2(a.beta2, a.beta2)), one,
                             mul2(mul2(g, g), pack2(a.one_minus_beta2, a.one_minus_beta2)));
    unpack2(m2, m[k], m[k + 1]);
    unpack2(v2, v[k], v[k + 1]);
    mx = max3_nan(mx, fabsf(m[k]), fabsf(m[k + 1]));
    vx = max3_nan(vx, v[k], v[k + 1]);
    vn = min3(vn, v[k], v[k + 1]);
    float d0, d1;
    unpack2(fma2(pack2(sqrt_approx<false>(v[k]), sqrt_approx<false>(v[k + 1])), pack2(a.inv_sqrt_bc2, a.inv_sqrt_bc2),
                 pack2(a.eps, a.eps)),
            d0, d1);
    const uint64_t w = pack2(b.w.x[k], b.w.x[k + 1]);
    const uint64_t q = mul2(m2, pack2(rcp_approx<false>(d0), rcp_approx<false>(d1)));
    const uint64_t u = fma2(w, pack2(p.decay, p.decay), mul2(q, pack2(p.alpha, p.alpha)));
    unpack2(fma2(u, pack2(-1.0f, -1.0f), w), b.w.x[k], b.w.x[k + 1]);
  }
  if (ALIGNED) {
    st_f8(p.w + i, b.w);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) p.w[i + k] = b.w.x[k];
  }
  const uint32_t me = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mx)) >> 23;
  const uint32_t ve = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vx)) >> 23;
  const uint32_t me2 = min(max(me, 15u), 253u), ve2 = min(max(ve, 31u), 253u);
  key += lane * (8u * kMixB);
  uint32_t om[2], ov[2];
  if (__any_sync(0xFFFFFFFFu, vn == 0.0f) || me >= 254u || ve >= 254u) {
    om[0] = om[1] = ov[0] = ov[1] = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t h = mix32(key + k * kMixB);
      om[k / 4] |= (me == 255u ? 0x7Fu : encode_m(m[k], me2, h >> 16)) << (8 * (k % 4));
      ov[k / 4] |= (ve == 255u ? 0x7Fu : encode_v(v[k], ve2, h & 0xFFFFu)) << (8 * (k % 4));
    }
  } else {
    // With the block's exponent below 254 a code cannot pass its largest (the
    // binade above the maximum), so only the lower ends are clamped: to code 0
    // for m, to code 1 for v. Shifted left by 4 a code is the top byte.
    const uint32_t mlo = m_base(me2), vlo = v_base(ve2);
    uint32_t tm[8], tv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t x = key + k * kMixB;
      x ^= x >> 16;
      x *= kMixA;
      x ^= x >> 15;
      x *= kMixB;
      const uint32_t hi = x >> 16, lo = (x ^ hi) & 0xFFFFu;  // the last step of mix32, by halves
      const uint32_t um = __float_as_uint(m[k]), uv = __float_as_uint(v[k]);
      tm[k] = (max(hi * 16u + (um & 0x7FFFFFFFu), mlo) * 16u - mlo * 16u) | (um & 0x80000000u);
      tv[k] = max(lo * 16u + uv, vlo + 0x100000u) * 16u - vlo * 16u;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      om[q] = __byte_perm(__byte_perm(tm[4 * q], tm[4 * q + 1], 0x0073u),
                          __byte_perm(tm[4 * q + 2], tm[4 * q + 3], 0x0073u), 0x5410u);
      ov[q] = __byte_perm(__byte_perm(tv[4 * q], tv[4 * q + 1], 0x0073u),
                          __byte_perm(tv[4 * q + 2], tv[4 * q + 3], 0x0073u), 0x5410u);
    }
  }
  *reinterpret_cast<uint2*>(p.m + i) = make_uint2(om[0], om[1]);
  *reinterpret_cast<uint2*>(p.v + i) = make_uint2(ov[0], ov[1]);
  em = me == 255u ? 0xFFu : me2;
  ev = ve == 255u ? 0xFFu : ve2;
}

// CTAs per SM: 64 registers a thread. With 5 (48, some spilled) or 3 the step is slower.
constexpr int kAdam8Ctas = 4;

// `count` whole blocks of one warp, from `block` on.
template <bool BF16, bool ALIGNED>
__device__ __forceinline__ void adam8_blocks(const AdamLaunch& a, const Adam8Ptrs& p, uint64_t block,
                                             uint32_t count, uint64_t block_begin) {
  // A block's key and exponents are the same for the whole warp: each lane makes
  // and moves those of one block. The new exponents leave after the last block,
  // since a byte written next to one still to be read holds that read up.
  const uint32_t lane = threadIdx.x & 31u;
  const uint32_t keys = block_key(a.key, block_begin + block + lane);
  uint32_t ems = 0, evs = 0;
  if (lane < count) {
    ems = p.m_exp[block + lane];
    evs = p.v_exp[block + lane];
  }
  auto one = [&](uint32_t k, Block8<BF16>& y) {
    uint32_t em = __shfl_sync(0xFFFFFFFFu, ems, int(k)), ev = __shfl_sync(0xFFFFFFFFu, evs, int(k));
    adam8_block_full<BF16, ALIGNED>(a, p, block + k, __shfl_sync(0xFFFFFFFFu, keys, int(k)), y, em, ev);
    if (lane == k) ems = em, evs = ev;
  };
#pragma unroll 1
  for (uint32_t k = 0; k < count; ++k) {
    Block8<BF16> y;
    load_block8<BF16, ALIGNED>(y, p, block + k);
    one(k, y);
  }
  if (lane < count) {
    p.m_exp[block + lane] = uint8_t(ems);
    p.v_exp[block + lane] = uint8_t(evs);
  }
}

// A tile is one, two or four blocks a warp, by the size of the plan. 1.54 billion
// parameters with BF16 gradients: 3.41 ms, 6.3 TB/s.
// MIXED: some tensor of the plan is not aligned for groups throughout. The kernel
// for aligned plans keeps its registers without the code for the others (3.41 ms
// against 3.48 with both in one). The other way of the general one serves whole
// blocks at any offset of weights and gradients: 60 million parameters with weights, BF16
// gradients or both one element off take 164 to 166 us (503 when each lane's elements were
// 32 apart), 136 on their groups; with FP32 gradients 188 and 143. Its element by element
// accesses are what that costs, and a few registers too many (112 bytes of them reread).
template <bool MIXED>
__global__ void __launch_bounds__(kAdamThreads, kAdam8Ctas) adam8_kernel(const __grid_constant__ AdamLaunch a) {
  stream_ready();
  const AdamTensorDesc* const desc = a.tensors + a.tile_tensor[blockIdx.x];
  const AdamTensorDesc d = *desc;
  Adam8Ptrs p{d.w, d.g, static_cast<uint8_t*>(d.m), static_cast<uint8_t*>(d.v), d.m_exp, d.v_exp,
              a.grad_scale ? *a.grad_scale : 1.0f, a.alpha * d.lr_scale,
              a.lr * d.lr_scale * d.weight_decay};
  if (p.g == nullptr || !isfinite(p.scale)) return;
  const uint64_t n = d.n, block_begin = d.block_begin;
  const uint32_t bf16 = d.grad_bf16, lead = d.lead;
  const uint32_t per_warp = a.tile / kAdamBlock / (kAdamThreads / 32);
  const uint64_t first = (blockIdx.x - d.tile_begin) * (a.tile / kAdamBlock) +
                         (threadIdx.x >> 5) * per_warp;
  // Blocks that take the short way. A graph keeps the kernel that its plan had when it was
  // captured, while the tensors it reads may since have new gradients: the kernel for
  // aligned plans looks at `lead` too, and takes the general way where it is not 0.
  const uint64_t whole = lead == 0u || (MIXED && lead == kAdamCodeGroups) ? n / kAdamBlock : 0u;
  uint32_t done = 0;
  if (first < whole) {
    done = uint32_t(min(whole - first, uint64_t(per_warp)));
    if (!MIXED || lead == 0u)
      bf16 ? adam8_blocks<true, true>(a, p, first, done, block_begin)
           : adam8_blocks<false, true>(a, p, first, done, block_begin);
    else
      bf16 ? adam8_blocks<true, false>(a, p, first, done, block_begin)
           : adam8_blocks<false, false>(a, p, first, done, block_begin);
  }
  for (; done < per_warp && (first + done) * kAdamBlock < n; ++done)
    adam8_block_any(a, desc, p.scale, p.alpha, p.decay, first + done);
}

// 8 values a lane and moment where the buffers are aligned for it: 2 bytes read and 8
// written, bound by memory. 1.54 billion parameters: 2.23 ms, 6.95 TB/s.
__global__ void __launch_bounds__(kAdamThreads)
    adam_export_kernel(const AdamTensorDesc* tensors, const uint32_t* tile_tensor, uint32_t tile) {
  stream_ready();
  const AdamTensorDesc& d = tensors[tile_tensor[blockIdx.x]];
  const uint64_t base = (blockIdx.x - d.tile_begin) * tile, n = d.n;
  const uint32_t len = uint32_t(min(n - base, uint64_t(tile)));
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint8_t* codes = static_cast<const uint8_t*>(q ? d.v : d.m) + base;
    const uint8_t* exps = (q ? d.v_exp : d.m_exp) + base / kAdamBlock;
    float* out = q ? d.v_out : d.m_out;
    if (out == nullptr) continue;
    out += base;
    const bool vec = ((reinterpret_cast<uintptr_t>(codes) & 7u) | (reinterpret_cast<uintptr_t>(out) & 31u)) == 0u;
    const uint32_t groups = vec ? len / 8u : 0u;
#pragma unroll 4
    for (uint32_t j = threadIdx.x; j < groups; j += kAdamThreads) {
      const uint2 c = ld_u2_no_l1(codes + 8u * j);
      const uint32_t e = exps[8u * j / kAdamBlock], w[2] = {c.x, c.y};
      F8 r;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t code = (w[k / 4] >> (8 * (k % 4))) & 0xFFu;
        r.x[k] = q ? decode_v(code, e) : decode_m(code, e);
      }
      st_f8(out + 8u * j, r);
    }
    for (uint32_t j = 8u * groups + threadIdx.x; j < len; j += kAdamThreads) {
      const uint32_t e = exps[j / kAdamBlock];
      out[j] = q ? decode_v(codes[j], e) : decode_m(codes[j], e);
    }
  }
}

// ------------------------------------------------------------ gradient norm

// A sum in two FP32 numbers, hi + lo, about 48 bits. FP64 would do, but runs at
// 1/64 of FP32's rate here: with it the smallest norm took 8.2 us, not 6.2.
struct Sum2 {
  float hi, lo;
};
// The sum of two such sums; the rounding error of hi + hi is recovered exactly.
__device__ __forceinline__ Sum2 add_sum(Sum2 a, Sum2 b) {
  const float s = __fadd_rn(a.hi, b.hi);
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  return {s, __fadd_rn(e, __fadd_rn(a.lo, b.lo))};
}

// The block's sum, in every thread of the first warp.
__device__ __forceinline__ Sum2 block_sum(Sum2 x, Sum2* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = add_sum(x, {__shfl_xor_sync(0xFFFFFFFFu, x.hi, o), __shfl_xor_sync(0xFFFFFFFFu, x.lo, o)});
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = smem[threadIdx.x % (kAdamThreads / 32)];
#pragma unroll
    for (int o = kAdamThreads / 64; o > 0; o >>= 1)
      x = add_sum(x, {__shfl_xor_sync(0xFFFFFFFFu, x.hi, o), __shfl_xor_sync(0xFFFFFFFFu, x.lo, o)});
  }
  return x;
}

// Sum of the squares of elements [lo, hi) of one tensor, this thread's share.
// Plain FP32 over the 8 * kNormUnroll elements that one turn loads.
constexpr int kNormUnroll = 4;
// CTAs per SM, all resident at once. With 4 loads a turn 4, 5 and 6 take 449, 434
// and 437 us for 1.54 billion BF16 gradients; 6 with 2 loads take 465.
constexpr int kNormCtas = 5;
// Elements that a CTA takes at a time.
constexpr uint32_t kNormPiece = 65536;

template <bool BF16>
__device__ __forceinline__ Sum2 sum_squares(const void* g, uint64_t lo, uint64_t hi) {
  constexpr uint32_t kBytes = BF16 ? 2 : 4;
  const char* p = static_cast<const char*>(g);
  auto at = [&](uint64_t i) {
    return BF16 ? __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p + i * 2)) << 16)
                : *reinterpret_cast<const float*>(p + i * 4);
  };
  const uint32_t lead = uint32_t((8u - ((reinterpret_cast<uintptr_t>(p) / kBytes + lo) % 8u)) % 8u);
  const uint64_t first = min(lo + lead, hi);
  const uint64_t groups = (hi - first) / 8u;
  Sum2 sum{0.0f, 0.0f};
  for (uint64_t j = threadIdx.x; j < groups; j += kNormUnroll * kAdamThreads) {
    float x[kNormUnroll][8];
#pragma unroll
    for (int r = 0; r < kNormUnroll; ++r) {
      const uint64_t q = j + r * kAdamThreads;
      if (q < groups) {
        const char* s = p + (first + 8u * q) * kBytes;
        if (BF16) {
          const uint4 u = ld_u4_no_l1(s);
          const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[r][2 * k] = __uint_as_float(v[k] << 16);
            x[r][2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
          }
        } else {
          const F8 u = ld_f8(reinterpret_cast<const float*>(s));
#pragma unroll
          for (int k = 0; k < 8; ++k) x[r][k] = u.x[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[r][k] = 0.0f;
      }
    }
    uint64_t acc[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < kNormUnroll; ++r)
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const uint64_t y = pack2(x[r][k], x[r][k + 1]);
        acc[(k / 2) % 2] = fma2(y, y, acc[(k / 2) % 2]);
      }
    float s[4];
    unpack2(acc[0], s[0], s[1]);
    unpack2(acc[1], s[2], s[3]);
    sum = add_sum(sum, {(s[0] + s[1]) + (s[2] + s[3]), 0.0f});
  }
  // what lies before the first group and after the last
  if (threadIdx.x < first - lo) {
    const float x = at(lo + threadIdx.x);
    sum = add_sum(sum, {x * x, 0.0f});
  }
  if (threadIdx.x < hi - first - 8u * groups) {
    const float x = at(first + 8u * groups + threadIdx.x);
    sum = add_sum(sum, {x * x, 0.0f});
  }
  return sum;
}

// The tiles are cut into equal pieces, as many for one CTA as for another, and the
// CTAs go through the gradients side by side, piece by piece. The CTA that finishes
// last adds the partial sums in CTA order, so the result does not depend on the
// schedule. Each gradient is read once and nothing else: bound by memory. 1.54
// billion BF16 gradients: 434 us, 7.1 TB/s (477 us with one long piece a CTA, whose
// distant streams the memory serves less well, 458 us with pieces of 131,072); the
// smallest calls are four trips to memory one after the other: 8 us for 1 million
// elements, the host's part included.
__global__ void __launch_bounds__(kAdamThreads, kNormCtas)
    grad_norm_kernel(const AdamTensorDesc* tensors, const uint32_t* tile_tensor, uint32_t tile,
                     uint64_t total_tiles, uint64_t pieces, Sum2* partials, uint32_t* ticket, float max_norm,
                     float* norm_out, float* clip_out) {
  __shared__ Sum2 smem[kAdamThreads / 32];
  __shared__ bool last;
  stream_ready();
  Sum2 sum{0.0f, 0.0f};
  for (uint64_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const uint64_t hi = total_tiles * (piece + 1) / pieces;
    for (uint64_t t = total_tiles * piece / pieces; t < hi;) {
      const AdamTensorDesc& d = tensors[tile_tensor[t]];
      const uint64_t begin = d.tile_begin, n = d.n;
      const uint64_t e0 = (t - begin) * tile, e1 = min((hi - begin) * tile, n);
      if (d.g != nullptr)
        sum = add_sum(sum, d.grad_bf16 ? sum_squares<true>(d.g, e0, e1) : sum_squares<false>(d.g, e0, e1));
      t = begin + (n + tile - 1) / tile;
    }
  }
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = sum;
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
    last = before == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  sum = {0.0f, 0.0f};
  for (uint32_t k = threadIdx.x; k < gridDim.x; k += kAdamThreads) {
    const float2 q = __ldcg(reinterpret_cast<const float2*>(partials) + k);
    sum = add_sum(sum, {q.x, q.y});
  }
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) {
    // past FP32's range hi is infinite and lo a NaN
    const float norm = __fsqrt_rn(isfinite(sum.hi) ? sum.hi + sum.lo : sum.hi);
    *norm_out = norm;
    if (clip_out)
      *clip_out = isfinite(norm) ? fminf(1.0f, max_norm / (norm + 1e-6f)) : __uint_as_float(0x7FC00000u);
    *ticket = 0u;
  }
}

}  // namespace

uint32_t adam_key(uint64_t seed, uint64_t step) {
  uint32_t x = 0;
  const uint32_t words[4] = {uint32_t(seed), uint32_t(seed >> 32), uint32_t(step), uint32_t(step >> 32)};
  for (uint32_t w : words) x = mix32(x + w + kMixB);
  return x;
}

cudaError_t launch_adam32(const AdamLaunch& a, cudaStream_t stream) {
  return launch_early(adam32_kernel, dim3(unsigned(a.total_tiles)), kAdamThreads, stream, a);
}

cudaError_t launch_adam8(const AdamLaunch& a, cudaStream_t stream) {
  return launch_early(a.mixed ? adam8_kernel<true> : adam8_kernel<false>, dim3(unsigned(a.total_tiles)), kAdamThreads,
                      stream, a);
}

cudaError_t launch_adam_export(const AdamTensorDesc* tensors, const uint32_t* tile_tensor,
                               uint32_t tile, uint64_t total_tiles, cudaStream_t stream) {
  return launch_early(adam_export_kernel, dim3(unsigned(total_tiles)), kAdamThreads, stream, tensors, tile_tensor, tile);
}

cudaError_t launch_grad_norm(const AdamTensorDesc* tensors, const uint32_t* tile_tensor,
                             uint32_t tile, uint64_t total_tiles, int sms, uint64_t* partials, uint32_t* ticket,
                             float max_norm, float* norm_out, float* clip_out, cudaStream_t stream) {
  uint64_t grid = uint64_t(sms) * kNormCtas;
  if (grid > uint64_t(kNormMaxCtas)) grid = kNormMaxCtas;
  if (grid > total_tiles) grid = total_tiles ? total_tiles : 1;
  const uint64_t turn = grid * (kNormPiece / tile);
  const uint64_t pieces = grid * ((total_tiles + turn - 1) / turn);
  return launch_early(grad_norm_kernel, dim3(unsigned(grid)), kAdamThreads, stream, tensors, tile_tensor, tile,
                      total_tiles, pieces, reinterpret_cast<Sum2*>(partials), ticket, max_norm, norm_out, clip_out);
}

}  // namespace pulse
