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

// Moments and weight of one element. Products and sums of the moments are
// rounded one by one (no fused multiply-add), so that 8-bit codes made from
// them are the same wherever they are computed.
__device__ __forceinline__ void adam_element(const AdamLaunch& a, float alpha, float decay, float g,
                                             float& m, float& v, float& w) {
  m = __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_minus_beta1));
  v = __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
  const float den = __fsqrt_rn(v) * a.inv_sqrt_bc2 + a.eps;
  w = w - (alpha * __fdiv_rn(m, den) + decay * w);
}

__global__ void __launch_bounds__(kAdamThreads) adam32_kernel(const __grid_constant__ AdamLaunch a) {
  const AdamTensorDesc d = a.tensors[a.tile_tensor[blockIdx.x]];
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  if (d.g == nullptr || !isfinite(scale)) return;
  const float alpha = a.alpha * d.lr_scale, decay = a.lr * d.lr_scale * d.weight_decay;
  const uint64_t base = (blockIdx.x - d.tile_begin) * kAdamTile;
  float* pm = static_cast<float*>(d.m);
  float* pv = static_cast<float*>(d.v);
  for (int j = threadIdx.x; j < kAdamTile; j += kAdamThreads) {
    const uint64_t i = base + j;
    if (i >= d.n) break;
    float m = pm[i], v = pv[i], w = d.w[i];
    adam_element(a, alpha, decay, load_grad(d, i) * scale, m, v, w);
    pm[i] = m;
    pv[i] = v;
    d.w[i] = w;
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

__global__ void __launch_bounds__(kAdamThreads) adam8_kernel(const __grid_constant__ AdamLaunch a) {
  const AdamTensorDesc d = a.tensors[a.tile_tensor[blockIdx.x]];
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  if (d.g == nullptr || !isfinite(scale)) return;
  const float alpha = a.alpha * d.lr_scale, decay = a.lr * d.lr_scale * d.weight_decay;
  const uint64_t tile = blockIdx.x - d.tile_begin;
  uint8_t* pm = static_cast<uint8_t*>(d.m);
  uint8_t* pv = static_cast<uint8_t*>(d.v);
  const uint32_t lane = threadIdx.x & 31u;
  for (uint32_t b = threadIdx.x >> 5; b < kAdamTile / kAdamBlock; b += kAdamThreads / 32) {
    const uint64_t block = tile * (kAdamTile / kAdamBlock) + b;
    const uint64_t base = block * kAdamBlock;
    if (base >= d.n) break;
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
        adam_element(a, alpha, decay, load_grad(d, i) * scale, m[k], v[k], w);
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
}

__global__ void __launch_bounds__(kAdamThreads)
    adam_export_kernel(const AdamTensorDesc* tensors, const uint32_t* tile_tensor) {
  const AdamTensorDesc& d = tensors[tile_tensor[blockIdx.x]];
  const uint64_t base = (blockIdx.x - d.tile_begin) * kAdamTile;
  const uint8_t* pm = static_cast<const uint8_t*>(d.m);
  const uint8_t* pv = static_cast<const uint8_t*>(d.v);
  for (int j = threadIdx.x; j < kAdamTile; j += kAdamThreads) {
    const uint64_t i = base + j;
    if (i >= d.n) break;
    if (d.m_out) d.m_out[i] = decode_m(pm[i], d.m_exp[i / kAdamBlock]);
    if (d.v_out) d.v_out[i] = decode_v(pv[i], d.v_exp[i / kAdamBlock]);
  }
}

// ------------------------------------------------------------ gradient norm

__device__ __forceinline__ double block_sum(double x, double* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int k = 0; k < kAdamThreads / 32; ++k) x += smem[k];
  __syncthreads();
  return x;
}

// Each CTA sums a fixed range of tiles; the CTA that finishes last adds the
// partial sums in CTA order, so the result does not depend on the schedule.
__global__ void __launch_bounds__(kAdamThreads)
    grad_norm_kernel(const AdamTensorDesc* tensors, const uint32_t* tile_tensor,
                     uint64_t total_tiles, double* partials, uint32_t* ticket, float max_norm,
                     float* norm_out, float* clip_out) {
  __shared__ double smem[kAdamThreads / 32];
  __shared__ bool last;
  const uint64_t lo = total_tiles * blockIdx.x / gridDim.x;
  const uint64_t hi = total_tiles * (blockIdx.x + 1) / gridDim.x;
  double sum = 0.0;
  for (uint64_t t = lo; t < hi; ++t) {
    const AdamTensorDesc& d = tensors[tile_tensor[t]];
    if (d.g == nullptr) continue;
    const uint64_t base = (t - d.tile_begin) * kAdamTile;
    float s = 0.0f;
    for (int j = threadIdx.x; j < kAdamTile; j += kAdamThreads) {
      const uint64_t i = base + j;
      if (i >= d.n) break;
      const float g = load_grad(d, i);
      s = fmaf(g, g, s);
    }
    sum += double(s);
  }
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = sum;
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  sum = 0.0;
  for (uint32_t k = threadIdx.x; k < gridDim.x; k += kAdamThreads) sum += __ldcg(partials + k);
  sum = block_sum(sum, smem);
  if (threadIdx.x == 0) {
    const float norm = float(sqrt(sum));
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
  adam32_kernel<<<unsigned(a.total_tiles), kAdamThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_adam8(const AdamLaunch& a, cudaStream_t stream) {
  adam8_kernel<<<unsigned(a.total_tiles), kAdamThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_adam_export(const AdamTensorDesc* tensors, const uint32_t* tile_tensor,
                               uint64_t total_tiles, cudaStream_t stream) {
  adam_export_kernel<<<unsigned(total_tiles), kAdamThreads, 0, stream>>>(tensors, tile_tensor);
  return cudaGetLastError();
}

cudaError_t launch_grad_norm(const AdamTensorDesc* tensors, const uint32_t* tile_tensor,
                             uint64_t total_tiles, int sms, double* partials, uint32_t* ticket,
                             float max_norm, float* norm_out, float* clip_out, cudaStream_t stream) {
  uint64_t grid = uint64_t(sms) * 8;
  if (grid > uint64_t(kNormMaxCtas)) grid = kNormMaxCtas;
  if (grid > total_tiles) grid = total_tiles ? total_tiles : 1;
  grad_norm_kernel<<<unsigned(grid), kAdamThreads, 0, stream>>>(
      tensors, tile_tensor, total_tiles, partials, ticket, max_norm, norm_out, clip_out);
  return cudaGetLastError();
}

}  // namespace pulse
