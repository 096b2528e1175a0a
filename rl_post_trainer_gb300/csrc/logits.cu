// logits.cu -- logit shaping (repetition, presence and frequency penalties,
// biases, temperature, grammar masks) and its gradient, with the formulas of
// include/pulse.h. One CTA per slice of a row's vocabulary: it reads the row's
// history, keeps what concerns its slice in shared memory, and then makes one
// pass over the slice.
#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

constexpr int kLogitsThreads = 256;
constexpr uint32_t kLogitsSlice = 4096;

__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const uint16_t* p) {
  return __uint_as_float(uint32_t(*p) << 16);
}
__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_elem(uint16_t* p, float x) {
  *p = uint16_t(bf16_rne_bits(__float_as_uint(x)));
}

// A temperature that is not above 0 (greedy decoding) leaves the row as it is.
__device__ __forceinline__ float inverse_temperature(const float* t, uint64_t row) {
  if (t == nullptr) return 1.0f;
  const float x = t[row];
  return x > 0.0f ? __fdiv_rn(1.0f, x) : 1.0f;
}

struct Range {
  int64_t begin, split, end;
};

// The row's history, empty (and recorded) where its offsets do not fit.
__device__ __forceinline__ Range history_of(const LogitsArgs& a, uint64_t row) {
  Range r{0, 0, 0};
  if (a.tokens == nullptr) return r;
  const int64_t b = a.begin[row], e = a.end[row];
  const int64_t s = a.split ? a.split[row] : b;
  if (b < 0 || e < b || e > a.ntokens || s < b || s > e) {
    if (threadIdx.x == 0) record_error(a.error_word, kErrIndex);
    return r;
  }
  r.begin = b;
  r.split = s;
  r.end = e;
  return r;
}

__device__ __forceinline__ Range bias_of(const LogitsArgs& a, uint64_t row) {
  Range r{0, 0, 0};
  if (a.bias_tokens == nullptr) return r;
  const int64_t b = a.bias_begin[row], e = a.bias_begin[row + 1];
  if (b < 0 || e < b || e > a.nbias) {
    if (threadIdx.x == 0) record_error(a.error_word, kErrIndex);
    return r;
  }
  r.begin = r.split = b;
  r.end = e;
  return r;
}

// The row's mask words, or null.
__device__ __forceinline__ const uint32_t* mask_of(const LogitsArgs& a, uint64_t row) {
  if (a.mask == nullptr) return nullptr;
  const int64_t m = a.mask_row ? int64_t(a.mask_row[row]) : int64_t(row);
  if (m < 0) return nullptr;
  if (m >= a.mask_rows) {
    if (threadIdx.x == 0) record_error(a.error_word, kErrIndex);
    return nullptr;
  }
  return a.mask + uint64_t(m) * a.mask_stride;
}

__device__ __forceinline__ bool bit_of(const uint32_t* words, uint32_t i) {
  return (words[i >> 5] >> (i & 31u)) & 1u;
}
__device__ __forceinline__ void set_bit(uint32_t* words, uint32_t i) {
  atomicOr(words + (i >> 5), 1u << (i & 31u));
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kLogitsThreads) shape_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t seen[kLogitsSlice / 32];    // in the history
  __shared__ uint32_t made[kLogitsSlice / 32];    // generated
  __shared__ uint32_t biased[kLogitsSlice / 32];  // in the bias list
  __shared__ uint32_t count[kLogitsSlice];        // times generated, of the made ones
  __shared__ int32_t entry[kLogitsSlice];         // last entry in the bias list, of the biased ones
  const uint64_t row = blockIdx.x / a.slices;
  const uint32_t lo = uint32_t(blockIdx.x % a.slices) * a.slice;
  const uint32_t len = min(a.slice, a.vocab - lo);
  const Range h = history_of(a, row);
  const Range bl = bias_of(a, row);
  const uint32_t* mask = mask_of(a, row);
  for (uint32_t i = threadIdx.x; i < kLogitsSlice / 32; i += kLogitsThreads)
    seen[i] = made[i] = biased[i] = 0u;
  __syncthreads();
  for (int64_t i = h.begin + threadIdx.x; i < h.end; i += kLogitsThreads) {
    const uint32_t t = uint32_t(a.tokens[i]), u = t - lo;
    if (t >= a.vocab) record_error(a.error_word, kErrIndex);
    if (t < a.vocab && u < len) {
      set_bit(seen, u);
      if (i >= h.split) {
        set_bit(made, u);
        count[u] = 0u;
      }
    }
  }
  for (int64_t i = bl.begin + threadIdx.x; i < bl.end; i += kLogitsThreads) {
    const uint32_t t = uint32_t(a.bias_tokens[i]), u = t - lo;
    if (t >= a.vocab) record_error(a.error_word, kErrIndex);
    if (t < a.vocab && u < len) {
      set_bit(biased, u);
      entry[u] = -1;
    }
  }
  __syncthreads();
  for (int64_t i = h.split + threadIdx.x; i < h.end; i += kLogitsThreads) {
    const uint32_t t = uint32_t(a.tokens[i]), u = t - lo;
    if (t < a.vocab && u < len) atomicAdd(count + u, 1u);
  }
  for (int64_t i = bl.begin + threadIdx.x; i < bl.end; i += kLogitsThreads) {
    const uint32_t t = uint32_t(a.bias_tokens[i]), u = t - lo;
    if (t < a.vocab && u < len) atomicMax(entry + u, int32_t(i));
  }
  __syncthreads();
  const float inv_t = inverse_temperature(a.temperature, row);
  const float rep = a.repetition ? a.repetition[row] : 1.0f;
  const float pres = a.presence ? a.presence[row] : 0.0f;
  const float freq = a.frequency ? a.frequency[row] : 0.0f;
  const TIn* src = static_cast<const TIn*>(a.src) + row * a.src_stride + lo;
  TOut* dst = static_cast<TOut*>(a.dst) + row * a.dst_stride + lo;
  for (uint32_t u = threadIdx.x; u < len; u += kLogitsThreads) {
    float x = load_elem(src + u);
    if (a.repetition && bit_of(seen, u)) x = x > 0.0f ? __fdiv_rn(x, rep) : x * rep;
    if (bit_of(made, u)) {
      if (a.frequency) x = __fsub_rn(x, __fmul_rn(freq, float(count[u])));
      if (a.presence) x = __fsub_rn(x, pres);
    }
    if (bit_of(biased, u)) x = __fadd_rn(x, a.bias_values[entry[u]]);
    x = __fmul_rn(x, inv_t);
    if (mask && !bit_of(mask, lo + u)) x = __uint_as_float(0xFF800000u);
    store_elem(dst + u, x);
  }
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kLogitsThreads)
    backward_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t seen[kLogitsSlice / 32];
  const uint64_t row = blockIdx.x / a.slices;
  const uint32_t lo = uint32_t(blockIdx.x % a.slices) * a.slice;
  const uint32_t len = min(a.slice, a.vocab - lo);
  const Range h = a.repetition ? history_of(a, row) : Range{0, 0, 0};
  const uint32_t* mask = mask_of(a, row);
  for (uint32_t i = threadIdx.x; i < kLogitsSlice / 32; i += kLogitsThreads) seen[i] = 0u;
  __syncthreads();
  for (int64_t i = h.begin + threadIdx.x; i < h.end; i += kLogitsThreads) {
    const uint32_t t = uint32_t(a.tokens[i]), u = t - lo;
    if (t >= a.vocab) record_error(a.error_word, kErrIndex);
    if (t < a.vocab && u < len) set_bit(seen, u);
  }
  __syncthreads();
  const float inv_t = inverse_temperature(a.temperature, row);
  const float rep = a.repetition ? a.repetition[row] : 1.0f;
  const TOut* src = static_cast<const TOut*>(a.src) + row * a.src_stride + lo;
  const TIn* raw = static_cast<const TIn*>(a.raw) + (a.raw ? row * a.raw_stride + lo : 0u);
  TIn* dst = static_cast<TIn*>(a.dst) + row * a.dst_stride + lo;
  for (uint32_t u = threadIdx.x; u < len; u += kLogitsThreads) {
    float x = __fmul_rn(load_elem(src + u), inv_t);
    if (bit_of(seen, u)) x = load_elem(raw + u) > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    if (mask && !bit_of(mask, lo + u)) x = 0.0f;
    store_elem(dst + u, x);
  }
}

}  // namespace

cudaError_t launch_logits_shape(LogitsArgs a, int in_type, int out_type, int, cudaStream_t stream) {
  a.slice = kLogitsSlice;
  a.slices = (a.vocab + a.slice - 1) / a.slice;
  const unsigned grid = unsigned(a.rows * a.slices);
  if (in_type == PULSE_F32)
    shape_kernel<float, float><<<grid, kLogitsThreads, 0, stream>>>(a);
  else if (out_type == PULSE_F32)
    shape_kernel<uint16_t, float><<<grid, kLogitsThreads, 0, stream>>>(a);
  else
    shape_kernel<uint16_t, uint16_t><<<grid, kLogitsThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_logits_backward(LogitsArgs a, int in_type, int out_type, int,
                                   cudaStream_t stream) {
  a.slice = kLogitsSlice;
  a.slices = (a.vocab + a.slice - 1) / a.slice;
  const unsigned grid = unsigned(a.rows * a.slices);
  if (in_type == PULSE_F32)
    backward_kernel<float, float><<<grid, kLogitsThreads, 0, stream>>>(a);
  else if (out_type == PULSE_F32)
    backward_kernel<uint16_t, float><<<grid, kLogitsThreads, 0, stream>>>(a);
  else
    backward_kernel<uint16_t, uint16_t><<<grid, kLogitsThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pulse
