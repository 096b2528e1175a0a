// logits.cu -- logit shaping (repetition, presence and frequency penalties,
// biases, temperature, grammar masks) and its gradient, with the formulas of
// include/pulse.h.
//
// One CTA takes a slice of a row's vocabulary. It reads the row's history and
// bias list once, keeps in shared memory what falls into its slice (a bit per
// token, the count of generated ones, the last bias entry), computes the few
// touched values with full warps, and then streams over the slice: scale, mask,
// and where a token's bit is set the value from shared memory.
#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

#ifndef PULSE_LOGITS_THREADS
#define PULSE_LOGITS_THREADS 256
#endif
#ifndef PULSE_LOGITS_SLICE
#define PULSE_LOGITS_SLICE 8192
#endif
#ifndef PULSE_LOGITS_SLICE_BACK
#define PULSE_LOGITS_SLICE_BACK 8192
#endif
#ifndef PULSE_LOGITS_BATCH
#define PULSE_LOGITS_BATCH 2
#endif
constexpr int kThreads = PULSE_LOGITS_THREADS;
constexpr uint32_t kSliceMin = 2048;
constexpr int kBatch = PULSE_LOGITS_BATCH;  // groups of 8 elements a thread has in flight

// A group is 8 elements of a row, 16 bytes of BF16 or 32 of FP32.
__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const uint16_t* p) {
  return __uint_as_float(uint32_t(*p) << 16);
}
__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_elem(uint16_t* p, float x) {
  *p = uint16_t(cvt_bf16x2_rn(x, 0.0f));
}
__device__ __forceinline__ void load_group(const float* p, float (&x)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}
__device__ __forceinline__ void load_group(const uint16_t* p, float (&x)[8]) {
  uint32_t u[4];
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
               : "l"(p));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(u[k] << 16);
    x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store_group(float* p, const float (&x)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]),
               "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
__device__ __forceinline__ void store_group(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(cvt_bf16x2_rn(x[0], x[1]), cvt_bf16x2_rn(x[2], x[3]),
                                            cvt_bf16x2_rn(x[4], x[5]), cvt_bf16x2_rn(x[6], x[7]));
}
// Elements from p to the next group boundary.
template <typename T>
__device__ __forceinline__ uint32_t lead_of(const T* p) {
  return uint32_t(0u - uint32_t(reinterpret_cast<uintptr_t>(p) / sizeof(T))) & 7u;
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

// The 8 mask bits from token t on; a group that ends inside the vocabulary.
__device__ __forceinline__ uint32_t mask_bits8(const uint32_t* mask, uint32_t t) {
  const uint32_t w = t >> 5, s = t & 31u;
  const uint32_t lo = mask[w], hi = s > 24u ? mask[w + 1] : 0u;
  return __funnelshift_r(lo, hi, s) & 0xFFu;
}

// This CTA's part of a row: tokens [first, stop), groups from `base` on. Token t
// has place t - base + 8 in the shared tables, so that a group's bits are a byte
// of the bitmap and the tokens before the first group (row start) have places
// below 8.
struct Slice {
  uint64_t row;
  uint32_t first, base, stop;
  bool grouped;  // source and destination rows share their group boundaries
};

template <typename TSrc, typename TDst>
__device__ __forceinline__ Slice slice_of(const LogitsArgs& a, const TSrc*& src, TDst*& dst) {
  Slice s;
  s.row = blockIdx.x / a.slices;
  const uint32_t k = uint32_t(blockIdx.x % a.slices);
  src += s.row * a.src_stride;
  dst += s.row * a.dst_stride;
  const uint32_t lead = lead_of(src);
  s.grouped = lead == lead_of(dst);
  s.base = (s.grouped ? lead : 0u) + k * a.slice;
  s.first = k == 0 ? 0u : min(s.base, a.vocab);
  s.stop = k + 1 == a.slices ? a.vocab : min(s.base + a.slice, a.vocab);
  return s;
}

// Calls f(token, position) for the entries [begin, end) of a list of tokens,
// spread over the CTA, four at a time where the list is aligned for it.
template <typename F>
__device__ __forceinline__ void scan_tokens(const int32_t* tokens, int64_t begin, int64_t end, F f) {
  const int64_t n = end - begin;
  const int32_t* p = tokens + begin;
  const int64_t lead = min(n, int64_t((0u - uint32_t(reinterpret_cast<uintptr_t>(p) / 4u)) & 3u));
  const int64_t quads = (n - lead) / 4;
#pragma unroll 2
  for (int64_t q = threadIdx.x; q < quads; q += kThreads) {
    const int4 t = __ldg(reinterpret_cast<const int4*>(p + lead) + q);
    const int64_t i = begin + lead + 4 * q;
    f(uint32_t(t.x), i);
    f(uint32_t(t.y), i + 1);
    f(uint32_t(t.z), i + 2);
    f(uint32_t(t.w), i + 3);
  }
  if (threadIdx.x < lead) f(uint32_t(p[threadIdx.x]), begin + threadIdx.x);
  const int64_t rest = lead + 4 * quads + threadIdx.x;
  if (rest < n) f(uint32_t(p[rest]), begin + rest);
}

// Shared tables of a slice of S tokens (S + 8 places, rounded up).
__host__ __device__ constexpr uint32_t places(uint32_t slice) { return (slice + 8u + 31u) & ~31u; }

// Marks place u and appends it to the list of touched places if it is new.
__device__ __forceinline__ void touch(uint32_t* bits, uint16_t* list, uint32_t* count, uint32_t u) {
  const uint32_t bit = 1u << (u & 31u);
  if (!(atomicOr(bits + (u >> 5), bit) & bit)) list[atomicAdd(count, 1u)] = uint16_t(u);
}

// Streams a slice: x -> override(x, place) where the place's bit is set, else
// plain(x); masked tokens become `masked` without being read.
template <typename TSrc, typename TDst, typename Plain, typename Override>
__device__ __forceinline__ void stream_slice(const Slice& s, const TSrc* src, TDst* dst,
                                             const uint32_t* mask, const uint32_t* bits,
                                             float masked, Plain plain, Override over) {
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(bits);
  auto one = [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = masked;
    if (mask == nullptr || (mask[t >> 5] >> (t & 31u)) & 1u) {
      const float x = load_elem(src + t);
      y = bits && (bits[u >> 5] >> (u & 31u)) & 1u ? over(x, u) : plain(x);
    }
    store_elem(dst + t, y);
  };
  if (!s.grouped) {
    for (uint32_t t = s.first + threadIdx.x; t < s.stop; t += kThreads) one(t);
    return;
  }
  const uint32_t groups = s.stop > s.base ? (s.stop - s.base) / 8u : 0u;
  for (uint32_t g = threadIdx.x; g < groups; g += kBatch * kThreads) {
    float x[kBatch][8];
    uint32_t ok[kBatch];
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      const uint32_t q = g + r * kThreads;
      ok[r] = q >= groups ? 0u : mask ? mask_bits8(mask, s.base + 8u * q) : 0xFFu;
    }
#pragma unroll
    for (int r = 0; r < kBatch; ++r)
      if (ok[r]) load_group(src + s.base + 8u * (g + r * kThreads), x[r]);
#pragma unroll
    for (int r = 0; r < kBatch; ++r) {
      const uint32_t q = g + r * kThreads;
      if (q >= groups) break;
      const uint32_t hit = bits ? bytes[q + 1u] & ok[r] : 0u;
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = plain(x[r][k]);
      if (hit) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((hit >> k) & 1u) y[k] = over(x[r][k], 8u * q + 8u + k);
      }
      if (ok[r] != 0xFFu) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!((ok[r] >> k) & 1u)) y[k] = masked;
      }
      store_group(dst + s.base + 8u * q, y);
    }
  }
  // the row's first tokens and its last, outside the groups
  const uint32_t head = s.first < s.base ? min(s.base, s.stop) - s.first : 0u;
  if (threadIdx.x < head) one(s.first + threadIdx.x);
  const uint32_t tail = s.base + 8u * groups + threadIdx.x;
  if (s.stop > s.base && tail < s.stop) one(tail);
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads) shape_kernel(const __grid_constant__ LogitsArgs a) {
  extern __shared__ uint4 smem[];
  __shared__ uint32_t touched;
  const uint32_t n = places(a.slice);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);         // a bit per place
  uint32_t* state = bits + n / 32u;                           // history, then the value as float bits
  uint16_t* list = reinterpret_cast<uint16_t*>(state + n);    // touched places
  uint32_t* entry = reinterpret_cast<uint32_t*>(list + n);    // 1 + place in the bias list (bias only)
  const TIn* src = static_cast<const TIn*>(a.src);
  TOut* dst = static_cast<TOut*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const Range h = a.repetition || a.presence || a.frequency ? history_of(a, s.row) : Range{0, 0, 0};
  const Range bl = bias_of(a, s.row);
  const uint32_t* mask = mask_of(a, s.row);
  const float inv_t = inverse_temperature(a.temperature, s.row);
  const bool any = h.end > h.begin || bl.end > bl.begin;
  if (any) {
    const bool bias = bl.end > bl.begin;
    if (threadIdx.x == 0) touched = 0u;
    for (uint32_t i = threadIdx.x; i < n / 32u; i += kThreads) bits[i] = 0u;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) state[i] = 0u;
    if (bias)
      for (uint32_t i = threadIdx.x; i < n; i += kThreads) entry[i] = 0u;
    __syncthreads();
    const uint32_t len = s.stop - s.first, off = s.first - s.base + 8u;
    // state: bit 31 for a token of the prompt, below it the times generated
    scan_tokens(a.tokens, h.begin, h.end, [&](uint32_t t, int64_t i) {
      if (t - s.first < len) {
        const uint32_t u = t - s.first + off;
        if (i >= h.split)
          atomicAdd(state + u, 1u);
        else
          atomicOr(state + u, 0x80000000u);
        touch(bits, list, &touched, u);
      } else if (t >= a.vocab) {
        record_error(a.error_word, kErrIndex);
      }
    });
    if (bias)
      scan_tokens(a.bias_tokens, bl.begin, bl.end, [&](uint32_t t, int64_t i) {
        if (t - s.first < len) {
          const uint32_t u = t - s.first + off;
          atomicMax(entry + u, uint32_t(i - bl.begin) + 1u);
          touch(bits, list, &touched, u);
        } else if (t >= a.vocab) {
          record_error(a.error_word, kErrIndex);
        }
      });
    __syncthreads();
    const float rep = a.repetition ? a.repetition[s.row] : 1.0f;
    const float pres = a.presence ? a.presence[s.row] : 0.0f;
    const float freq = a.frequency ? a.frequency[s.row] : 0.0f;
    for (uint32_t i = threadIdx.x; i < touched; i += kThreads) {
      const uint32_t u = list[i], st = state[u], count = st & 0x7FFFFFFFu;
      float x = load_elem(src + (s.base + u - 8u));
      if (a.repetition && st != 0u) x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
      if (count != 0u) {
        if (a.frequency) x = __fsub_rn(x, __fmul_rn(freq, float(count)));
        if (a.presence) x = __fsub_rn(x, pres);
      }
      if (bias && entry[u] != 0u) x = __fadd_rn(x, a.bias_values[bl.begin + entry[u] - 1u]);
      state[u] = __float_as_uint(__fmul_rn(x, inv_t));
    }
    __syncthreads();
  }
  stream_slice(
      s, src, dst, mask, any ? bits : nullptr, __uint_as_float(0xFF800000u),
      [&](float x) { return __fmul_rn(x, inv_t); },
      [&](float, uint32_t u) { return __uint_as_float(state[u]); });
}

template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ LogitsArgs a) {
  extern __shared__ uint4 smem[];
  __shared__ uint32_t touched;
  const uint32_t n = places(a.slice);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);         // a bit per place of the history
  uint32_t* above = bits + n / 32u;                           // its raw logit is above 0
  uint16_t* list = reinterpret_cast<uint16_t*>(above + n / 32u);
  const TOut* src = static_cast<const TOut*>(a.src);
  TIn* dst = static_cast<TIn*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const Range h = a.repetition ? history_of(a, s.row) : Range{0, 0, 0};
  const uint32_t* mask = mask_of(a, s.row);
  const float inv_t = inverse_temperature(a.temperature, s.row);
  const bool any = h.end > h.begin;
  float rep = 1.0f;
  if (any) {
    rep = a.repetition[s.row];
    if (threadIdx.x == 0) touched = 0u;
    for (uint32_t i = threadIdx.x; i < n / 32u; i += kThreads) bits[i] = above[i] = 0u;
    __syncthreads();
    const uint32_t len = s.stop - s.first, off = s.first - s.base + 8u;
    scan_tokens(a.tokens, h.begin, h.end, [&](uint32_t t, int64_t) {
      if (t - s.first < len)
        touch(bits, list, &touched, t - s.first + off);
      else if (t >= a.vocab)
        record_error(a.error_word, kErrIndex);
    });
    __syncthreads();
    const TIn* raw = static_cast<const TIn*>(a.raw) + s.row * a.raw_stride;
    for (uint32_t i = threadIdx.x; i < touched; i += kThreads) {
      const uint32_t u = list[i];
      if (load_elem(raw + (s.base + u - 8u)) > 0.0f) atomicOr(above + (u >> 5), 1u << (u & 31u));
    }
    __syncthreads();
  }
  stream_slice(
      s, src, dst, mask, any ? bits : nullptr, 0.0f, [&](float x) { return __fmul_rn(x, inv_t); },
      [&](float x, uint32_t u) {
        const float d = __fmul_rn(x, inv_t);
        return (above[u >> 5] >> (u & 31u)) & 1u ? __fdiv_rn(d, rep) : __fmul_rn(d, rep);
      });
}

// Slices of a row: the largest that still gives every SM several CTAs, since a
// slice costs one more reading of the history.
void cut_rows(LogitsArgs& a, uint32_t most, int sms) {
  uint32_t slice = most;
  while (slice > kSliceMin && a.rows * ((a.vocab + slice - 1) / slice) < uint64_t(sms) * 4) slice /= 2;
  a.slices = (a.vocab + slice - 1) / slice;
  a.slice = slice;
}

template <typename K>
cudaError_t launch(K kernel, const LogitsArgs& a, uint32_t smem, cudaStream_t stream) {
  if (smem > 48u * 1024u) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
  }
  kernel<<<unsigned(a.rows * a.slices), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits_shape(LogitsArgs a, int in_type, int out_type, int sms, cudaStream_t stream) {
  cut_rows(a, PULSE_LOGITS_SLICE, sms);
  const bool history = a.tokens && (a.repetition || a.presence || a.frequency);
  const uint32_t n = places(a.slice);
  uint32_t smem = 0;
  if (history || a.bias_tokens) smem = n / 8u + n * 6u + (a.bias_tokens ? n * 4u : 0u);
  if (in_type == PULSE_F32) return launch(shape_kernel<float, float>, a, smem, stream);
  if (out_type == PULSE_F32) return launch(shape_kernel<uint16_t, float>, a, smem, stream);
  return launch(shape_kernel<uint16_t, uint16_t>, a, smem, stream);
}

cudaError_t launch_logits_backward(LogitsArgs a, int in_type, int out_type, int sms,
                                   cudaStream_t stream) {
  cut_rows(a, PULSE_LOGITS_SLICE_BACK, sms);
  const uint32_t n = places(a.slice);
  const uint32_t smem = a.tokens && a.repetition ? n / 4u + n * 2u : 0u;
  if (in_type == PULSE_F32) return launch(backward_kernel<float, float>, a, smem, stream);
  if (out_type == PULSE_F32) return launch(backward_kernel<uint16_t, float>, a, smem, stream);
  return launch(backward_kernel<uint16_t, uint16_t>, a, smem, stream);
}

}  // namespace pulse
