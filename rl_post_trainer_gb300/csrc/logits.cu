// logits.cu -- logit shaping (repetition, presence and frequency penalties,
// biases, temperature, grammar masks) and its gradient, with the formulas of
// include/pulse.h.
//
// A row is cut into slices, one CTA each. A CTA asks for its slice, reads the
// row's history and bias list meanwhile, keeps a bit for every token of its slice
// that they name (and, where tokens are counted or biased, a word), and then works
// off the slice from registers.
#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

#ifndef PULSE_LOGITS_MIN
#define PULSE_LOGITS_MIN 4
#endif
#ifndef PULSE_LOGITS_GROUPS
#define PULSE_LOGITS_GROUPS 4
#endif
#ifndef PULSE_LOGITS_THREADS
#define PULSE_LOGITS_THREADS 256
#endif
constexpr int kThreads = PULSE_LOGITS_THREADS;
constexpr int kMinCtas = PULSE_LOGITS_MIN;
// Groups of 8 elements a thread holds: its whole part of a slice, asked for
// before the history is read.
constexpr int kGroups = PULSE_LOGITS_GROUPS;
constexpr uint32_t kSliceMin = 2048;
constexpr uint32_t kSliceMax = 8u * kThreads * kGroups - 32u;
constexpr uint32_t kWords = (kSliceMax + 8u + 31u) / 32u;  // of a bitmap of a slice's places
constexpr uint32_t kPlaces = kWords * 32u;

// A group is 8 elements of a row, 16 bytes of BF16 or 32 of FP32.
__device__ __forceinline__ float load_elem(const float* p) { return *p; }
__device__ __forceinline__ float load_elem(const uint16_t* p) {
  return __uint_as_float(uint32_t(*p) << 16);
}
__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_elem(uint16_t* p, float x) {
  *p = uint16_t(cvt_bf16x2_rn(x, 0.0f));
}
// A group as it lies in memory.
template <typename T>
struct Raw {
  uint32_t u[2 * sizeof(T)];
};
__device__ __forceinline__ void load_group(const float* p, Raw<float>& x) {
  asm volatile("ld.global.L1::no_allocate.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(x.u[0]), "=r"(x.u[1]), "=r"(x.u[2]), "=r"(x.u[3]), "=r"(x.u[4]), "=r"(x.u[5]),
                 "=r"(x.u[6]), "=r"(x.u[7])
               : "l"(p));
}
__device__ __forceinline__ void load_group(const uint16_t* p, Raw<uint16_t>& x) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x.u[0]), "=r"(x.u[1]), "=r"(x.u[2]), "=r"(x.u[3])
               : "l"(p));
}
__device__ __forceinline__ void values(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(r.u[k]);
}
__device__ __forceinline__ void values(const Raw<uint16_t>& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(r.u[k] << 16);
    x[2 * k + 1] = __uint_as_float(r.u[k] & 0xFFFF0000u);
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

struct Range {
  int64_t begin, split, end;
};

// The row's history, empty (and recorded) where its offsets do not fit.
__device__ __forceinline__ Range history_of(const LogitsArgs& a, uint64_t row) {
  const int64_t b = a.begin[row], e = a.end[row];
  const int64_t s = a.split ? a.split[row] : b;
  if (b >= 0 && s >= b && e >= s && e <= a.ntokens) return {b, s, e};
  record_error(a.error_word, kErrIndex);
  return {0, 0, 0};
}

__device__ __forceinline__ Range bias_of(const LogitsArgs& a, uint64_t row) {
  const int64_t b = a.bias_begin[row], e = a.bias_begin[row + 1];
  if (b >= 0 && e >= b && e <= a.nbias) return {b, b, e};
  record_error(a.error_word, kErrIndex);
  return {0, 0, 0};
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
// has place t - base + 8, so that a group's bits are a byte of the bitmap and the
// tokens in front of the first group (row start) have places below 8.
struct Slice {
  uint32_t row;
  uint32_t first, base, stop;
  bool grouped;  // all rows involved share their group boundaries
};

template <typename TSrc, typename TDst>
__device__ __forceinline__ Slice slice_of(const LogitsArgs& a, const TSrc*& src, TDst*& dst) {
  Slice s;
  s.row = blockIdx.x / a.slices;
  const uint32_t k = blockIdx.x % a.slices;
  src += s.row * a.src_stride;
  dst += s.row * a.dst_stride;
  uint32_t lead = lead_of(src);
  s.grouped = lead == lead_of(dst);
  if (!s.grouped) lead = 0u;
  s.base = lead + k * a.slice;
  s.first = k == 0 ? 0u : min(s.base, a.vocab);
  s.stop = k + 1 == a.slices ? a.vocab : min(s.base + a.slice, a.vocab);
  return s;
}

// Calls f(in, place, position) for the entries [begin, end) of a list of tokens,
// a warp's lanes together; `in`: the entry belongs to the slice. Calls in which no
// lane has one are left out: with a dozen slices a row that is most of them. Tokens
// outside the vocabulary are recorded.
template <typename F>
__device__ __forceinline__ void scan_tokens(const LogitsArgs& a, const Slice& s, const int32_t* tokens,
                                            int64_t begin, int64_t end, F f) {
  const int32_t* p = tokens + begin;
  const uint32_t len = s.stop - s.first, off = s.first - s.base + 8u;
  const uint32_t vocab = a.vocab;
  uint32_t bad = 0u;
  auto one = [&](uint32_t t, int64_t i) {
    const bool in = t - s.first < len;
    bad |= t >= vocab;
    if (__any_sync(0xFFFFFFFFu, in)) f(in, t - s.first + off, i);
  };
  const int64_t n = end - begin;
  const int64_t lead = min(n, int64_t((0u - uint32_t(reinterpret_cast<uintptr_t>(p) / 4u)) & 3u));
  const int64_t quads = (n - lead) / 4, rest = lead + 4 * quads;
  const int4* quad = reinterpret_cast<const int4*>(p + lead);
  for (int64_t q = threadIdx.x & ~31u; q < quads; q += kThreads) {
    const int64_t at = q + (threadIdx.x & 31u);
    int4 t = make_int4(-1, -1, -1, -1);
    const bool have = at < quads;
    if (have) t = __ldg(quad + at);
    const int64_t i = begin + lead + 4 * at;
    const uint32_t before = bad;
    one(uint32_t(t.x), i);
    one(uint32_t(t.y), i + 1);
    one(uint32_t(t.z), i + 2);
    one(uint32_t(t.w), i + 3);
    if (!have) bad = before;
  }
  // up to 3 entries in front of the aligned ones and 3 behind, by the first warp
  if (threadIdx.x < 32u) {
    const int64_t i = threadIdx.x < lead ? threadIdx.x : rest + (threadIdx.x - lead);
    const bool have = i < n;
    const uint32_t before = bad;
    one(have ? uint32_t(p[i]) : 0xFFFFFFFFu, begin + i);
    if (!have) bad = before;
  }
  if (bad) record_error(a.error_word, kErrIndex);
}

// This thread's groups of a slice. Masked tokens are not read where a whole group
// is masked.
template <typename TSrc>
struct Groups {
  Raw<TSrc> x[kGroups];
  uint32_t ok[kGroups];  // a bit a token: open (0 past the slice)
  uint32_t count;        // of the slice

  __device__ __forceinline__ void load(const Slice& s, const TSrc* src, const uint32_t* mask) {
    count = s.grouped && s.stop > s.base ? (s.stop - s.base) / 8u : 0u;
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      const uint32_t q = threadIdx.x + r * kThreads;
      ok[r] = q >= count ? 0u : mask ? mask_bits8(mask, s.base + 8u * q) : 0xFFu;
    }
#pragma unroll
    for (int r = 0; r < kGroups; ++r)
      if (ok[r]) load_group(src + s.base + 8u * (threadIdx.x + r * kThreads), x[r]);
  }
};

template <typename TDst>
__device__ __forceinline__ void store_masked(TDst* p, float (&y)[8], uint32_t ok, float masked) {
  if (ok != 0xFFu) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (!((ok >> k) & 1u)) y[k] = masked;
  }
  store_group(p, y);
}

// Calls f(t) for the tokens outside the groups: all of them where there are no
// groups, else the row's first few and last few.
template <typename F>
__device__ __forceinline__ void each_single(const Slice& s, uint32_t groups, F f) {
  if (!s.grouped) {
    for (uint32_t t = s.first + threadIdx.x; t < s.stop; t += kThreads) f(t);
    return;
  }
  const uint32_t head = s.first < s.base ? min(s.base, s.stop) - s.first : 0u;
  if (threadIdx.x < head) f(s.first + threadIdx.x);
  const uint32_t tail = s.base + 8u * groups + threadIdx.x;
  if (s.stop > s.base && tail < s.stop) f(tail);
}

__device__ __forceinline__ bool open_token(const uint32_t* mask, uint32_t t) {
  return mask == nullptr || ((mask[t >> 5] >> (t & 31u)) & 1u);
}

constexpr float kClosed = -__builtin_huge_valf();

// What thread 0 reads of the row for all.
struct RowSettings {
  Range history, bias;
  float rep, inv_rep, pres, freq, inv_t;
};

__device__ __forceinline__ void read_row(const LogitsArgs& a, uint32_t row, bool history, RowSettings& r) {
  r.history = history ? history_of(a, row) : Range{0, 0, 0};
  r.bias = a.bias_tokens ? bias_of(a, row) : Range{0, 0, 0};
  r.rep = a.repetition ? a.repetition[row] : 1.0f;
  r.inv_rep = __frcp_rn(r.rep);
  r.pres = a.presence ? a.presence[row] : 0.0f;
  r.freq = a.frequency ? a.frequency[row] : 0.0f;
  const float t = a.temperature ? a.temperature[row] : 1.0f;
  r.inv_t = t > 0.0f ? __frcp_rn(t) : 1.0f;  // not above 0, greedy decoding: the row stays as it is
}

// Repetition penalty and temperature alone: a bit a token is all there is to keep.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas) scale_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t bits[kWords];
  __shared__ RowSettings row;
  const TIn* src = static_cast<const TIn*>(a.src);
  TOut* dst = static_cast<TOut*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const uint32_t* mask = mask_of(a, s.row);
  Groups<TIn> g;
  g.load(s, src, mask);
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) bits[i] = 0u;
  if (threadIdx.x == 0) read_row(a, s.row, a.tokens && a.repetition, row);
  __syncthreads();
  if (row.history.end > row.history.begin) {
    scan_tokens(a, s, a.tokens, row.history.begin, row.history.end, [&](bool in, uint32_t u, int64_t) {
      if (in) atomicOr(bits + (u >> 5), 1u << (u & 31u));
    });
    __syncthreads();
  }
  const float inv_t = row.inv_t, rep = row.rep, inv_rep = row.inv_rep;
  auto seen = [&](float x) { return __fmul_rn(__fmul_rn(x, x > 0.0f ? inv_rep : rep), inv_t); };
#pragma unroll
  for (int r = 0; r < kGroups; ++r) {
    const uint32_t q = threadIdx.x + r * kThreads;
    if (q < g.count) {
      const uint32_t hit = reinterpret_cast<const uint8_t*>(bits)[q + 1u];
      float x[8], y[8];
      values(g.x[r], x);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(x[k], inv_t);
      if (hit) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = (hit >> k) & 1u ? seen(x[k]) : y[k];
      }
      store_masked(dst + s.base + 8u * q, y, g.ok[r], kClosed);
    }
  }
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = kClosed;
    if (open_token(mask, t)) {
      const float x = load_elem(src + t);
      y = (bits[u >> 5] >> (u & 31u)) & 1u ? seen(x) : __fmul_rn(x, inv_t);
    }
    store_elem(dst + t, y);
  });
}

// Everything: tokens are counted and biased.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas) shape_kernel(const __grid_constant__ LogitsArgs a) {
  extern __shared__ uint4 smem[];
  // a word a place: bit 31 for a token of the prompt, below it the times it was
  // generated; then the logit as the penalties and the bias leave it
  uint32_t* word = reinterpret_cast<uint32_t*>(smem);
  uint16_t* list = reinterpret_cast<uint16_t*>(word + kPlaces);  // places of the history, each once
  __shared__ uint32_t bits[kWords];                              // places whose word is a logit
  __shared__ uint32_t listed;
  __shared__ RowSettings row;
  const TIn* src = static_cast<const TIn*>(a.src);
  TOut* dst = static_cast<TOut*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const uint32_t* mask = mask_of(a, s.row);
  Groups<TIn> g;
  g.load(s, src, mask);
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) bits[i] = 0u;
  for (uint32_t i = threadIdx.x; i < (a.slice + 8u + 3u) / 4u; i += kThreads)
    reinterpret_cast<uint4*>(word)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (threadIdx.x == 0) {
    listed = 0u;
    read_row(a, s.row, a.tokens && (a.repetition || a.presence || a.frequency), row);
  }
  __syncthreads();
  const uint32_t lane = threadIdx.x & 31u;
  if (row.history.end > row.history.begin) {
    const int64_t split = row.history.split;
    scan_tokens(a, s, a.tokens, row.history.begin, row.history.end, [&](bool in, uint32_t u, int64_t i) {
      uint32_t old = 1u;
      if (in) old = i >= split ? atomicAdd(word + u, 1u) : atomicOr(word + u, 0x80000000u);
      const uint32_t fresh = __ballot_sync(0xFFFFFFFFu, old == 0u);
      if (fresh) {
        uint32_t at = 0u;
        if (lane == 0) at = atomicAdd(&listed, uint32_t(__popc(fresh)));
        at = __shfl_sync(0xFFFFFFFFu, at, 0);
        if (old == 0u) list[at + __popc(fresh & lanemask_lt())] = uint16_t(u);
      }
    });
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < listed; i += kThreads) {
      const uint32_t u = list[i], made = word[u] & 0x7FFFFFFFu;
      float x = load_elem(src + (s.base + u - 8u));
      x = __fmul_rn(x, x > 0.0f ? row.inv_rep : row.rep);
      if (made != 0u) x = __fsub_rn(__fsub_rn(x, __fmul_rn(row.freq, float(made))), row.pres);
      word[u] = __float_as_uint(x);
      atomicOr(bits + (u >> 5), 1u << (u & 31u));
    }
    __syncthreads();
  }
  if (row.bias.end > row.bias.begin) {
    // Every warp reads the list backwards, 32 entries at a time, and serves the
    // places that are its own: the last entry of a token comes first, and the
    // bit it leaves in `done` turns the others away.
    uint32_t* done = reinterpret_cast<uint32_t*>(list);
    for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) done[i] = 0u;
    __syncthreads();
    const uint32_t len = s.stop - s.first, off = s.first - s.base + 8u, warp = threadIdx.x >> 5;
    uint32_t bad = 0u;
    for (int64_t last = row.bias.end; last > row.bias.begin; last -= 32) {
      const int64_t i = last - 1 - lane;  // the lowest lane has the latest entry
      const bool have = i >= row.bias.begin;
      const uint32_t t = have ? uint32_t(a.bias_tokens[i]) : 0xFFFFFFFFu, u = t - s.first + off;
      bad |= have && t >= a.vocab;
      const bool own = t - s.first < len && u * (kThreads / 32u) / kPlaces == warp;
      const uint32_t owners = __ballot_sync(0xFFFFFFFFu, own);
      if (!own) continue;
      const uint32_t same = __match_any_sync(owners, u), bit = 1u << (u & 31u);
      if (lane != uint32_t(__ffs(same) - 1)) continue;
      if (atomicOr(done + (u >> 5), bit) & bit) continue;
      const bool seen = (bits[u >> 5] & bit) != 0u;
      const float x = seen ? __uint_as_float(word[u]) : load_elem(src + (s.base + u - 8u));
      word[u] = __float_as_uint(__fadd_rn(x, a.bias_values[i]));
      atomicOr(bits + (u >> 5), bit);
    }
    if (bad) record_error(a.error_word, kErrIndex);
    __syncthreads();
  }
  const float inv_t = row.inv_t;
#pragma unroll
  for (int r = 0; r < kGroups; ++r) {
    const uint32_t q = threadIdx.x + r * kThreads;
    if (q < g.count) {
      float x[8];
      values(g.x[r], x);
      const uint32_t hit = reinterpret_cast<const uint8_t*>(bits)[q + 1u];
      if (hit) {
        const uint4 lo = reinterpret_cast<const uint4*>(word)[2u * q + 2u];
        const uint4 hi = reinterpret_cast<const uint4*>(word)[2u * q + 3u];
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = (hit >> k) & 1u ? __uint_as_float(w[k]) : x[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(x[k], inv_t);
      store_masked(dst + s.base + 8u * q, x, g.ok[r], kClosed);
    }
  }
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = kClosed;
    if (open_token(mask, t)) {
      const bool touched = (bits[u >> 5] >> (u & 31u)) & 1u;
      y = __fmul_rn(touched ? __uint_as_float(word[u]) : load_elem(src + t), inv_t);
    }
    store_elem(dst + t, y);
  });
}

// Backward: a bit a token of the history, and the raw logits of groups that have one.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas) backward_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t bits[kWords];
  __shared__ RowSettings row;
  const TOut* src = static_cast<const TOut*>(a.src);
  TIn* dst = static_cast<TIn*>(a.dst);
  Slice s = slice_of(a, src, dst);
  const TIn* raw = static_cast<const TIn*>(a.raw) + (a.raw ? s.row * a.raw_stride : 0u);
  if (a.raw && lead_of(raw) != lead_of(src)) s.grouped = false;  // places stay as they are
  const uint32_t* mask = mask_of(a, s.row);
  Groups<TOut> g;
  g.load(s, src, mask);
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) bits[i] = 0u;
  if (threadIdx.x == 0) read_row(a, s.row, a.tokens && a.repetition, row);
  __syncthreads();
  if (row.history.end > row.history.begin) {
    scan_tokens(a, s, a.tokens, row.history.begin, row.history.end, [&](bool in, uint32_t u, int64_t) {
      if (in) atomicOr(bits + (u >> 5), 1u << (u & 31u));
    });
    __syncthreads();
  }
  const float inv_t = row.inv_t, rep = row.rep, inv_rep = row.inv_rep;
  Raw<TIn> x[kGroups];
#pragma unroll
  for (int r = 0; r < kGroups; ++r) {
    const uint32_t q = threadIdx.x + r * kThreads;
    if (g.ok[r] && reinterpret_cast<const uint8_t*>(bits)[q + 1u]) load_group(raw + s.base + 8u * q, x[r]);
  }
#pragma unroll
  for (int r = 0; r < kGroups; ++r) {
    const uint32_t q = threadIdx.x + r * kThreads;
    if (q < g.count) {
      const uint32_t hit = reinterpret_cast<const uint8_t*>(bits)[q + 1u];
      float d[8];
      values(g.x[r], d);
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = __fmul_rn(d[k], inv_t);
      if (hit) {
        float v[8];
        values(x[r], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = (hit >> k) & 1u ? __fmul_rn(d[k], v[k] > 0.0f ? inv_rep : rep) : d[k];
      }
      store_masked(dst + s.base + 8u * q, d, g.ok[r], 0.0f);
    }
  }
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = 0.0f;
    if (open_token(mask, t)) {
      y = __fmul_rn(load_elem(src + t), inv_t);
      if ((bits[u >> 5] >> (u & 31u)) & 1u) y = __fmul_rn(y, load_elem(raw + t) > 0.0f ? inv_rep : rep);
    }
    store_elem(dst + t, y);
  });
}

// Slices of a row: as few as possible, since every one reads the history, but
// more where there are too few rows to give every SM two CTAs.
void cut_rows(LogitsArgs& a, int sms) {
  uint32_t k = (a.vocab + kSliceMax - 1) / kSliceMax;
  while (a.rows * k < uint64_t(sms) * 2 && a.vocab / (2 * k) >= kSliceMin) k *= 2;
  a.slices = k;
  a.slice = ((a.vocab + k - 1) / k + 7u) & ~7u;
}

template <typename K>
cudaError_t launch_full(K kernel, const LogitsArgs& a, cudaStream_t stream) {
  constexpr uint32_t kBytes = kPlaces * 6u;  // word, list
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kBytes));
  if (e != cudaSuccess) return e;
  kernel<<<unsigned(a.rows * a.slices), kThreads, kBytes, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logits_shape(LogitsArgs a, int in_type, int out_type, int sms, cudaStream_t stream) {
  cut_rows(a, sms);
  if (a.bias_tokens || (a.tokens && (a.presence || a.frequency))) {
    if (in_type == PULSE_F32) return launch_full(shape_kernel<float, float>, a, stream);
    if (out_type == PULSE_F32) return launch_full(shape_kernel<uint16_t, float>, a, stream);
    return launch_full(shape_kernel<uint16_t, uint16_t>, a, stream);
  }
  const unsigned grid = unsigned(a.rows * a.slices);
  if (in_type == PULSE_F32)
    scale_kernel<float, float><<<grid, kThreads, 0, stream>>>(a);
  else if (out_type == PULSE_F32)
    scale_kernel<uint16_t, float><<<grid, kThreads, 0, stream>>>(a);
  else
    scale_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_logits_backward(LogitsArgs a, int in_type, int out_type, int sms,
                                   cudaStream_t stream) {
  cut_rows(a, sms);
  const unsigned grid = unsigned(a.rows * a.slices);
  if (in_type == PULSE_F32)
    backward_kernel<float, float><<<grid, kThreads, 0, stream>>>(a);
  else if (out_type == PULSE_F32)
    backward_kernel<uint16_t, float><<<grid, kThreads, 0, stream>>>(a);
  else
    backward_kernel<uint16_t, uint16_t><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pulse
