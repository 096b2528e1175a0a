// fp8.cu -- FP8 (E4M3) codes with an FP32 scale for each block of 128 columns: the view
// of weights (128 rows a block), of activations (1 row a block), and the residual
// addition and RMS norm in front of them.
//
// Mathematics. scale = max(amax / 448, 2^-126), code = E4M3(x / scale). The quotient is
// the correctly rounded one: q = x * r with r the rounded reciprocal, and one correction
// q + (x - q * scale) * r in fused operations (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). A quotient that is off by its
// last bit would land on the other side of a tie between two codes, and in BF16 inputs
// ties are frequent: their values are short fractions of the block's largest. The correction needs x - q * scale exactly.
// That is a multiple of 2^-57 of the scale's binade (x above 2^-11 of it: smaller ones have code 0 whatever their last
// bits), so below a scale of 2^-92 it could pass the smallest FP32 number: blocks below 2^-90 are lifted by 2^64 first.
// amax takes a NaN along, and across lanes it is a maximum of bit patterns without the sign, under which NaN lies above
// infinity, infinity above every number: a block with either of them is found by the same maximum.
//
// Every kernel is bound by memory: an element is read once, its code written once, and
// everything between stays in registers. Measured, of the 6.8 TB/s of a copy: the view of 151936 x 1536 BF16 weights
// (701 MB) 102 us, 6.9 TB/s; 16384 x 4096 BF16 activations through the norm with a residual (472 MB) 75 us, 6.2 TB/s;
// rows off 16 bytes, 20011 x 5003 BF16, 79 us, 3.8 TB/s, bound by instructions: accesses of 2 and 1 bytes.
#include <cuda_fp8.h>

#include <type_traits>

#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126
constexpr float kSmallScale = 0x1p-90f, kLift = 0x1p64f;

// ------------------------------------------------------------------ layouts
//
// A warp holds runs of 128 columns, 32 bytes a lane: 8 FP32 values of two runs, 16 BF16 values
// of four. Packed: a run in 16 or 8 lanes, a lane's columns in a row, for matrices whose rows begin at
// multiples of 16 bytes. Loose, for all others: a run in 32 lanes, lane i columns i, i + 32, i + 64,
// i + 96, so that a warp's accesses of single elements lie side by side (333 x 5003 FP32 through
// the norm: 6 us; with 8 columns in a row a lane, 30 us), none of them behind a branch, so that all are under way at once.
// What a run costs beside its elements (scale, reciprocal,
// maximum, addresses) is most of the instructions: 16 values a lane instead of 8 took the embedding's BF16 view of
// 151936 x 1536 from 149 to 104 us, arithmetic by pairs 16384 x 8960 from 78 to 73 us. Values are kept as they are read until they are needed.
template <typename T>
constexpr int kEach = 32 / int(sizeof(T));
template <typename T>
constexpr int kRuns = kEach<T> / 4;

struct Raw {
  uint32_t v[8];
};
__device__ __forceinline__ void unpack(const Raw& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(r.v[k]);
}
__device__ __forceinline__ void unpack(const Raw& r, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __uint_as_float(r.v[k] << 16);
    x[2 * k + 1] = __uint_as_float(r.v[k] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ Raw negated(const Raw& r, const float*) {
  Raw n;
#pragma unroll
  for (int k = 0; k < 8; ++k) n.v[k] = r.v[k] ^ 0x80000000u;
  return n;
}
__device__ __forceinline__ Raw negated(const Raw& r, const uint16_t*) {
  Raw n;
#pragma unroll
  for (int k = 0; k < 8; ++k) n.v[k] = r.v[k] ^ 0x80008000u;
  return n;
}

template <typename T>
struct Run {
  T* p;           // column 0
  uint32_t left;  // columns of the matrix from there on, 128 at most; 0: nothing there
};
__device__ __forceinline__ uint32_t left_of(uint32_t col, uint32_t cols) { return col < cols ? min(cols - col, 128u) : 0u; }

template <typename T>
__device__ __forceinline__ uint32_t bits_of(T x) {
  if constexpr (sizeof(T) == 4)
    return __float_as_uint(x);
  else
    return x;
}

// Loose: value k is of run k / 4, this column.
__device__ __forceinline__ uint32_t loose_col(uint32_t k) { return (threadIdx.x & 31u) + 32u * (k & 3u); }
// Packed: the run that a lane works on, and its first column there.
template <typename T>
__device__ __forceinline__ uint32_t own_run() { return (threadIdx.x & 31u) / (128 / kEach<T>); }
template <typename T>
__device__ __forceinline__ uint32_t own_col() { return (threadIdx.x & (128 / kEach<T> - 1)) * kEach<T>; }

// `at(h)`: run h of the warp. kFull: loose, all runs have 128 columns, known to be there (a check of each element, or a branch
// for each run, took the 1-row view of 20011 x 5003 BF16 from 80 to 112 and 137 us).
template <typename T, bool kLoose, bool kFull, typename At>
__device__ __forceinline__ Raw load_runs(At at) {
  Raw out;
  if constexpr (!kLoose) {
    const auto r = at(own_run<T>());
    const uint32_t col = own_col<T>();
    const T* p = r.p + col;
    if (col + kEach<T> <= r.left) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
      out.v[0] = a.x, out.v[1] = a.y, out.v[2] = a.z, out.v[3] = a.w;
      out.v[4] = b.x, out.v[5] = b.y, out.v[6] = b.z, out.v[7] = b.w;
      return out;
    }
    constexpr int kPer = 4 / int(sizeof(T));
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      out.v[k] = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (col + k * kPer + j < r.left) out.v[k] |= bits_of(p[k * kPer + j]) << (16 * j);
    }
  } else {
#pragma unroll
    for (int h = 0; h < kRuns<T>; ++h) {
      const auto r = at(h);
      uint32_t e[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) e[j] = kFull || loose_col(j) < r.left ? bits_of(r.p[loose_col(j)]) : 0u;
      if constexpr (sizeof(T) == 4)
        out.v[h * 4] = e[0], out.v[h * 4 + 1] = e[1], out.v[h * 4 + 2] = e[2], out.v[h * 4 + 3] = e[3];
      else
        out.v[h * 2] = __byte_perm(e[0], e[1], 0x5410), out.v[h * 2 + 1] = __byte_perm(e[2], e[3], 0x5410);
    }
  }
  return out;
}

// The same words back.
template <typename T, bool kLoose, bool kFull, typename At>
__device__ __forceinline__ void store_runs(At at, const Raw& x) {
  auto element = [&](uint32_t k) {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(x.v[k]);
    else
      return uint16_t(x.v[k >> 1] >> (16 * (k & 1)));
  };
  if constexpr (!kLoose) {
    const Run<T> r = at(own_run<T>());
    const uint32_t col = own_col<T>();
    T* p = r.p + col;
    if (col + kEach<T> <= r.left) {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(x.v[0], x.v[1], x.v[2], x.v[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(x.v[4], x.v[5], x.v[6], x.v[7]);
    } else {
#pragma unroll
      for (uint32_t k = 0; k < kEach<T>; ++k)
        if (col + k < r.left) p[k] = element(k);
    }
  } else {
#pragma unroll
    for (int h = 0; h < kRuns<T>; ++h) {
      const Run<T> r = at(h);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (kFull || loose_col(j) < r.left) r.p[loose_col(j)] = element(h * 4 + j);
    }
  }
}

// The sums of two sets of words, rounded; `out`: their values.
__device__ __forceinline__ Raw add_raw(const Raw& a, const Raw& b, float (&out)[8]) {
  Raw s;
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = __fadd_rn(__uint_as_float(a.v[k]), __uint_as_float(b.v[k])), s.v[k] = __float_as_uint(out[k]);
  return s;
}
__device__ __forceinline__ Raw add_raw(const Raw& a, const Raw& b, float (&out)[16]) {
  Raw s;
  float x[16];
  unpack(a, x);
  unpack(b, out);
  uint32_t nan = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __fadd_rn(x[2 * k], out[2 * k]), x[2 * k + 1] = __fadd_rn(x[2 * k + 1], out[2 * k + 1]);
    s.v[k] = cvt_bf16x2_rn(x[2 * k], x[2 * k + 1]);
    if (k & 1) nan |= any_nan4(x[2 * k - 2], x[2 * k - 1], x[2 * k], x[2 * k + 1]);
  }
  if (nan)
#pragma unroll
    for (int k = 0; k < 8; ++k) s.v[k] = canon_nan_pair(s.v[k], x[2 * k], x[2 * k + 1]);
  unpack(s, out);
  return s;
}

// max(amax / 448, 2^-126), NaN for a NaN or an infinity. The quotient as at the head of the file, with the rounded 1 / 448.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  constexpr float kInverse = 1.0f / 448.0f;
  const float x = __uint_as_float(amax), q = __fmul_rn(x, kInverse), s = __fmaf_rn(__fmaf_rn(q, -448.0f, x), kInverse, q);
  return amax >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(s, kLeastScale);
}
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// Codes of x[0] .. x[3], whose negatives `n` holds, with divisor s: (q s - x)(-1 / s) + q, two at a time. With these signs -0 stays -0.
__device__ __forceinline__ uint32_t codes4(const float* n, float s, float inv) {
  const unsigned long long s2 = pair_of(s, s), i2 = pair_of(-inv, -inv);
  uint32_t c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const unsigned long long x = pair_of(n[2 * k], n[2 * k + 1]), q = mul2(x, i2);
    unsigned long long t = x, v = q;
    fma2(t, q, s2);
    fma2(v, t, i2);
    float lo, hi;
    unpair(v, lo, hi);
    c[k] = codes2(lo, hi);
  }
  return __byte_perm(c[0], c[1], 0x5410);
}

// The divisor of kCount values, whose negatives are `n`: their scale, both lifted where it is small.
template <int kCount>
__device__ __forceinline__ float divisor_of(float* n, float s) {
  if (!(s < kSmallScale)) return s;
#pragma unroll
  for (int k = 0; k < kCount; ++k) n[k] = __fmul_rn(n[k], kLift);
  return __fmul_rn(s, kLift);
}

// Scales of the runs: packed, s[0] is the own run's.
template <typename T, bool kLoose>
__device__ __forceinline__ void scales_of(const float (&x)[kEach<T>], float (&s)[kRuns<T>]) {
  if constexpr (kLoose) {
#pragma unroll
    for (int h = 0; h < kRuns<T>; ++h)
      s[h] = scale_of(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(max_abs3(max_abs3(x[h * 4], x[h * 4 + 1], x[h * 4 + 2]), x[h * 4 + 3], 0.0f))));
  } else {
    float most = max_abs3(x[0], x[1], 0.0f);
#pragma unroll
    for (int k = 2; k < kEach<T>; k += 2) most = max_abs3(most, x[k], x[k + 1]);
    uint32_t m = __float_as_uint(most);
#pragma unroll
    for (int d = 64 / kEach<T>; d; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    s[0] = scale_of(m);
  }
}

// Codes of the warp's runs, whose negatives are `n` (not needed after): `at(h)` gives run h's. kUsual: no scale is small.
template <typename T, bool kLoose, bool kFull, bool kUsual = false, typename At>
__device__ __forceinline__ void store_codes(At at, float (&n)[kEach<T>], const float (&s)[kRuns<T>]) {
  if constexpr (!kLoose) {
    const Run<uint8_t> r = at(own_run<T>());
    const uint32_t col = own_col<T>();
    const float d = kUsual ? s[0] : divisor_of<kEach<T>>(n, s[0]), inv = __frcp_rn(d);
    uint32_t c[kEach<T> / 4];
#pragma unroll
    for (int k = 0; k < kEach<T> / 4; ++k) c[k] = codes4(n + 4 * k, d, inv);
    uint8_t* p = r.p + col;
    if (col + kEach<T> <= r.left) {
      if constexpr (kEach<T> == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(c[0], c[1]);
      else
        *reinterpret_cast<uint4*>(p) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
#pragma unroll
      for (uint32_t k = 0; k < kEach<T>; ++k)
        if (col + k < r.left) p[k] = uint8_t(c[k >> 2] >> (8 * (k & 3)));
    }
  } else {
    float d[kRuns<T>], least = s[0];
#pragma unroll
    for (int h = 0; h < kRuns<T>; ++h) d[h] = s[h], least = fminf(least, s[h]);
    if (!kUsual && least < kSmallScale)  // one branch for all runs
#pragma unroll
      for (int h = 0; h < kRuns<T>; ++h) d[h] = divisor_of<4>(n + h * 4, s[h]);
#pragma unroll
    for (int h = 0; h < kRuns<T>; ++h) {
      const Run<uint8_t> r = at(h);
      const uint32_t c = codes4(n + h * 4, d[h], __frcp_rn(d[h]));
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (kFull || loose_col(j) < r.left) r.p[loose_col(j)] = uint8_t(c >> (8 * j));
    }
  }
}
// A run's scale, by one lane: `put(h, scale)` for every run of the warp.
template <typename T, bool kLoose, typename Put>
__device__ __forceinline__ void store_scales(const float (&s)[kRuns<T>], Put put) {
  if constexpr (!kLoose) {
    if (own_col<T>() == 0) put(own_run<T>(), s[0]);
  } else {
    if ((threadIdx.x & 31u) == 0)
#pragma unroll
      for (int h = 0; h < kRuns<T>; ++h) put(h, s[h]);
  }
}

// ------------------------------------------------------------- a row a block
constexpr int kRowThreads = 256, kRowTurns = 2;  // a warp's sets of runs

template <typename T, bool kLoose>
__global__ void __launch_bounds__(kRowThreads) quantize_rows_kernel(Fp8Args a) {
  stream_ready();
  constexpr uint32_t kStep = kRowThreads / 32 * kRuns<T>;
  const uint32_t first = blockIdx.x * kStep * kRowTurns + (threadIdx.x >> 5) * kRuns<T>;
  struct Place {
    uint32_t row, block;
  };
  auto place = [&](uint32_t unit) {
    const uint32_t row = a.rows == 1 ? 0u : a.blocks == 1 ? unit : __umulhi(unit, a.by_blocks) >> a.by_blocks_shift;
    return Place{row, unit - row * a.blocks};
  };
  // run h of a set that begins at `unit`; loose, the runs are asked for one after the other
  auto follow = [&](uint32_t unit, Place from) {
    return [&a, &place, unit, from](uint32_t h) mutable {
      if constexpr (!kLoose) return place(unit + h);
      if (h && ++from.block == a.blocks) from.block = 0, ++from.row;
      return from;
    };
  };
  auto full = [&](uint32_t unit, const Place& p) { return kLoose && unit < a.units && (p.block + kRuns<T>) * 128 <= a.cols; };
  Raw raw[kRowTurns];
  Place from[kRowTurns];
#pragma unroll
  for (int j = 0; j < kRowTurns; ++j) {
    const uint32_t unit = first + j * kStep;
    from[j] = place(unit);
    if (full(unit, from[j])) {
      const T* x = static_cast<const T*>(a.x) + from[j].row * a.stride + uint64_t(from[j].block) * 128;
      raw[j] = load_runs<T, kLoose, true>([&](uint32_t h) { return Run<const T>{x + h * 128, 128}; });
    } else {
      auto run = follow(unit, from[j]);
      raw[j] = load_runs<T, kLoose, false>([&](uint32_t h) {
        const Place p = run(h);
        const bool in = unit + h < a.units;
        return Run<const T>{static_cast<const T*>(a.x) + (in ? p.row * a.stride + uint64_t(p.block) * 128 : 0), in ? left_of(p.block * 128, a.cols) : 0u};
      });
    }
  }
#pragma unroll
  for (int j = 0; j < kRowTurns; ++j) {
    const uint32_t unit = first + j * kStep;
    float x[kEach<T>], s[kRuns<T>];  // the negatives
    unpack(negated(raw[j], static_cast<const T*>(nullptr)), x);
    scales_of<T, kLoose>(x, s);
    auto run = follow(unit, from[j]), again = run;
    store_scales<T, kLoose>(s, [&](uint32_t h, float scale) {
      const Place p = run(h);
      if (unit + h < a.units) a.scales[p.row * a.scales_stride + p.block] = scale;
    });
    if (full(unit, from[j])) {
      uint8_t* codes = a.codes + from[j].row * a.codes_stride + uint64_t(from[j].block) * 128;
      store_codes<T, kLoose, true>([&](uint32_t h) { return Run<uint8_t>{codes + h * 128, 128}; }, x, s);
    } else {
      store_codes<T, kLoose, false>(
          [&](uint32_t h) {
            const Place p = again(h);
            const bool in = unit + h < a.units;
            return Run<uint8_t>{a.codes + (in ? p.row * a.codes_stride + uint64_t(p.block) * 128 : 0), in ? left_of(p.block * 128, a.cols) : 0u};
          },
          x, s);
    }
  }
}

// --------------------------------------------------------- 128 rows a block
constexpr int kTallThreads = 512;
template <typename T>
constexpr int kTallTurns = 128 / (kTallThreads / 32 * kRuns<T>);  // sets of rows a warp takes

template <typename T, bool kLoose>
__global__ void __launch_bounds__(kTallThreads, sizeof(T) == 4 ? 2 : kLoose ? 3 : 4) quantize_tall_kernel(Fp8Args a) {
  __shared__ uint32_t most[kTallThreads / 32];
  stream_ready();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t group = blockIdx.x / a.blocks, block = blockIdx.x - group * a.blocks, left = left_of(block * 128, a.cols);
  auto row_of = [&](int j, uint32_t h) { return uint64_t(group) * 128 + (j * (kTallThreads / 32) + warp) * kRuns<T> + h; };
  const bool full = kLoose && left == 128 && (uint64_t(group) + 1) * 128 <= a.rows;
  Raw raw[kTallTurns<T>];
  auto load = [&](auto all) {
#pragma unroll
    for (int j = 0; j < kTallTurns<T>; ++j)
      raw[j] = load_runs<T, kLoose, decltype(all)::value>([&](uint32_t h) {
        const uint64_t row = row_of(j, h);
        const bool in = decltype(all)::value || row < a.rows;
        return Run<const T>{static_cast<const T*>(a.x) + (in ? row * a.stride + uint64_t(block) * 128 : 0), in ? left : 0u};
      });
  };
  if (full)
    load(std::true_type{});
  else
    load(std::false_type{});
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kTallTurns<T>; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      m = sizeof(T) == 4 ? max(m, raw[j].v[k] & 0x7FFFFFFFu) : __vmaxu2(m, raw[j].v[k] & 0x7FFF7FFFu);
  if (sizeof(T) == 2) m = max(m << 16, m & 0xFFFF0000u);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) most[warp] = m;
  __syncthreads();
  m = __reduce_max_sync(0xFFFFFFFFu, lane < kTallThreads / 32 ? most[lane] : 0u);
  float s[kRuns<T>];
#pragma unroll
  for (int h = 0; h < kRuns<T>; ++h) s[h] = scale_of(m);
  if (threadIdx.x == 0) a.scales[uint64_t(group) * a.scales_stride + block] = s[0];
  auto store = [&](auto all, auto usual) {
#pragma unroll
    for (int j = 0; j < kTallTurns<T>; ++j) {
      float x[kEach<T>];  // the negatives
      unpack(negated(raw[j], static_cast<const T*>(nullptr)), x);
      store_codes<T, kLoose, decltype(all)::value, decltype(usual)::value>(
          [&](uint32_t h) {
            const uint64_t row = row_of(j, h);
            const bool in = decltype(all)::value || row < a.rows;
            return Run<uint8_t>{a.codes + (in ? row * a.codes_stride + uint64_t(block) * 128 : 0), in ? left : 0u};
          },
          x, s);
    }
  };
  // one choice for all: with one in each set 151936 x 1536 took 104 us instead of 102
  if (s[0] < kSmallScale)
    store(std::false_type{}, std::false_type{});
  else if (full)
    store(std::true_type{}, std::true_type{});
  else
    store(std::false_type{}, std::true_type{});
}

// --------------------------------------------------------------- RMS norm
// A CTA a row, kRuns * 128 columns a warp and turn. kTurns > 0: the row stays in registers, and the next one
// is asked for before this one is normed; 0: rows of more than 2 * 8192 columns, whose sum (or x)
// is read again for the second half.
template <typename T, bool kLoose>
struct NormRow {
  const Fp8Args& a;
  uint64_t row;
  template <typename V>
  __device__ Run<V> run(V* p, uint64_t stride, uint32_t col) const {
    const uint32_t left = left_of(col, a.cols);
    return Run<V>{p + row * stride + (left ? col : 0u), left};
  }
  __device__ Raw load(const void* p, uint64_t stride, uint32_t col) const {
    auto at = [&](uint32_t h) { return run(static_cast<const T*>(p), stride, col + h * 128); };
    return full(col) ? load_runs<T, kLoose, true>(at) : load_runs<T, kLoose, false>(at);
  }
  __device__ bool full(uint32_t col) const { return kLoose && col + kRuns<T> * 128 <= a.cols; }
  // x + residual, rounded and stored
  __device__ void add(uint32_t col, const Raw& x, const Raw& res, float (&h)[kEach<T>]) const {
    if (!a.residual) return unpack(x, h);
    const Raw sum = add_raw(x, res, h);
    auto at = [&](uint32_t i) { return run(static_cast<T*>(a.sum), a.sum_stride, col + i * 128); };
    if (full(col))
      store_runs<T, kLoose, true>(at, sum);
    else
      store_runs<T, kLoose, false>(at, sum);
  }
  __device__ void store(uint32_t col, const float (&h)[kEach<T>], const float (&g)[kEach<T>], float rstd) const {
    float y[kEach<T>], s[kRuns<T>];  // the negatives
    const unsigned long long by = pair_of(-rstd, -rstd);
#pragma unroll
    for (int k = 0; k < kEach<T>; k += 2)
      unpair(mul2(mul2(pair_of(h[k], h[k + 1]), by), pair_of(g[k], g[k + 1])), y[k], y[k + 1]);
    scales_of<T, kLoose>(y, s);
    store_scales<T, kLoose>(s, [&](uint32_t i, float scale) {
      if (col + i * 128 < a.cols) a.scales[row * a.scales_stride + (col >> 7) + i] = scale;
    });
    auto at = [&](uint32_t i) { return run(a.codes, a.codes_stride, col + i * 128); };
    if (full(col))
      store_codes<T, kLoose, true>(at, y, s);
    else
      store_codes<T, kLoose, false>(at, y, s);
  }
};

template <typename T, bool kLoose>
__device__ __forceinline__ void load_weight(const Fp8Args& a, uint32_t col, float (&g)[kEach<T>]) {
#pragma unroll
  for (uint32_t k = 0; k < kEach<T>; ++k) {
    const uint32_t c = col + (kLoose ? loose_col(k) + 128u * (k >> 2) : (threadIdx.x & 31u) * kEach<T> + k);
    g[k] = 1.0f;
    if (a.weight && c < a.cols)
      g[k] = a.weight_bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t*>(a.weight)[c]) << 16) : static_cast<const float*>(a.weight)[c];
  }
}

// Two sums of squares in one register pair.
template <int kCount>
__device__ __forceinline__ void add_squares(unsigned long long& squares, const float (&v)[kCount]) {
#pragma unroll
  for (int k = 0; k < kCount; k += 2) {
    const unsigned long long p = pair_of(v[k], v[k + 1]);
    fma2(squares, p, p);
  }
}
// Of all threads; `part`: one for each warp, with a barrier before it is used again.
__device__ __forceinline__ float sum_of(float v, float* part) {
  const uint32_t warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ float mean_of(const Fp8Args& a, unsigned long long squares, float* part) {
  float lo, hi;
  unpair(squares, lo, hi);
  return __fadd_rn(__fdiv_rn(sum_of(lo + hi, part), float(a.cols)), a.eps);
}
// Squares are off by 2^-150 each, no more than 2^-50 of a mean (with eps) in this range. NaN, too, has no better one.
__device__ __forceinline__ bool fits(float mean) { return !(mean < 0x1p-100f || mean > 3.4028234e38f); }

// The CTA's rows whose mean does not fit, once more: read again, times a power of two that takes a row's largest, or the
// root of eps, near 1. All rows' sums are taken again, in the same order, to know which they are: noted down, or treated in the
// loop itself, they cost the other rows (16384 x 4096 BF16 without residual 53 to 55 us instead of 50).
template <typename T, bool kLoose>
__device__ __noinline__ void norm_lifted(const Fp8Args& args, float (&part)[2][32]) {
  const Fp8Args a = args;
  constexpr uint32_t kWide = kRuns<T> * 128;
  const uint32_t warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const NormRow<T, kLoose> now{a, row};
    auto each = [&](auto f) {  // a thread reads what it has stored of the sum itself
#pragma unroll 1
      for (uint32_t col = warp * kWide; col < a.cols; col += warps * kWide) {
        float v[kEach<T>];
        unpack(a.residual ? now.load(a.sum, a.sum_stride, col) : now.load(a.x, a.stride, col), v);
        f(col, v);
      }
    };
    unsigned long long squares = 0;
    each([&](uint32_t, float (&v)[kEach<T>]) { add_squares<kEach<T>>(squares, v); });
    __syncthreads();
    if (fits(mean_of(a, squares, part[0]))) continue;
    uint32_t most = 0;
    each([&](uint32_t, float (&v)[kEach<T>]) {
#pragma unroll
      for (int k = 0; k < kEach<T>; ++k) most = max(most, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    });
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) part[1][warp] = __uint_as_float(most);
    __syncthreads();
    most = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? __float_as_uint(part[1][lane]) : 0u);
    int up = 127 - int(most >> 23);
    if (a.eps > 0.0f) up = min(up, (127 - int(__float_as_uint(a.eps) >> 23)) / 2);
    const float lift = __uint_as_float(uint32_t(max(-126, min(126, up)) + 127) << 23);
    float ss = 0.0f;
    each([&](uint32_t, float (&v)[kEach<T>]) {
#pragma unroll
      for (int k = 0; k < kEach<T>; ++k) {
        v[k] = __fmul_rn(v[k], lift);
        ss = __fmaf_rn(v[k], v[k], ss);
      }
    });
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum_of(ss, part[0]), float(a.cols)), __fmul_rn(__fmul_rn(a.eps, lift), lift)));
    each([&](uint32_t col, float (&v)[kEach<T>]) {
      float g[kEach<T>];
      load_weight<T, kLoose>(a, col, g);
#pragma unroll
      for (int k = 0; k < kEach<T>; ++k) v[k] = __fmul_rn(v[k], lift);
      now.store(col, v, g, rstd);
    });
  }
}

template <typename T>
constexpr int kNormThreads = 8192 / kEach<T>;  // a row of 8192 columns

template <typename T, int kTurns, bool kLoose>
__global__ void __launch_bounds__(kNormThreads<T>, sizeof(T) == 2 && kTurns < 2 ? 2 : 1) norm_kernel(Fp8Args a) {
  __shared__ float part[2][32];
  stream_ready();
  constexpr int kKeep = kTurns ? kTurns : 1;
  constexpr uint32_t kWide = kRuns<T> * 128;
  const uint32_t warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  auto col_of = [&](int t) { return (t * warps + warp) * kWide; };
  float g[kKeep][kEach<T>];
  Raw x[kKeep], res[kKeep];
  auto ask = [&](uint64_t row) {
    const NormRow<T, kLoose> r{a, row};
#pragma unroll
    for (int t = 0; t < kKeep; ++t) {
      x[t] = r.load(a.x, a.stride, col_of(t));
      if (a.residual) res[t] = r.load(a.residual, a.residual_stride, col_of(t));
    }
  };
  if (kTurns) {
    ask(blockIdx.x);
#pragma unroll
    for (int t = 0; t < kKeep; ++t) load_weight<T, kLoose>(a, col_of(t), g[t]);
  }
  int turn = 0;
  bool whole = true;  // FP32 has held every mean square so far
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const NormRow<T, kLoose> now{a, row};
    float h[kKeep][kEach<T>];
    unsigned long long squares = 0;
    if (kTurns) {
#pragma unroll
      for (int t = 0; t < kKeep; ++t) {
        now.add(col_of(t), x[t], res[t], h[t]);
        add_squares<kEach<T>>(squares, h[t]);
      }
      if (row + gridDim.x < a.rows) ask(row + gridDim.x);
    } else {
      for (uint32_t col = warp * kWide; col < a.cols; col += warps * kWide) {
        x[0] = now.load(a.x, a.stride, col);
        if (a.residual) res[0] = now.load(a.residual, a.residual_stride, col);
        now.add(col, x[0], res[0], h[0]);
        add_squares<kEach<T>>(squares, h[0]);
      }
    }
    // two sets of parts: a warp may be a row ahead of one that still reads
    const float mean = mean_of(a, squares, part[turn]), rstd = __frsqrt_rn(mean);
    whole = whole && fits(mean);
    if (kTurns) {
#pragma unroll
      for (int t = 0; t < kKeep; ++t) now.store(col_of(t), h[t], g[t], rstd);
    } else {
      for (uint32_t col = warp * kWide; col < a.cols; col += warps * kWide) {
        unpack(a.residual ? now.load(a.sum, a.sum_stride, col) : now.load(a.x, a.stride, col), h[0]);
        load_weight<T, kLoose>(a, col, g[0]);
        now.store(col, h[0], g[0], rstd);
      }
    }
  }
  if (!whole) norm_lifted<T, kLoose>(a, part);
}

template <typename T, bool kLoose>
cudaError_t norm_of(const Fp8Args& a, int sms, cudaStream_t stream) {
  constexpr uint32_t kWide = kRuns<T> * 128;
  const uint32_t warps = (a.cols + kWide - 1) / kWide, most = kNormThreads<T> / 32;
  const unsigned threads = (warps < most ? warps : most) * 32;
  const uint64_t ctas = uint64_t(sms) * (2048u / threads < 16u ? 2048u / threads : 16u);
  const dim3 grid(unsigned(a.rows < ctas ? a.rows : ctas));
  if (a.cols <= 8192) return launch_early(norm_kernel<T, 1, kLoose>, grid, threads, stream, a);
  if (a.cols <= 16384) return launch_early(norm_kernel<T, 2, kLoose>, grid, threads, stream, a);
  return launch_early(norm_kernel<T, 0, kLoose>, grid, threads, stream, a);
}

template <typename T, bool kLoose>
cudaError_t quantize_of(Fp8Args a, bool tall, cudaStream_t stream) {
  if (tall)
    return launch_early(quantize_tall_kernel<T, kLoose>, dim3(unsigned((a.rows + 127) / 128 * a.blocks)), kTallThreads, stream, a);
  const uint64_t all = a.rows * a.cols;
  if (a.cols % 128 == 0 && a.stride == a.cols && a.codes_stride == a.cols && a.scales_stride == a.blocks && all < (1ull << 31)) {
    a.rows = 1;  // whole rows behind one another are one long row
    a.cols = uint32_t(all);
    a.blocks = a.units;
  }
  // unit / blocks for units below 2^31: 2^(31 + s) / blocks rounded up, 2^s >= blocks, is off by less than 2^s of 2^(31 + s)
  uint32_t bits = 1;
  while ((1ull << bits) < a.blocks) ++bits;
  a.by_blocks = uint32_t(((1ull << (31 + bits)) + a.blocks - 1) / a.blocks);
  a.by_blocks_shift = bits - 1;
  constexpr uint32_t kUnits = kRowThreads / 32 * kRuns<T> * kRowTurns;
  return launch_early(quantize_rows_kernel<T, kLoose>, dim3((a.units + kUnits - 1) / kUnits), kRowThreads, stream, a);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8Args& a, bool bf16, bool tall, cudaStream_t stream) {
  if (bf16) return a.packed ? quantize_of<uint16_t, false>(a, tall, stream) : quantize_of<uint16_t, true>(a, tall, stream);
  return a.packed ? quantize_of<float, false>(a, tall, stream) : quantize_of<float, true>(a, tall, stream);
}

cudaError_t launch_rmsnorm_fp8(const Fp8Args& a, bool bf16, int sms, cudaStream_t stream) {
  if (bf16) return a.packed ? norm_of<uint16_t, false>(a, sms, stream) : norm_of<uint16_t, true>(a, sms, stream);
  return a.packed ? norm_of<float, false>(a, sms, stream) : norm_of<float, true>(a, sms, stream);
}

}  // namespace pulse
