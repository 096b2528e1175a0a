// logits.cu -- logit shaping (repetition, presence and frequency penalties,
// biases, temperature, grammar masks) and its gradient, with the formulas of
// include/pulse.h.
//
// A row is cut into slices, one CTA each. A CTA asks for its slice, reads the
// row's history and bias list meanwhile, keeps a bit for every token of its slice
// that they name (and, where tokens are counted or biased, a word), and then works
// off the slice from registers. So logits are read and written once, whatever the
// lists say, and nothing depends on the order of the tokens' atomics: bits are ORed
// and counts are integers. Everything is computed in FP32, rounded step by step as the
// formulas say, and rounded once more where the output is BF16.
//
// Quotients are products with the divisor's rounded reciprocal, one unit further from
// the quotient than its own rounding at most. Dividing where a token was seen costs
// instructions and registers (spills) in kernels that have neither to spare: 256 rows of
// 128,256 with histories up to 8,192 take 66 us instead of 52.5, the gradient of 4,096
// rows 545 instead of 453, 3,001 FP32 rows of 32,003 120 instead of 112.5; dividing by the
// temperature too 76, 809 and 136.
#include <type_traits>

#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"

namespace pulse {
namespace {

constexpr int kThreads = 256;
// CTAs per SM: as many as the registers of a slice's groups leave. One more spills; the
// FP32 gradient, which holds the raw logits beside its groups, spills as it is (168 bytes
// stored and 196 loaded a thread: 2,000 rows of 32,003 take 99 us for 76 us of bytes).
template <typename TSrc>
constexpr int kMinCtas = sizeof(TSrc) == 4 ? 4 : 5;
// Groups of 8 elements a thread holds: its whole part of a slice, asked for before the
// history is read. Longer slices would scan each history fewer times, but hold more
// registers; 512 threads a CTA served only few rows with long histories better.
constexpr int kGroups = 4;
constexpr uint32_t kSliceMin = 2048;
constexpr uint32_t kRound = 8u * kThreads;  // tokens of a group a thread
constexpr uint32_t kSliceMax = kRound * kGroups;
constexpr uint32_t kWords = (kSliceMax + 8u + 31u) / 32u;  // of a bitmap of a slice's places
constexpr uint32_t kPlaces = kWords * 32u;
constexpr uint32_t kBlock = 2048;       // tokens that are sorted together
constexpr uint32_t kSortSlices = 250;   // most slices that are sorted for
constexpr unsigned kRowsY = 32768;      // rows of a grid's second dimension

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
// y = x * f, two products an instruction.
__device__ __forceinline__ void scale8(const float (&x)[8], float f, float (&y)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 2)
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(y[k]), "=f"(y[k + 1])
        : "f"(x[k]), "f"(x[k + 1]), "f"(f));
}
// Elements from p to the next group boundary.
template <typename T>
__device__ __forceinline__ uint32_t lead_of(const T* p) {
  return uint32_t(0u - uint32_t(reinterpret_cast<uintptr_t>(p) / sizeof(T))) & 7u;
}

// A row's settings. Ranges that do not fit their lists
// are empty (and recorded).
struct RowSettings {
  const int32_t* tokens;   // the history; not read where the tokens are sorted
  uint32_t history, made;  // its length, and where its generated part starts
  uint32_t block, from;    // sorted tokens: first block, and the history's place in it
  uint32_t biased;         // length of the bias list
  const int32_t* bias_tokens;
  const float* bias_values;
  const uint32_t* mask;    // null: all tokens are open
  float rep, inv_rep, pres, freq, inv_t;
};

// A warp for each kind of setting: what a single one would do for all holds the
// others up at the barrier.
__device__ __forceinline__ void read_row(const LogitsArgs& a, uint32_t row, bool history, RowSettings& r) {
  const uint32_t lane = threadIdx.x & 31u;
  if (threadIdx.x < 32u) {
    const int64_t* p = lane == 0 ? a.begin : lane == 1 ? (a.split ? a.split : a.begin) : a.end;
    const int64_t v = history && lane < 3 ? p[row] : 0;
    const int64_t begin = __shfl_sync(0xFFFFFFFFu, v, 0), split = __shfl_sync(0xFFFFFFFFu, v, 1),
                  end = __shfl_sync(0xFFFFFFFFu, v, 2);
    const bool ok = begin >= 0 && split >= begin && end >= split && end <= a.ntokens && end - begin < (1ll << 31);
    if (lane == 0) {
      r.tokens = a.tokens + begin;
      r.history = ok ? uint32_t(end - begin) : 0u;
      r.made = uint32_t(split - begin);
      r.block = uint32_t(begin / kBlock);
      r.from = uint32_t(begin % kBlock);
      if (!ok) record_error(a.error_word, kErrIndex);
    }
  } else if (threadIdx.x < 64u) {
    const int64_t v = a.bias_tokens && lane < 2 ? a.bias_begin[row + lane] : 0;
    const int64_t begin = __shfl_sync(0xFFFFFFFFu, v, 0), end = __shfl_sync(0xFFFFFFFFu, v, 1);
    const bool ok = begin >= 0 && end >= begin && end <= a.nbias;
    if (lane == 0) {
      r.biased = ok ? uint32_t(end - begin) : 0u;
      r.bias_tokens = a.bias_tokens + begin;
      r.bias_values = a.bias_values + begin;
      if (!ok) record_error(a.error_word, kErrIndex);
    }
  } else if (threadIdx.x < 96u) {
    const float* p = lane == 0 ? a.repetition : lane == 1 ? a.temperature : lane == 2 ? a.presence : a.frequency;
    const float v = lane < 4 && p ? p[row] : lane < 2 ? 1.0f : 0.0f;
    if (lane == 0) r.rep = v, r.inv_rep = __frcp_rn(v);
    if (lane == 1) r.inv_t = v > 0.0f ? __frcp_rn(v) : 1.0f;  // not above 0, greedy decoding: the row stays as it is
    if (lane == 2) r.pres = v;
    if (lane == 3) r.freq = v;
  } else if (threadIdx.x == 96u) {
    const int64_t m = a.mask == nullptr ? -1 : a.mask_row ? int64_t(a.mask_row[row]) : int64_t(row);
    r.mask = m >= 0 && m < a.mask_rows ? a.mask + uint64_t(m) * a.mask_stride : nullptr;
    if (a.mask && m >= a.mask_rows) record_error(a.error_word, kErrIndex);
  }
}

// This CTA's part of a row: tokens [first, stop), groups from `base` on, up to 7
// tokens later. Token t has place t - base + 8, so that a group's bits are a byte
// of the bitmap and the tokens in front of the first group have places below 8.
struct Slice {
  uint32_t row, index;
  uint32_t first, base, stop;
  bool grouped;  // all rows involved share their group boundaries
};

template <typename TSrc, typename TDst>
__device__ __forceinline__ Slice slice_of(const LogitsArgs& a, const TSrc*& src, TDst*& dst) {
  Slice s;
  s.row = blockIdx.z * kRowsY + blockIdx.y;
  s.index = blockIdx.x;
  src += s.row * a.src_stride;
  dst += s.row * a.dst_stride;
  s.first = s.index * a.slice;
  s.stop = min(s.first + a.slice, a.vocab);
  const uint32_t lead = lead_of(src);
  s.grouped = lead == lead_of(dst);
  s.base = s.first + (s.grouped ? lead : 0u);
  return s;
}

// Four entries a lane of a list of tokens: which of them belong to the slice, at
// which place, and which were generated.
struct Four {
  bool in[4], made[4];
  uint32_t u[4];
};

// Calls f(four) for the history, a warp's lanes together. Calls in which no lane has
// an entry of the slice are left out: with a dozen slices a row that is most of
// them. Tokens outside the vocabulary are recorded.
template <typename F>
__device__ __forceinline__ void scan_tokens(const LogitsArgs& a, const Slice& s, const RowSettings& row, F f) {
  const int32_t* p = row.tokens;
  const uint32_t n = row.history, made = row.made;
  const uint32_t len = s.stop - s.first, off = s.first - s.base + 8u;
  uint32_t bad = 0u;
  auto four = [&](const int4& t, uint32_t i, bool have) {
    const uint32_t v[4] = {uint32_t(t.x), uint32_t(t.y), uint32_t(t.z), uint32_t(t.w)};
    Four x;
    bool any = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x.in[k] = have && v[k] - s.first < len;
      x.made[k] = i + k >= made;
      x.u[k] = v[k] - s.first + off;
      bad |= have && v[k] >= a.vocab;
      any |= x.in[k];
    }
    if (__any_sync(0xFFFFFFFFu, any)) f(x);
  };
  const uint32_t lead = min(n, (0u - uint32_t(reinterpret_cast<uintptr_t>(p) / 4u)) & 3u);
  const uint32_t quads = (n - lead) / 4u, rest = lead + 4u * quads;
  const int4* quad = reinterpret_cast<const int4*>(p + lead);
  const int4 none = make_int4(-1, -1, -1, -1);
  uint32_t at = threadIdx.x;
  int4 next = at < quads ? quad[at] : none;
  for (uint32_t q = threadIdx.x & ~31u; q < quads; q += kThreads, at += kThreads) {
    const int4 t = next;
    next = at + kThreads < quads ? quad[at + kThreads] : none;
    four(t, lead + 4u * at, at < quads);
  }
  // up to 3 entries in front of the aligned ones and 3 behind, one a lane of the first warp
  if (threadIdx.x < 32u) {
    const uint32_t i = threadIdx.x < lead ? threadIdx.x : rest + (threadIdx.x - lead);
    const uint32_t t = i < n ? uint32_t(p[i]) : 0xFFFFFFFFu;
    bad |= i < n && t >= a.vocab;
    Four x{};
    x.in[0] = t - s.first < len;
    x.made[0] = i >= made;
    x.u[0] = t - s.first + off;
    f(x);
  }
  if (bad) record_error(a.error_word, kErrIndex);
}

// ---- histories sorted by slice
//
// Every slice of a row reads the row's whole history, which for long histories is
// most of the work. With enough of it the token list is therefore sorted first:
// block by block of kBlock tokens, the tokens of one slice side by side. A slice
// then reads its own part of the blocks its history touches. The sorting of 1.3
// million tokens takes 8 us, its waits one after the other. The next kernel starts
// under it, but reads nothing before its own wait: that the sorting has waited for
// what is in front of it makes those writes visible to the sorting alone.
// entries: place in the slice's vocabulary | position in the block << 16; offs:
// for every block, where each slice's entries begin (slices + 2 words; the slice
// past the last holds tokens outside the vocabulary).
__global__ void __launch_bounds__(256) sort_kernel(const int32_t* tokens, uint64_t ntokens, uint32_t vocab,
                                                   uint32_t slice, uint32_t slices, uint32_t* entries,
                                                   uint16_t* offs) {
  __shared__ uint32_t count[256];
  __shared__ uint32_t begin[256];
  constexpr int kEach = kBlock / 256;
  const uint64_t base = uint64_t(blockIdx.x) * kBlock;
  // the kernel that reads the entries may start: it clears its tables, then waits
  stream_ready();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  count[threadIdx.x] = 0u;
  uint32_t token[kEach], bucket[kEach], place[kEach] = {};
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const uint64_t i = base + threadIdx.x + 256 * k;
    token[k] = i < ntokens ? uint32_t(tokens[i]) : 0xFFFFFFFFu;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    bucket[k] = token[k] < vocab ? token[k] / slice : slices;
    token[k] -= token[k] < vocab ? bucket[k] * slice : token[k];
    // frequent tokens have low numbers: most lanes may want the same count
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, bucket[k]), first = __ffs(same) - 1;
    if ((threadIdx.x & 31u) == first) place[k] = atomicAdd(count + bucket[k], uint32_t(__popc(same)));
    place[k] = __shfl_sync(0xFFFFFFFFu, place[k], int(first)) + __popc(same & lanemask_lt());
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t sum = 0u;
    for (uint32_t w = 0; w < slices + 2u; w += 32) {
      const uint32_t own = count[w + threadIdx.x];
      uint32_t x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (threadIdx.x >= uint32_t(o)) x += y;
      }
      begin[w + threadIdx.x] = sum + x - own;
      sum += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
  }
  __syncthreads();
  if (threadIdx.x < slices + 2u) offs[uint64_t(blockIdx.x) * (slices + 2u) + threadIdx.x] = uint16_t(begin[threadIdx.x]);
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    entries[base + begin[bucket[k]] + place[k]] = token[k] | ((threadIdx.x + 256u * k) << 16);
}

// As scan_tokens, of sorted tokens.
template <typename F>
__device__ __forceinline__ void scan_sorted(const LogitsArgs& a, const Slice& s, const RowSettings& row, F f) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, pitch = a.slices + 2u;
  const uint32_t blocks = (row.from + row.history + kBlock - 1u) / kBlock;
  // warps share a block where there are fewer blocks than warps
  constexpr uint32_t kWarps = kThreads / 32;
  const uint32_t share = blocks == 1u ? kWarps : blocks == 2u ? kWarps / 2u : blocks <= 4u ? kWarps / 4u : 1u;
  const uint32_t off = s.first - s.base + 8u, part = warp % share;
  uint32_t bad = 0u;
  for (uint32_t b = warp / share; b < blocks; b += kWarps / share) {
    const uint64_t block = uint64_t(row.block) + b;
    const uint16_t* o = a.sorted_offs + block * pitch + s.index;
    const uint32_t* e = a.sorted + block * kBlock;
    const uint32_t lo = o[0], hi = o[1];
    // the history's part of the block, and where its generated part starts
    const uint32_t from = b == 0u ? row.from : 0u, to = min(row.from + row.history - b * kBlock, kBlock);
    const uint32_t split = row.from + row.made, made = split > b * kBlock ? split - b * kBlock : 0u;
    if (s.index == 0u && part == 0u)  // tokens outside the vocabulary, among the row's
      for (uint32_t i = o[a.slices] + lane; i < o[a.slices + 1u]; i += 32u) bad |= (e[i] >> 16) - from < to - from;
    for (uint32_t i = lo + part * 128u; i < hi; i += share * 128u) {
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = i + lane + 32u * k < hi ? e[i + lane + 32u * k] : 0xFFFF0000u;
      Four x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t at = v[k] >> 16;
        x.in[k] = at - from < to - from;
        x.made[k] = at >= made;
        x.u[k] = (v[k] & 0xFFFFu) + off;
      }
      f(x);
    }
  }
  if (bad) record_error(a.error_word, kErrIndex);
}

template <typename F>
__device__ __forceinline__ void scan_history(const LogitsArgs& a, const Slice& s, const RowSettings& row, F f) {
  if (a.sorted)
    scan_sorted(a, s, row, f);
  else
    scan_tokens(a, s, row, f);
}

// Shared-memory reductions under a predicate; a branch for each would cost more
// than the rest of a scan.
__device__ __forceinline__ void add_if(bool p, uint32_t* at, uint32_t x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared::cta.add.u32 [%1], %2;\n\t}" ::"r"(uint32_t(p)),
               "r"(smem_addr(at)), "r"(x)
               : "memory");
}
__device__ __forceinline__ void or_if(bool p, uint32_t* at, uint32_t x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared::cta.or.b32 [%1], %2;\n\t}" ::"r"(uint32_t(p)),
               "r"(smem_addr(at)), "r"(x)
               : "memory");
}

__device__ __forceinline__ void prefetch_if(bool p, const void* at) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p prefetch.global.L2 [%1];\n\t}" ::"r"(uint32_t(p)),
               "l"(at));
}

// Sets the bits of the history. Where the tokens' elements of a second row are needed
// next, `near` is that row at place 0, and they are asked for here.
template <typename T = void>
__device__ __forceinline__ void mark_history(const LogitsArgs& a, const Slice& s, const RowSettings& row,
                                             uint32_t* bits, const T* near = nullptr) {
  scan_history(a, s, row, [&](const Four& x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (!std::is_void_v<T>) prefetch_if(x.in[k], near + x.u[k]);
      or_if(x.in[k], bits + (x.u[k] >> 5), 1u << (x.u[k] & 31u));
    }
  });
}

// The slice's mask words, copied to shared memory while other things go on;
// mask_ready() before the barrier after which they are read.
__device__ __forceinline__ void copy_mask(const uint32_t* mask, const Slice& s, uint32_t* words) {
  if (mask == nullptr) return;
  const uint32_t n = (s.stop - s.first + 31u) / 32u;
  for (uint32_t i = threadIdx.x; i < n; i += kThreads)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(words + i)), "l"(mask + s.first / 32u + i)
                 : "memory");
}
__device__ __forceinline__ void mask_ready() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The bits of the 8 tokens from t on, a group that ends inside the slice.
__device__ __forceinline__ uint32_t mask_bits8(const uint32_t* words, const Slice& s, uint32_t t) {
  const uint32_t i = t - s.first;
  return __funnelshift_r(words[i >> 5], words[(i + 7u) >> 5], i & 31u) & 0xFFu;
}

// This thread's groups of a slice.
template <typename TSrc>
struct Groups {
  Raw<TSrc> x[kGroups];
  uint32_t count;  // of the slice

  __device__ __forceinline__ void load(const Slice& s, const TSrc* src) {
    count = s.grouped && s.stop > s.base ? (s.stop - s.base) / 8u : 0u;
    const TSrc* p = src + s.base + 8u * threadIdx.x;
#pragma unroll
    for (int r = 0; r < kGroups; ++r)
      if (threadIdx.x + r * kThreads < count) load_group(p + r * kRound, x[r]);
  }
};

// Calls f(true type) for a slice without a mask whose threads all have a group in
// every round but the last, else f(false type): f leaves out the checks.
template <typename F>
__device__ __forceinline__ void rounds(uint32_t groups, const uint32_t* mask, F f) {
  if (mask == nullptr && groups >= (kGroups - 1) * uint32_t(kThreads))
    f(std::true_type{});
  else
    f(std::false_type{});
}
template <bool PLAIN>
__device__ __forceinline__ bool in_round(int r, uint32_t groups) {
  return (PLAIN && r < kGroups - 1) || threadIdx.x + r * kThreads < groups;
}

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

__device__ __forceinline__ bool open_token(const uint32_t* mask, const uint32_t* words, const Slice& s, uint32_t t) {
  return mask == nullptr || ((words[(t - s.first) >> 5] >> (t & 31u)) & 1u);
}

constexpr float kClosed = -__builtin_huge_valf();

// Repetition penalty and temperature alone: a bit a token is all there is to keep.
//   y = (seen ? x * (x > 0 ? 1/r : r) : x) * (1/T), -inf where the mask is closed
// Bound by memory where rows are many: 3,001 FP32 rows of 32,003 with up to 3,001
// tokens before each take 113 us, 6.8 TB/s.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas<TIn>) scale_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t bits[kWords], open[kWords];
  __shared__ RowSettings row;
  const TIn* src = static_cast<const TIn*>(a.src);
  TOut* dst = static_cast<TOut*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const bool history = a.tokens && a.repetition;
  if (s.row >= a.rows) return;
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) bits[i] = 0u;
  stream_ready();
  Groups<TIn> g;
  g.load(s, src);
  read_row(a, s.row, history, row);
  __syncthreads();
  const uint32_t* mask = row.mask;
  copy_mask(mask, s, open);
  if (row.history) mark_history(a, s, row, bits);
  mask_ready();
  __syncthreads();
  const float inv_t = row.inv_t, rep = row.rep, inv_rep = row.inv_rep;
  TOut* out = dst + s.base + 8u * threadIdx.x;
  auto seen = [&](float x) { return __fmul_rn(__fmul_rn(x, x > 0.0f ? inv_rep : rep), inv_t); };
  rounds(g.count, mask, [&](auto plain) {
    constexpr bool kPlain = decltype(plain)::value;
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      if (!in_round<kPlain>(r, g.count)) continue;
      const uint32_t q = threadIdx.x + r * kThreads;
      const uint32_t hit = reinterpret_cast<const uint8_t*>(bits)[q + 1u];
      float x[8], y[8];
      values(g.x[r], x);
      scale8(x, inv_t, y);
      if (hit) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = (hit >> k) & 1u ? seen(x[k]) : y[k];
      }
      store_masked(out + r * kRound, y, !kPlain && mask ? mask_bits8(open, s, s.base + 8u * q) : 0xFFu, kClosed);
    }
  });
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = kClosed;
    if (open_token(mask, open, s, t)) {
      const float x = load_elem(src + t);
      y = (bits[u >> 5] >> (u & 31u)) & 1u ? seen(x) : __fmul_rn(x, inv_t);
    }
    store_elem(dst + t, y);
  });
}

// Everything: tokens are counted and biased.
//   y = (p(x) - f * n - (n > 0 ? presence : 0) + b) * (1/T), p(x) as above, n the times
//   that the token was generated, -inf where the mask is closed
// A word a place is zeroed for all logits and read for groups of 8 with a token that a
// list names (1,024 rows with up to 64 tokens each: 95 us, 8 more when all were read).
// Zeroing the named ones alone took a second pass over the history and a third barrier,
// and was slower everywhere. Instructions and the waits between the barriers bound this
// kernel (issue slots 47 %, DRAM 21 %): 256 BF16 rows of 128,256 with histories up to
// 8,192, 100 biases and half of the rows masked take 52 us, 27 us with up to 64 tokens
// and neither biases nor masks, where the logits alone would move in 20.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas<TIn>) shape_kernel(const __grid_constant__ LogitsArgs a) {
  // a word a place: the times that the token was generated; where its bit in `final`
  // is set, the logit with penalties and bias. `used`: the tokens of the history
  __shared__ __align__(16) uint32_t word[kPlaces];
  __shared__ uint32_t used[kWords], final[kWords], open[kWords];
  __shared__ uint32_t twice;  // a token of the bias list is listed twice
  __shared__ RowSettings row;
  const TIn* src = static_cast<const TIn*>(a.src);
  TOut* dst = static_cast<TOut*>(a.dst);
  const Slice s = slice_of(a, src, dst);
  const bool history = a.tokens && (a.repetition || a.presence || a.frequency);
  if (s.row >= a.rows) return;
  if (threadIdx.x == 0) twice = 0u;
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) final[i] = used[i] = 0u;
  for (uint32_t i = threadIdx.x; i < (a.slice + 8u + 3u) / 4u; i += kThreads)
    reinterpret_cast<uint4*>(word)[i] = make_uint4(0u, 0u, 0u, 0u);
  stream_ready();
  Groups<TIn> g;
  g.load(s, src);
  read_row(a, s.row, history, row);
  __syncthreads();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t* mask = row.mask;
  copy_mask(mask, s, open);
  // A bias list of at most an entry a thread is read here, with the logit and the
  // value that an entry in the slice needs; bits in `final` claim its tokens. A token
  // listed twice is met there and sends the whole list the slow way, which longer
  // lists go anyhow. (256 rows of 128,256 with 100 biases each: 59 us when every
  // list went the slow way, 54 us so, 56 us with two entries a thread.)
  const uint32_t biased = row.biased, len = s.stop - s.first, off = s.first - s.base + 8u;
  const bool quick = biased <= uint32_t(kThreads);
  uint32_t mine = 0u;  // place of this thread's entry, 0: none
  float logit, value;
  if (quick && threadIdx.x < biased) {
    const uint32_t t = uint32_t(row.bias_tokens[threadIdx.x]);
    if (t - s.first < len) {
      mine = t - s.first + off;
      logit = load_elem(src + t);
      value = row.bias_values[threadIdx.x];
      const uint32_t bit = 1u << (mine & 31u);
      if (atomicOr(final + (mine >> 5), bit) & bit) twice = 1u;
    } else if (t >= a.vocab) {
      record_error(a.error_word, kErrIndex);
    }
  }
  const float rep = row.rep, inv_rep = row.inv_rep, freq = row.freq, pres = row.pres, inv_t = row.inv_t;
  auto penalized = [&](float x, uint32_t made) {
    x = __fmul_rn(x, x > 0.0f ? inv_rep : rep);
    return made == 0u ? x : __fsub_rn(__fsub_rn(x, __fmul_rn(freq, float(made))), pres);
  };
  auto seen = [&](uint32_t u) { return (used[u >> 5] >> (u & 31u)) & 1u; };
  if (row.history) {
    scan_history(a, s, row, [&](const Four& x) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        add_if(x.in[k] && x.made[k], word + x.u[k], 1u);
        or_if(x.in[k], used + (x.u[k] >> 5), 1u << (x.u[k] & 31u));
      }
    });
  }
  if (biased) {
    __syncthreads();
    if (quick && !twice) {
      if (mine) word[mine] = __float_as_uint(__fadd_rn(seen(mine) ? penalized(logit, word[mine]) : logit, value));
    } else {
      // Every warp reads the list backwards, 32 entries at a time, and serves the
      // places that are its own: the last entry of a token comes first, and its bit
      // turns the others away.
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) final[i] = 0u;
      __syncthreads();
      for (uint32_t back = lane; back - lane < biased; back += 32u) {
        const uint32_t i = biased - 1u - back;
        const uint32_t t = back < biased ? uint32_t(row.bias_tokens[i]) : 0xFFFFFFFFu, u = t - s.first + off;
        if (back < biased && t >= a.vocab) record_error(a.error_word, kErrIndex);
        const bool own = t - s.first < len && u * (kThreads / 32u) / kPlaces == warp;
        const uint32_t owners = __ballot_sync(0xFFFFFFFFu, own);
        if (!own) continue;
        const uint32_t same = __match_any_sync(owners, u), bit = 1u << (u & 31u);
        if (lane != uint32_t(__ffs(same) - 1)) continue;  // a lane with a later entry
        if (atomicOr(final + (u >> 5), bit) & bit) continue;
        const float x = load_elem(src + (s.base + u - 8u));
        word[u] = __float_as_uint(__fadd_rn(seen(u) ? penalized(x, word[u]) : x, row.bias_values[i]));
      }
    }
  }
  mask_ready();
  __syncthreads();
  TOut* out = dst + s.base + 8u * threadIdx.x;
  rounds(g.count, mask, [&](auto plain) {
    constexpr bool kPlain = decltype(plain)::value;
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      if (!in_round<kPlain>(r, g.count)) continue;
      const uint32_t q = threadIdx.x + r * kThreads;
      float x[8];
      values(g.x[r], x);
      const uint32_t fin = reinterpret_cast<const uint8_t*>(final)[q + 1u];
      const uint32_t hit = reinterpret_cast<const uint8_t*>(used)[q + 1u];
      if (fin | hit) {
        const uint4 lo = reinterpret_cast<const uint4*>(word)[2u * q + 2u];
        const uint4 hi = reinterpret_cast<const uint4*>(word)[2u * q + 3u];
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if ((hit >> k) & 1u) x[k] = penalized(x[k], w[k]);
        }
        if (fin) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = (fin >> k) & 1u ? __uint_as_float(w[k]) : x[k];
        }
      }
      scale8(x, inv_t, x);
      store_masked(out + r * kRound, x, !kPlain && mask ? mask_bits8(open, s, s.base + 8u * q) : 0xFFu, kClosed);
    }
  });
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = kClosed;
    if (open_token(mask, open, s, t)) {
      float x = load_elem(src + t);
      if ((final[u >> 5] >> (u & 31u)) & 1u)
        x = __uint_as_float(word[u]);
      else if (seen(u))
        x = penalized(x, word[u]);
      y = __fmul_rn(x, inv_t);
    }
    store_elem(dst + t, y);
  });
}

// Backward: a bit a token of the history, and the raw logits of groups that have one.
//   dx = open ? dy * (1/T) * (seen ? (x > 0 ? 1/r : r) : 1) : 0
// (counts and biases are added, so they leave the gradient alone). Raw logits are read
// only where a token was seen, asked for while it is marked (7 us less in the case below).
// 4,096 BF16 rows of 151,936 with up to 4,096 tokens before each: 455 us, 5.5 TB/s;
// 376 us, 6.7 TB/s, with 64 tokens, so what bounds it is the waits for the history.
template <typename TIn, typename TOut>
__global__ void __launch_bounds__(kThreads, kMinCtas<TOut>) backward_kernel(const __grid_constant__ LogitsArgs a) {
  __shared__ uint32_t bits[kWords], open[kWords];
  __shared__ RowSettings row;
  const TOut* src = static_cast<const TOut*>(a.src);
  TIn* dst = static_cast<TIn*>(a.dst);
  Slice s = slice_of(a, src, dst);
  const bool history = a.tokens && a.repetition;
  if (s.row >= a.rows) return;
  for (uint32_t i = threadIdx.x; i < kWords; i += kThreads) bits[i] = 0u;
  stream_ready();
  const TIn* raw = static_cast<const TIn*>(a.raw) + (a.raw ? s.row * a.raw_stride : 0u);
  if (a.raw && lead_of(raw) != lead_of(src)) s.grouped = false;  // places stay as they are
  Groups<TOut> g;
  g.load(s, src);
  read_row(a, s.row, history, row);
  __syncthreads();
  const uint32_t* mask = row.mask;
  copy_mask(mask, s, open);
  if (row.history) mark_history(a, s, row, bits, raw + int64_t(s.base) - 8);
  mask_ready();
  __syncthreads();
  const float inv_t = row.inv_t, rep = row.rep, inv_rep = row.inv_rep;
  const TIn* near = raw + s.base + 8u * threadIdx.x;
  TIn* out = dst + s.base + 8u * threadIdx.x;
  rounds(g.count, mask, [&](auto plain) {
    constexpr bool kPlain = decltype(plain)::value;
    Raw<TIn> x[kGroups];
    uint32_t hit[kGroups];  // open tokens of the history
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      const uint32_t q = threadIdx.x + r * kThreads;
      hit[r] = in_round<kPlain>(r, g.count) ? reinterpret_cast<const uint8_t*>(bits)[q + 1u] : 0u;
      if (!kPlain && hit[r] && mask) hit[r] &= mask_bits8(open, s, s.base + 8u * q);
      if (hit[r]) load_group(near + r * kRound, x[r]);
    }
#pragma unroll
    for (int r = 0; r < kGroups; ++r) {
      if (!in_round<kPlain>(r, g.count)) continue;
      float d[8];
      values(g.x[r], d);
      scale8(d, inv_t, d);
      if (hit[r]) {
        float v[8];
        values(x[r], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = (hit[r] >> k) & 1u ? __fmul_rn(d[k], v[k] > 0.0f ? inv_rep : rep) : d[k];
      }
      const uint32_t t = s.base + 8u * (threadIdx.x + r * kThreads);
      store_masked(out + r * kRound, d, !kPlain && mask ? mask_bits8(open, s, t) : 0xFFu, 0.0f);
    }
  });
  each_single(s, g.count, [&](uint32_t t) {
    const uint32_t u = t - s.base + 8u;
    float y = 0.0f;
    if (open_token(mask, open, s, t)) {
      y = __fmul_rn(load_elem(src + t), inv_t);
      if ((bits[u >> 5] >> (u & 31u)) & 1u) y = __fmul_rn(y, load_elem(raw + t) > 0.0f ? inv_rep : rep);
    }
    store_elem(dst + t, y);
  });
}

dim3 grid_of(const LogitsArgs& a) {
  return dim3(a.slices, unsigned(a.rows < kRowsY ? a.rows : kRowsY), unsigned((a.rows + kRowsY - 1) / kRowsY));
}

template <typename K>
cudaError_t launch(K kernel, const LogitsArgs& a, cudaStream_t stream) {
  return launch_early(kernel, grid_of(a), kThreads, stream, a);
}

}  // namespace

// Counter words for calls on a stream that has none and is being captured, where
// nothing can be allocated.
__device__ uint32_t g_capture_counters[64];

uint32_t* logits_capture_counters() {
  void* p = nullptr;
  return cudaGetSymbolAddress(&p, g_capture_counters) == cudaSuccess ? static_cast<uint32_t*>(p) : nullptr;
}

// Slices of a row: as few as possible, since every one reads the history, but
// more where there are too few rows to give every SM two CTAs.
void logits_cut(LogitsArgs& a, int sms) {
  uint32_t k = (a.vocab + kSliceMax - 1) / kSliceMax, unit = kRound;
  while (a.rows * k < uint64_t(sms) * 2 && a.vocab / (2 * k) >= kSliceMin) k *= 2, unit = 32u;
  a.slice = ((a.vocab + k - 1) / k + unit - 1) / unit * unit;
  a.slices = (a.vocab + a.slice - 1) / a.slice;
}

// Sorting costs a launch and 6 us a million tokens and saves a slice the tokens of the
// others, but adds a wait (offsets, then entries), so it needs many tokens and several
// waves of slices. What the rows read of the token list is known on the device only;
// two bounds stand for it: the list read once by each slice, and, for a list that rows
// share, up to a token more with each row. Times unsorted and sorted, in us, of BF16
// rows of 128,256 with a quarter to all of the given history: 64 rows of 32,768 31, 36;
// 128 of 8,192 24, 27; 128 of 32,768 52, 48; 256 of 2,048 34, 35; 256 of 8,192 46, 45;
// 256 of 32,768 94, 78; 512 of 2,048 62, 63; 512 of 8,192 86, 81; 1,024 of 8,192 164, 153.
// Rows of one sequence: gradients of 1,024 104, 109, of 2,048 213, 215, of 4,096 467,
// 453. The list should also be small
// next to the rows, as it is all sorted, used or not.
bool logits_sorts(const LogitsArgs& a, int sms) {
  const uint64_t n = uint64_t(a.ntokens), ctas = a.rows * a.slices;
  if (a.slices < 2 || a.slices > kSortSlices || ctas < uint64_t(sms) * 10 || n > a.rows * a.vocab / 4) return false;
  return n * a.slices >= (1u << 24) || ctas * (n < a.rows ? n : a.rows) >= (1u << 27);
}
uint64_t logits_sort_blocks(const LogitsArgs& a) { return (uint64_t(a.ntokens) + kBlock - 1) / kBlock; }
uint64_t logits_sort_entries(const LogitsArgs& a) { return logits_sort_blocks(a) * kBlock; }
uint64_t logits_sort_offs(const LogitsArgs& a) { return logits_sort_blocks(a) * (a.slices + 2); }

cudaError_t launch_logits_sort(const LogitsArgs& a, uint32_t* entries, uint16_t* offs, cudaStream_t stream) {
  return launch_early(sort_kernel, dim3(unsigned(logits_sort_blocks(a))), 256, stream, a.tokens, uint64_t(a.ntokens),
                      a.vocab, a.slice, a.slices, entries, offs);
}

cudaError_t launch_logits_shape(const LogitsArgs& a, int in_type, int out_type, cudaStream_t stream) {
  if (a.bias_tokens || (a.tokens && (a.presence || a.frequency))) {
    if (in_type == PULSE_F32) return launch(shape_kernel<float, float>, a, stream);
    if (out_type == PULSE_F32) return launch(shape_kernel<uint16_t, float>, a, stream);
    return launch(shape_kernel<uint16_t, uint16_t>, a, stream);
  }
  if (in_type == PULSE_F32) return launch(scale_kernel<float, float>, a, stream);
  if (out_type == PULSE_F32) return launch(scale_kernel<uint16_t, float>, a, stream);
  return launch(scale_kernel<uint16_t, uint16_t>, a, stream);
}

cudaError_t launch_logits_backward(const LogitsArgs& a, int in_type, int out_type, cudaStream_t stream) {
  if (in_type == PULSE_F32) return launch(backward_kernel<float, float>, a, stream);
  if (out_type == PULSE_F32) return launch(backward_kernel<uint16_t, float>, a, stream);
  return launch(backward_kernel<uint16_t, uint16_t>, a, stream);
}

}  // namespace pulse
