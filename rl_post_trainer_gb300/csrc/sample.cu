// sample.cu -- a token a row from a given uniform number, under temperature, top-k, top-p
// and min-p, and its log-probability.
//
// Mathematics. Weights w = exp((x - max) / T) are whole multiples of 2^-S (S = 47, less for
// a vocabulary past 2^15, so that a row's sum stays below 2^62): sums do not depend on their
// order, no atomic changes a result, and "the first token whose running sum passes u times
// the total" has one answer. That answer has to be the real one: with u uniform, a token is
// wrong with a probability of about the tokens of weight times the error of a sum, so errors
// of FP32's exponential (2^-22) would show once in some hundred rows of a flat
// distribution. exp_fixed has 2^-44.
//
// Top-k, the nucleus and the draw are one search: the place where a running sum (of ones,
// or of weights) over tokens in a given order (falling logits, or rising tokens) reaches a
// target. It goes 9 bits of the order's key at a time, with a histogram of the sums.
//
// A row is read once: a cluster of CTAs holds it in shared memory, a slice each. What the
// cut needs is seldom more than a few hundred tokens: those above a bound that is known to lie
// below the cut go to a list in the first CTA, which ends the row alone. The bound is, for top-k,
// the k / CTAs-th largest of the threads' own maxima in each CTA, the least of them; for top-p
// the weight of which the whole vocabulary would make up the part that is left out. A row
// whose list runs over is searched by all CTAs of the cluster in their slices, and one
// without top-k and top-p by sums of warps.
//
// Sums over whole rows are taken in FP32 first, with a bound of their error. Where that leaves
// more than one answer (a number within 2^-18 of the total from a border between two tokens, a
// nucleus whose last token it could change) they are taken again with exp_fixed, ten times the work.
//
// Measured (us; top-k 50, no cut, top-p 0.9 of a flat row, whose nucleus are tens of thousands of tokens, greedy): a row of 151936
// FP32 10, 8, 33, 6; 256 rows of 128256 BF16 57, 79, 255, 40 (the bytes alone 10); 2001 rows of 32003 FP32 169, 161, 432, 118 (the
// bytes alone 38). Not memory bounds it (13 % of DRAM's cycles with top-k) but the chain of a CTA: load, largest, bound, list, search or
// draw, each behind a barrier of the cluster; with a cut in a flat row the instructions of exp_fixed.
#include <atomic>
#include <type_traits>

#include "pulse.h"
#include "pulse_device.cuh"
#include "pulse_internal.h"
#include "slice_edges.h"

namespace pulse {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBits = 9, kBins = 1 << kBits;
static_assert(kBins == 2 * kThreads, "two bins a thread");
constexpr uint32_t kList = 1536;                  // tokens of a list
// Wanted of a slice: four CTAs per SM. 256 rows of 128256 BF16, us with 16, 32, 64 KB when this was chosen: top-k 50 92, 55, 55;
// no cut 121, 104, 129; top-p 0.9 390, 293, 363. 2001 rows of 32003 FP32, no cut: 258, 192, 214.
constexpr uint32_t kSliceBytes = 32 * 1024;
constexpr uint32_t kSliceMost = 180 * 1024;       // more than that stays in global memory
constexpr uint32_t kCtas = 16;                    // of a cluster
constexpr float kLeastT = 0x1p-127f;              // log2(e) over less is no FP32 number

// 2^(j / 64) * 2^47, rounded to nearest
__device__ const unsigned long long kExp2[64] = {
    0x800000000000ull, 0x8164D1F3BC03ull, 0x82CD8698AC2Cull, 0x843A28C3ACDEull, 0x85AAC367CC48ull, 0x871F61969E8Dull,
    0x88980E8092DBull, 0x8A14D575496Full, 0x8B95C1E3EA8Cull, 0x8D1ADF5B7E5Cull, 0x8EA4398B45CDull, 0x9031DC431467ull,
    0x91C3D373AB12ull, 0x935A2B2F13E7ull, 0x94F4EFA8FEF7ull, 0x96942D372018ull, 0x9837F0518DB9ull, 0x99E0459320B8ull,
    0x9B8D39B9D54Eull, 0x9D3ED9A72D00ull, 0x9EF5326091A1ull, 0xA0B0510FB971ull, 0xA27043030C49ull, 0xA43515AE09E7ull,
    0xA5FED6A9B151ull, 0xA7CD93B4E965ull, 0xA9A15AB4EA7Cull, 0xAB7A39B5A93Full, 0xAD583EEA42A1ull, 0xAF3B78AD690Aull,
    0xB123F581D2ACull, 0xB311C412A911ull, 0xB504F333F9DEull, 0xB6FD91E328D1ull, 0xB8FBAF4762FCull, 0xBAFF5AB2133Eull,
    0xBD08A39F580Cull, 0xBF1799B67A73ull, 0xC12C4CCA6671ull, 0xC346CCDA2497ull, 0xC5672A115507ull, 0xC78D74C8ABBAull,
    0xC9B9BD866E2Full, 0xCBEC14FEF272ull, 0xCE248C151F85ull, 0xD06333DAEF2Bull, 0xD2A81D91F12Bull, 0xD4F35AABCFEEull,
    0xD744FCCAD69Dull, 0xD99D15C278B0ull, 0xDBFBB797DAF2ull, 0xDE60F4825E0Full, 0xE0CCDEEC2A95ull, 0xE33F8972BE8Aull,
    0xE5B906E77C83ull, 0xE8396A503C4Cull, 0xEAC0C6E7DD24ull, 0xED4F301ED994ull, 0xEFE4B99BDCDBull, 0xF281773C5A00ull,
    0xF5257D152487ull, 0xF7D0DF730AD1ull, 0xFA83B2DB722Aull, 0xFD3E0C0CF487ull,
};
constexpr float kLn2Hi = 0x1.62e430p-1f, kLn2Lo = -0x1.05c610p-29f;
constexpr float kLog2EHi = 0x1.715476p+0f, kLog2ELo = 0x1.4ae0c0p-26f;

__device__ __forceinline__ float lowest() { return __uint_as_float(0xFF800000u); }

struct Row {
  float top;       // the largest logit
  float ch, cl;    // log2(e) / T as a sum
  int scale;       // S
  float c0;        // exp_fast: x ch + c0 = (x - top) ch
  float unit;      // what a sum of exp_fast is in multiples of 2^-S
  bool plain;      // exp_fast may be used: nothing passes its range, and 2^-S is small against its errors
};

// -0 to +0, NaN to -infinity
__device__ __forceinline__ float plain(float x) { return x == x ? x + 0.0f : lowest(); }

// Unsigned numbers in the order of the floats, and back. Of a BF16 logit the upper 16 bits are the key.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
template <typename T>
struct Keys {  // float
  static constexpr int kLow = 0;
  static __device__ uint32_t of(float x) { return key_of(x); }
  static __device__ float value(uint32_t k) { return of_key(k); }
};
template <>
struct Keys<uint16_t> {
  static constexpr int kLow = 16;
  static __device__ uint32_t of(float x) { return key_of(x) & 0xFFFF0000u; }
  static __device__ float value(uint32_t k) { return of_key(k >> 31 ? k : k | 0xFFFFu); }
};

// 2^S * exp((x - top) / T), rounded; 2^-44 off at most, relatively, and half a unit. The difference and
// its product with log2(e) / T are sums of two floats (Dekker, Knuth); 2^z = 2^n 2^(j/64) (1 + p)
// with |z - n - j/64| <= 1/128, the second factor from a table, p from the exponential's series.
// p goes into the table's entry in two parts: multiples of 2^-22 as a whole number, the rest (below
// 2^-22) as a float. No branch, so that several can be under way in a thread.
__device__ __forceinline__ uint64_t exp_fixed(float x, const Row& r, const unsigned long long* table) {
  const float d = __fsub_rn(x, r.top);
  const float zh = fmaxf(__fmul_rn(d, r.ch), -64.0f);  // NaN, of infinities, to -64
  const float b = __fsub_rn(d, x);
  const float dl = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(r.top, b));
  float zl = __fmaf_rn(d, r.ch, -zh);
  zl = __fmaf_rn(d, r.cl, zl);
  zl = __fmaf_rn(dl, r.ch, zl);
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, found in the low bits
  const float shifted = __fmaf_rn(zh, 64.0f, kRound);
  const int k = __float_as_int(shifted) - 0x4B400000;
  const float f = __fmaf_rn(__fsub_rn(shifted, kRound), -0.015625f, zh);
  const float a = __fmul_rn(f, kLn2Hi);
  float al = __fmaf_rn(f, kLn2Hi, -a);
  al = __fmaf_rn(f, kLn2Lo, al);
  al = __fmaf_rn(zl, kLn2Hi, al);
  const float half = __fmul_rn(0.5f, a), q = __fmul_rn(half, a);
  float rest = __fmaf_rn(half, a, -q);
  rest = __fmaf_rn(a, al, rest);
  rest = __fmaf_rn(__fmul_rn(a, q), __fmaf_rn(a, 1.0f / 12.0f, 1.0f / 3.0f), rest);  // a^3 / 6 + a^4 / 24
  const float s = __fadd_rn(a, q);
  rest = __fadd_rn(rest, __fadd_rn(al, __fsub_rn(q, __fsub_rn(s, a))));
  const float big = __fmaf_rn(s, 4194304.0f, kRound);
  const int h = __float_as_int(big) - 0x4B400000;  // s in multiples of 2^-22
  rest = __fadd_rn(rest, __fmaf_rn(__fsub_rn(big, kRound), -0x1p-22f, s));
  const int64_t t = int64_t(table[k & 63]);
  const float tf = __uint_as_float(0x3F800000u | (uint32_t(uint64_t(t) >> 24) & 0x7FFFFFu));  // the entry as a float in [1, 2)
  const uint64_t w = uint64_t(t + ((t * h) >> 22) + __float2int_rn(__fmul_rn(rest, tf) * 0x1p47f));
  const int shift = 47 - r.scale - (k >> 6);  // at most 64 + 47 - S
  const uint64_t v = shift > 0 ? ((w >> (shift - 1)) + 1) >> 1 : w;
  return x == r.top ? 1ull << r.scale : zh > -float(r.scale + 2) ? v : 0;
}

__device__ __forceinline__ float ex2(float z) {
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(z));
  return w;
}
// exp((x - top) / T) in FP32, times a factor near 1 that Row::unit takes out (c0 is rounded). Off by
// 2^-22 for the exponential and |z| 2^-23 ln 2 for the exponent z. NaN and -infinity give 0.
__device__ __forceinline__ float exp_fast(float x, const Row& r) { return ex2(fmaxf(__fmaf_rn(x, r.ch, r.c0), -200.0f)); }
__device__ __forceinline__ uint64_t fixed_of(float w, const Row& r) { return uint64_t(__float2ll_rn(__fmul_rn(w, r.unit))); }

struct alignas(16) Shared {
  uint32_t low[2][kBins], high[2][kBins];  // histograms, halves of 64-bit sums; all zero but while in use
  unsigned long long part[kWarps], part2[kWarps];
  unsigned long long table[64];
  unsigned long long before, target, size;
  // what every CTA of the cluster has posted; sums in two sets in turn, since one may still be read
  unsigned long long sums[2][2][kCtas];
  uint32_t tops[kCtas], bounds[kCtas], firsts[kCtas], counts[kCtas];
  // the row's settings as the first CTA has read them: what the CTAs do together hangs on nothing else
  float t, p, u, min_p, ch, cl, down;
  uint32_t k;
  uint32_t sure, cut[3];
  uint32_t bin, end, crowd;
  uint32_t listed;                         // tokens of this CTA's list, or of the row's
  uint32_t keys[kList], tokens[kList];
};

// ------------------------------------------------------------------- clusters

struct Cluster {
  uint32_t size, rank;
  uint32_t turn;  // of the two histograms the next one: another CTA may still read the last one
  uint32_t flip;  // and of the two sets of sums
  __device__ void arrive() const {
    if (size > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  }
  __device__ void wait() const {
    if (size > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  }
  __device__ void sync() const {
    if (size == 1) {
      __syncthreads();
    } else {
      arrive();
      wait();
    }
  }
  // the address of a shared variable in CTA `r`
  template <typename V>
  __device__ uint32_t at(const V* p, uint32_t r) const {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(r));
    return a;
  }
  __device__ uint64_t load(const unsigned long long* p, uint32_t r) const {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at(p, r)) : "memory");
    return v;
  }
  __device__ void store(uint32_t* p, uint32_t r, uint32_t v) const {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at(p, r)), "r"(v) : "memory");
  }
  __device__ void store(float* p, uint32_t r, float v) const {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at(p, r)), "f"(v) : "memory");
  }
  __device__ void store(unsigned long long* p, uint32_t r, uint64_t v) const {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at(p, r)), "l"(v) : "memory");
  }
  // A CTA's value to all CTAs (the first warp does this); there after the next sync().
  template <typename V>
  __device__ void post(V* p, V v) const {
    if (threadIdx.x < size) store(&p[rank], threadIdx.x, v);
  }
};

// ------------------------------------------------------------- sums of a CTA

__device__ __forceinline__ uint64_t warp_up(uint64_t v) {  // running sum over the lanes
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if ((threadIdx.x & 31u) >= unsigned(d)) v += o;
  }
  return v;
}
// Of a warp, in all lanes: three parts of 22, 22 and 20 bits, whose sums of 32 fit into 32.
__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
  const uint32_t a = __reduce_add_sync(0xFFFFFFFFu, uint32_t(v) & 0x3FFFFFu), b = __reduce_add_sync(0xFFFFFFFFu, uint32_t(v >> 22) & 0x3FFFFFu),
                 c = __reduce_add_sync(0xFFFFFFFFu, uint32_t(v >> 44));
  return uint64_t(a) + (uint64_t(b) << 22) + (uint64_t(c) << 44);
}
// Of all threads, in all threads; sh.part holds the sums of the warps then. Both ends are barriers.
__device__ __forceinline__ uint64_t sum_of(uint64_t v, Shared& sh) {
  v = warp_total(v);
  __syncthreads();
  if ((threadIdx.x & 31u) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) v += sh.part[k];
  return v;
}
// Sums over all warps of `cluster`, b where kTwo; `front`: the first one over the warps in front of this one. Every CTA
// posts its own to all.
template <bool kTwo>
__device__ __forceinline__ void sums_of(uint64_t a, uint64_t b, Shared& sh, Cluster& cluster, uint64_t* a_out, uint64_t* b_out, uint64_t* front) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  a = warp_total(a);
  if (kTwo) b = warp_total(b);
  __syncthreads();
  if (lane == 0) {
    sh.part[warp] = a;
    if (kTwo) sh.part2[warp] = b;
  }
  __syncthreads();
  a = b = 0;
  uint64_t before = 0;
#pragma unroll
  for (uint32_t k = 0; k < kWarps; ++k) {
    if (k < warp) before += sh.part[k];
    a += sh.part[k];
    if (kTwo) b += sh.part2[k];
  }
  if (cluster.size > 1) {
    unsigned long long(&sums)[2][kCtas] = sh.sums[cluster.flip];
    cluster.flip ^= 1u;
    cluster.post(sums[0], static_cast<unsigned long long>(a));
    if (kTwo) cluster.post(sums[1], static_cast<unsigned long long>(b));
    cluster.sync();
    a = lane < cluster.size ? sums[0][lane] : 0;
    before += warp_total(lane < cluster.rank ? a : 0);
    a = warp_total(a);
    if (kTwo) b = warp_total(lane < cluster.size ? sums[1][lane] : 0);
  }
  *a_out = a, *front = before;
  if (kTwo) *b_out = b;
}
__device__ __forceinline__ uint32_t max_of(uint32_t v, Shared& sh) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31u) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) v = max(v, uint32_t(sh.part[k]));
  return v;
}

struct Found {
  uint64_t before, size;  // sums of the values before a key, and of it
};

// Over (key, value) pairs, keys in [low, high], in the order of falling keys: the key at which the
// running sum of the values reaches `target` (1 at least; the total where it is less). Of all CTAs of
// `cluster`. `least_bits`: low bits of the keys that are zero. kCount: the values are 1.
template <bool kCount, typename Each>
__device__ uint32_t search(Shared& sh, Cluster& cluster, uint32_t low, uint32_t high, int least_bits, uint64_t target,
                           Found* found, Each each) {
  const int bits = 32 - __clz((high - low) | 1u);
  int shift = least_bits + (max(bits - least_bits, 1) + kBits - 1) / kBits * kBits;
  uint32_t prefix = 0, above = 0;  // of key - low; bits from `shift` on are known
  uint64_t before = 0;
  do {
    shift -= kBits;
    uint32_t *lo = sh.low[cluster.turn], *hi = sh.high[cluster.turn];
    cluster.turn ^= 1u;
    each([&](uint32_t key, auto value) {
      const uint32_t k = key - low;
      if ((k & above) != prefix) return;
      const uint32_t bin = (k >> shift) & (kBins - 1);
      if (kCount) {
        atomicAdd(&lo[bin], 1u);
      } else if (const uint64_t v = value()) {
        const uint32_t old = atomicAdd(&lo[bin], uint32_t(v));
        const uint32_t up = uint32_t(v >> 32) + (old + uint32_t(v) < old ? 1u : 0u);
        if (up) atomicAdd(&hi[bin], up);
      }
    });
    if (threadIdx.x == 0) sh.bin = 0, sh.before = before, sh.target = target, sh.size = 0;
    cluster.sync();
    // two bins a thread, the upper one first
    const uint32_t bin = kBins - 1 - 2 * threadIdx.x;
    uint64_t v[2] = {0, 0};
    if (cluster.size == 1) {
#pragma unroll
      for (uint32_t j = 0; j < 2; ++j) v[j] = lo[bin - j] | (kCount ? 0 : uint64_t(hi[bin - j]) << 32);
    } else {
      for (uint32_t r = 0; r < cluster.size; r += 8) {  // eight CTAs' bins bin - 1 and bin at once
        uint64_t l[8], h[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          l[j] = h[j] = 0;
          if (r + j < cluster.size) {
            l[j] = cluster.load(reinterpret_cast<const unsigned long long*>(&lo[bin - 1]), r + j);
            if (!kCount) h[j] = cluster.load(reinterpret_cast<const unsigned long long*>(&hi[bin - 1]), r + j);
          }
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
          v[0] += (l[j] >> 32) + ((h[j] >> 32) << 32);
          v[1] += uint32_t(l[j]) + (h[j] << 32);
        }
      }
    }
    // the other histogram, which no CTA reads any more, is the next one
    sh.low[cluster.turn][bin] = sh.low[cluster.turn][bin - 1] = 0;
    sh.high[cluster.turn][bin] = sh.high[cluster.turn][bin - 1] = 0;
    const uint64_t up = warp_up(v[0] + v[1]);
    if ((threadIdx.x & 31u) == 31u) sh.part[threadIdx.x >> 5] = up;
    __syncthreads();
    uint64_t total = before, at = before + up - v[0] - v[1];
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) {
      const uint64_t w = sh.part[k];
      total += w;
      if (k < (threadIdx.x >> 5)) at += w;
    }
    const uint64_t goal = target < total ? target : total;
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
      if (at < goal && goal <= at + v[j]) sh.bin = bin - j, sh.before = at, sh.target = goal, sh.size = v[j];
      at += v[j];
    }
    __syncthreads();
    before = sh.before;
    target = sh.target;
    prefix |= sh.bin << shift;
    above |= uint32_t(kBins - 1) << shift;
    *found = Found{before, sh.size};
    __syncthreads();
  } while (shift > least_bits);
  return low + prefix;
}

// The tokens up to a place in the order of falling logits (equal ones: rising tokens).
struct Cut {
  uint32_t key = 0, token = 0xFFFFFFFFu;
  __device__ bool keeps(uint32_t k, uint32_t t) const { return k > key || (k == key && t <= token); }
};

struct Settings {
  float t, p, u;
  int32_t k;
  // min-p: logits from `surely` on are kept, below `maybe` they are not, between the two the weight decides
  float maybe, surely;
  uint64_t least;  // weight
  __device__ bool keeps(float v, const Row& r, const unsigned long long* table) const {
    return v >= surely || (v >= maybe && exp_fixed(plain(v), r, table) >= least);
  }
};

// floor and ceiling of f * v, f in (0, 1)
__device__ __forceinline__ uint64_t part_of(float f, uint64_t v, bool up) {
  const uint64_t bits = __float2ull_rd(__fmul_rn(f, 18446744073709551616.0f));  // f * 2^64
  return __umul64hi(bits, v) + (up && bits * v != 0 ? 1u : 0u);
}
// Where u falls: a token's share begins at or before this sum and ends after it.
__device__ __forceinline__ uint64_t place_of(float u, uint64_t mass) {
  return !(u > 0.0f) ? 0 : u < 1.0f ? part_of(u, mass, false) : mass - 1;
}

// The first `room` of the `tied` tokens of `each` with that key that `within` keeps.
template <typename Each>
__device__ Cut tie_of(Shared& sh, Cluster& cluster, uint32_t vocab, uint32_t key, uint64_t room, uint64_t tied, const Cut& within, Each each) {
  Cut c;
  c.key = key;
  c.token = within.key == key ? within.token : 0xFFFFFFFFu;
  if (room < tied) {
    Found f;
    c.token = ~search<true>(sh, cluster, ~(vocab - 1), ~0u, 0, room, &f, [&](auto add) {
      each([&](uint32_t k, uint32_t i) { if (k == key && within.keeps(k, i)) add(~i, [] { return 1; }); });
    });
  }
  return c;
}

// The first s.k tokens of `each` (key, token), which hold at least those.
template <typename T, typename Each>
__device__ Cut top_k_of(Shared& sh, Cluster& cluster, const Settings& s, uint32_t vocab, uint32_t low, uint32_t high, Each each) {
  Found found;
  const uint32_t key = search<true>(sh, cluster, low, high, Keys<T>::kLow, uint64_t(s.k), &found, [&](auto add) {
    each([&](uint32_t k, uint32_t) { add(k, [] { return 1; }); });
  });
  return tie_of(sh, cluster, vocab, key, uint64_t(s.k) - found.before, found.size, Cut{}, each);
}

// Those of the tokens within `cut` in front of which less than s.p of `mass`, their sum, lies. `off`: what mass
// may be off by; false where that could move the cut. `front`: the sum of tokens that are likelier than all of `each`;
// false where the cut is not among those of `each`.
template <typename T, typename Each>
__device__ bool nucleus_of(Shared& sh, Cluster& cluster, const Settings& s, const Row& r, uint32_t vocab, uint32_t low, uint32_t high,
                           uint64_t mass, uint64_t off, uint64_t front, Cut* cut, Each each) {
  auto weight = [&](uint32_t key) { return exp_fixed(Keys<T>::value(key), r, sh.table); };
  const uint64_t share = s.p > 0.0f ? part_of(s.p, mass - off, true) : 0, goal = (share < 1 ? 1 : share) - front;
  if (int64_t(goal) <= 0) return false;
  Found found;
  const Cut within = *cut;
  const uint32_t key = search<false>(sh, cluster, low, high, Keys<T>::kLow, goal, &found, [&](auto add) {
    each([&](uint32_t k, uint32_t i) { if (within.keeps(k, i)) add(k, [&] { return weight(k); }); });
  });
  if (goal > found.before + found.size) return false;
  const uint64_t one = weight(key), tied = found.size / one, room = (goal - found.before + one - 1) / one;
  if (off && s.p > 0.0f) {
    const uint64_t most = part_of(s.p, mass + off, true) - front;
    if (most > found.before + found.size || (most - found.before + one - 1) / one != room) return false;
  }
  *cut = tie_of(sh, cluster, vocab, key, room, tied, within, each);
  return true;
}

// ---------------------------------------------------------------- a slice

__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4], const float*) {
  v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8], const uint16_t*) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
// The largest of 16 bytes of logits and `most`; NaN is passed over.
__device__ __forceinline__ float max_with(const uint4& q, float most, const float*) {
  return fmaxf(fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))), most);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
__device__ __forceinline__ float max_with(const uint4& q, float most, const uint16_t*) {
  const uint32_t m = max2(max2(q.x, q.y), max2(q.z, q.w));
  return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), most);
}

// Tokens [begin, begin + count) of a row in pieces of 16 bytes as they lie in memory: the first
// and the last piece may be cut off. Elements outside read as -infinity.
template <typename T, bool kResident>
struct Slice {
  static constexpr int kPiece = 16 / sizeof(T);
  const T* row;       // element 0 of the slice
  uint32_t begin, count, lead;  // lead: elements of the first piece in front of the slice
  uint32_t pieces;
  const uint4* kept;  // kResident: the pieces in shared memory

  // From global memory. A piece that is cut off is read whole, too, and what is not of the slice replaced, but for pieces that
  // leave the matrix's own range of addresses (slice_edges). Those are read
  // by elements, in a function of its own (inlined, it would be most of the kernel's code).
  bool low_edge, high_edge;
  __device__ bool at_edge(uint32_t i) const { return (i == 0 && low_edge) || (i + 1 == pieces && high_edge); }
  __device__ uint4 fetch(uint32_t i) const { return reinterpret_cast<const uint4*>(row - lead)[i]; }
  __device__ bool partial(uint32_t i) const { return (i == 0 && lead) || (i + 1 == pieces && (lead + count) % kPiece); }
  __device__ __noinline__ uint4 masked(uint32_t i, uint4 q) const {
    const int64_t at = int64_t(uint64_t(i) * kPiece) - lead;
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      const bool in = at + k >= 0 && at + k < count;
      if (sizeof(T) == 2)
        w[k / 2] = in ? w[k / 2] : __byte_perm(w[k / 2], 0xFF80u, k & 1 ? 0x5410 : 0x3254);
      else
        w[k & 3] = in ? w[k & 3] : 0xFF800000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __noinline__ uint4 edge(uint32_t i) const {
    const int64_t at = int64_t(uint64_t(i) * kPiece) - lead;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      const int64_t j = at + k;
      const bool in = j >= 0 && j < count;
      if (sizeof(T) == 2)
        w[k / 2] |= (in ? uint32_t(*reinterpret_cast<const uint16_t*>(row + j)) : 0xFF80u) << (16 * (k & 1));
      else
        w[k & 3] = in ? *reinterpret_cast<const uint32_t*>(row + j) : 0xFF800000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ uint4 read(uint32_t i) const { return at_edge(i) ? edge(i) : partial(i) ? masked(i, fetch(i)) : fetch(i); }
  __device__ void piece(uint32_t i, float (&v)[kPiece]) const {
    unpack(kResident ? kept[i] : read(i), v, static_cast<const T*>(nullptr));
  }
  __device__ uint32_t token(uint32_t i) const { return begin + i * kPiece - lead; }  // of the first element of piece i
  __device__ float logit(uint32_t j) const {  // of token begin + j; -0 and NaN replaced
    const T* p = kResident ? reinterpret_cast<const T*>(kept) + lead + j : row + j;
    return plain(sizeof(T) == 2 ? __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16) : *reinterpret_cast<const float*>(p));
  }

  template <typename F>
  __device__ void each(F f) const {  // (logit, token); -0 and NaN replaced
    for (uint32_t i = threadIdx.x; i < pieces; i += kThreads) {
      float v[kPiece];
      piece(i, v);
      const uint32_t t = token(i);
#pragma unroll
      for (int k = 0; k < kPiece; ++k) f(plain(v[k]), t + k);
    }
  }
};

struct Drawn {
  bool here, sure;
  uint32_t token;
  float logit;
};

// Draws among the tokens within `cut` (kCut; else all) that min-p keeps, in the order of the tokens: sums of warps, each a
// stretch of pieces. kExact: with exp_fixed; else in FP32, and `sure` tells whether the place is
// further from the borders of its token than the sums can be off.
//   FP32, relative to the total: a weight 2^-z is off by 2^-22 for the exponential and z 2^-23 ln 2 for the rounding of z; the
//   mean of z by weight is the entropy of the weights less log2 of their sum, so log2 of the vocabulary at most, 20: 2^-22 +
//   20 * 2^-23.5. A sum of 8: 7 * 2^-24, its product with the unit 2^-24, roundings to multiples of 2^-S: 2^-22.8. Together below
//   2^-18.5. With e in front of the place and e' behind it, u times the total and the running sum differ by
//   u e' - (1 - u) e: not more. So the token is sure where the place is 2^-18 of the total away from its borders.
template <bool kExact, bool kCut, typename T, bool kResident>
__device__ Drawn draw_spread(Shared& sh, Cluster& cluster, const Slice<T, kResident>& slice, const Settings& s, const Row& r, const Cut& cut,
                             uint64_t* whole_out) {
  constexpr int kPiece = Slice<T, kResident>::kPiece;
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;
  const uint32_t turns = (slice.pieces + kThreads - 1) / kThreads;  // a warp: turns * 32 pieces in a row
  const uint32_t p0 = warp * turns * 32u;
  const bool some_only = kCut || s.maybe > lowest();
  auto keep = [&](float v, uint32_t t) {
    return v >= s.maybe && (!kCut || cut.keeps(Keys<T>::of(plain(v)), t)) && (v >= s.surely || s.keeps(v, r, sh.table));
  };
  uint64_t mass = 0, whole = 0;
  for (uint32_t i = 0; i < turns; ++i) {
    const uint32_t p = p0 + i * 32u + lane;
    if (p >= slice.pieces) break;
    float v[kPiece];
    slice.piece(p, v);
    const uint32_t t = slice.token(p);
    if (kExact) {
#pragma unroll
      for (int k = 0; k < kPiece; ++k) {
        const uint64_t w = exp_fixed(plain(v[k]), r, sh.table);
        whole += w;
        if (some_only && w && keep(v[k], t + k)) mass += w;
      }
    } else {
      float w[kPiece], all = 0.0f;
#pragma unroll
      for (int k = 0; k < kPiece; ++k) all += w[k] = exp_fast(v[k], r);
      whole += fixed_of(all, r);
      if (some_only) {
        float some = 0.0f;
#pragma unroll
        for (int k = 0; k < kPiece; ++k) some += keep(v[k], t + k) ? w[k] : 0.0f;
        if (some > 0.0f) mass += fixed_of(some, r);
      }
    }
  }
  uint64_t all, at;
  if (some_only) {
    sums_of<true>(mass, whole, sh, cluster, &all, whole_out, &at);
  } else {
    sums_of<false>(whole, 0, sh, cluster, &all, nullptr, &at);
    *whole_out = all;
  }
  const uint64_t under = place_of(s.u, all);
  Drawn d{false, false, 0, 0.0f};
  uint64_t from = at, mine = 0;  // sums in front of this CTA, and its own
#pragma unroll
  for (uint32_t k = 0; k < kWarps; ++k) {
    if (k < warp) from -= sh.part[k];
    mine += sh.part[k];
  }
  if (from <= under && under < from + mine) {  // one CTA of the cluster: the warp in whose stretch the token lies
    uint32_t who = 0;
    uint64_t edge = from;
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) {
      edge += sh.part[k];
      if (under >= edge) who = k + 1, from = edge;
    }
    for (uint32_t i = 0; i < turns; i += kWarps) {  // each warp takes a turn of that stretch
      const uint32_t p = (who * turns + i + warp) * 32u + lane;
      const bool in = i + warp < turns && p < slice.pieces;
      float v[kPiece];
      uint64_t w[kPiece], own = 0;
      if (in) slice.piece(p, v);
#pragma unroll
      for (int k = 0; k < kPiece; ++k) {
        w[k] = in && (!some_only || keep(v[k], slice.token(p) + k)) ? (kExact ? exp_fixed(plain(v[k]), r, sh.table) : fixed_of(exp_fast(v[k], r), r)) : 0;
        own += w[k];
      }
      const uint64_t up = warp_up(own);
      __syncthreads();
      if (lane == 31) sh.part2[warp] = up;
      __syncthreads();
      uint64_t next = from, front = from;
#pragma unroll
      for (uint32_t k = 0; k < kWarps; ++k) {
        if (k < warp) front += sh.part2[k];
        next += sh.part2[k];
      }
      if (under < next) {
        front += up - own;
        if (front <= under && under < front + own) {
          uint32_t which = 0;
#pragma unroll
          for (int j = 0; j + 1 < kPiece; ++j)
            if (which == uint32_t(j) && under >= front + w[j]) front += w[j], which = j + 1;
          uint64_t size = 0;
#pragma unroll
          for (int j = 0; j < kPiece; ++j)
            if (which == uint32_t(j)) size = w[j], d.logit = v[j];
          const uint64_t off = all >> 18;
          d.here = true;
          d.token = slice.token(p) + which;
          d.sure = kExact || (under - front > off && front + size - under > off);
        }
        break;
      }
      from = next;
    }
  }
  return d;
}

template <typename T, bool kResident>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a, uint32_t ctas, uint32_t per) {
  __shared__ Shared sh;
  extern __shared__ uint4 pieces[];
  Cluster cluster{ctas, ctas > 1 ? blockIdx.x % ctas : 0u, 0, 0}, alone{1, 0, 0, 0};
  if (threadIdx.x == 0) sh.listed = sh.sure = sh.crowd = 0;
  cluster.arrive();  // so that every CTA of the cluster is known to run before one writes into another's memory
  stream_ready();
  const unsigned long long entry = kExp2[threadIdx.x & 63u];  // stored once the row is on its way: the arrival above would wait for it
  const uint32_t row = blockIdx.x / ctas;
  constexpr int kPiece = Slice<T, kResident>::kPiece;
  Slice<T, kResident> slice;
  slice.begin = min(a.vocab, cluster.rank * per);
  slice.count = min(a.vocab - slice.begin, per);
  slice.row = static_cast<const T*>(a.logits) + row * a.stride + slice.begin;
  slice.lead = uint32_t(reinterpret_cast<uintptr_t>(slice.row) & 15u) / sizeof(T);
  const SliceEdges edges = slice_edges(row * a.stride + slice.begin, slice.count, slice.lead, kPiece, (a.rows - 1) * a.stride + a.vocab);
  slice.pieces = edges.pieces;
  slice.kept = pieces;
  slice.low_edge = edges.low;
  slice.high_edge = edges.high;

  Settings s;
  s.t = a.temperature ? a.temperature[row] : 1.0f;
  s.p = a.top_p ? a.top_p[row] : 1.0f;
  s.k = a.top_k ? a.top_k[row] : 0;
  s.u = a.uniform[row];
  float min_p = a.min_p ? a.min_p[row] : 0.0f;

  float most = lowest();
  auto take = [&](uint32_t i, const uint4& q) {
    if (kResident) pieces[i] = q;
    most = max_with(q, most, static_cast<const T*>(nullptr));
  };
  const uint32_t p0 = slice.low_edge ? 1 : 0, p1 = slice.pieces - (slice.high_edge ? 1 : 0);
  constexpr int kAhead = 8;
  for (uint32_t i = p0 + threadIdx.x; i < p1; i += kThreads * kAhead) {
    uint4 q[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kThreads < p1) q[j] = slice.fetch(i + j * kThreads);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i + j * kThreads < p1) take(i + j * kThreads, slice.partial(i + j * kThreads) ? slice.masked(i + j * kThreads, q[j]) : q[j]);
  }
  if (threadIdx.x == 0 && p0) take(0, slice.edge(0));
  if (threadIdx.x == 32 && p1 < slice.pieces && p1 >= p0) take(p1, slice.edge(p1));

  if (threadIdx.x < 64) sh.table[threadIdx.x] = entry;

  bool greedy, cuts, nucleus;
  auto decide = [&]() {
    greedy = !(s.t > 0.0f);
    cuts = !greedy && s.k > 0 && uint32_t(s.k) < a.vocab, nucleus = !greedy && s.p < 1.0f;
  };
  decide();
  if (cuts || nucleus)
    for (uint32_t i = threadIdx.x; i < 2 * kBins; i += kThreads) sh.low[0][i] = 0, sh.high[0][i] = 0;

  // the largest, and a bound below the k-th largest of the row
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5, own_key = key_of(plain(most));
  uint32_t bound = 0;
  if (cuts) {
    sh.keys[threadIdx.x] = own_key >> 16;
    __syncthreads();
    const uint32_t part = (uint32_t(s.k) + ctas - 1) / ctas;
    if (warp == 0 && part <= kThreads) {  // the part-th largest of the threads' own, to 16 bits, by halving
      uint32_t key[kThreads / 32], end = 0;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) key[k] = sh.keys[k * 32 + lane], end = max(end, key[k]);
      end = __reduce_max_sync(0xFFFFFFFFu, end) + 1;
      auto at_least = [&](uint32_t k) {
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < kThreads / 32; ++j) n += key[j] >= k ? 1u : 0u;
        return __reduce_add_sync(0xFFFFFFFFu, n);
      };
      // between the top and 8 binades below it, as a rule
      bound = key_of(lowest()) >> 16;
      const uint32_t near = max(bound, end - min(end, 1024u));
      if (at_least(near) >= part)
        bound = near;
      else
        end = near;
      while (end - bound > 4) {  // at least `part` are at or above bound; 4: a thirtieth of the logit
        const uint32_t mid = bound + (end - bound) / 2;
        if (at_least(mid) >= part)
          bound = mid;
        else
          end = mid;
      }
      bound <<= 16;
    }
  }
  sh.tokens[warp] = __reduce_max_sync(0xFFFFFFFFu, own_key);
  __syncthreads();
  cluster.wait();
  if (warp == 0) {
    cluster.post(sh.tops, __reduce_max_sync(0xFFFFFFFFu, lane < kWarps ? sh.tokens[lane] : 0u));
    cluster.post(sh.bounds, bound);
  }
  if (cluster.rank == 0 && warp == kWarps - 1 && lane < ctas) {
    const float t = greedy ? 1.0f : fmaxf(s.t, kLeastT), ch = __fdiv_rn(kLog2EHi, t);  // log2(e) / T as a sum of two floats
    const float cl = __fdiv_rn(__fadd_rn(__fmaf_rn(-ch, t, kLog2EHi), kLog2ELo), t);
    cluster.store(&sh.t, lane, greedy ? s.t : t);
    cluster.store(&sh.p, lane, s.p);
    cluster.store(&sh.u, lane, s.u);
    cluster.store(&sh.min_p, lane, min_p);
    cluster.store(&sh.ch, lane, ch);
    cluster.store(&sh.cl, lane, fabsf(cl) <= ch ? cl : 0.0f);  // not at the ends of the range of temperatures
    cluster.store(&sh.down, lane, -__fmul_rn(t, logf(fminf(min_p, 1.0f))));  // off by 2^-22 at most
    cluster.store(&sh.k, lane, uint32_t(s.k));
  }
  cluster.sync();
  s.t = sh.t, s.p = sh.p, s.u = sh.u, s.k = int32_t(sh.k), min_p = sh.min_p;
  decide();
  if (greedy) s.t = 1.0f;
  uint32_t high = __reduce_max_sync(0xFFFFFFFFu, lane < ctas ? sh.tops[lane] : 0u);
  bound = __reduce_min_sync(0xFFFFFFFFu, lane < ctas ? sh.bounds[lane] : 0xFFFFFFFFu);
  if (!cuts) bound = 0;
  Row r;
  r.top = of_key(high);
  if (r.top == lowest()) {
    if (threadIdx.x == 0 && cluster.rank == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = r.top;
    }
    return;
  }
  r.ch = sh.ch, r.cl = sh.cl;
  r.scale = min(47, 30 + __clz((a.vocab - 1) | 1));
  r.c0 = -__fmul_rn(r.top, r.ch);
  r.plain = fabsf(r.c0) <= 1048576.0f && r.ch <= 1048576.0f && a.vocab <= (1u << 20);
  const float unit = __int_as_float((127 + r.scale) << 23);
  r.unit = r.plain ? __fmul_rn(unit, ex2(-__fmaf_rn(r.top, r.ch, r.c0))) : unit;
  s.maybe = s.surely = lowest();
  s.least = 0;
  if (min_p > 0.0f && !greedy) {
    s.maybe = s.surely = r.top;
    if (min_p < 1.0f) {
      const float down = sh.down;
      s.maybe = r.top - down * (1.0f + 0x1p-18f) - fabsf(r.top) * 0x1p-22f;
      s.surely = fminf(r.top, r.top - down * (1.0f - 0x1p-18f) + fabsf(r.top) * 0x1p-22f);
      s.least = __float2ull_ru(__fmul_rn(min_p, unit));
      if (!(s.maybe < s.surely)) s.maybe = s.surely;
    }
  }
  auto finish = [&](uint32_t token, float v, uint64_t whole) {  // one thread
    a.tokens[row] = int32_t(token);
    if (a.logprobs) {
      const float z = v == r.top ? 0.0f : __fdiv_rn(__fsub_rn(v, r.top), s.t);
      a.logprobs[row] = z - logf(__fmul_rn(__ull2float_rn(whole), __int_as_float((127 - r.scale) << 23)));
    }
  };

  // draws from the slices: in FP32, and again where that leaves it open
  uint64_t whole = 0;
  auto draw = [&](const Cut& cut, auto cutting) {
    constexpr bool kCut = decltype(cutting)::value;
    uint64_t sum;
    if (r.plain) {
      const Drawn d = draw_spread<false, kCut>(sh, cluster, slice, s, r, cut, &sum);
      if (!kCut) whole = sum;
      if (__any_sync(0xFFFFFFFFu, d.here && d.sure) && lane < ctas) cluster.store(&sh.sure, lane, 1u);
      if (d.here && d.sure) finish(d.token, d.logit, whole);
      cluster.sync();
      if (sh.sure) return;
    }
    const Drawn d = draw_spread<true, kCut>(sh, cluster, slice, s, r, cut, &sum);
    if (!kCut) whole = sum;
    if (d.here) finish(d.token, d.logit, whole);
  };
  if (!cuts && !nucleus && !greedy) {
    draw(Cut{}, std::false_type{});
    return;
  }

  // the whole row's sum, in FP32 where it can be, and the first of the largest
  uint32_t first = 0xFFFFFFFFu;
  if (a.logprobs || greedy || !cuts) {
    if (r.plain) {
      for (uint32_t i = threadIdx.x; i < slice.pieces; i += kThreads) {
        float v[kPiece], sum = 0.0f;
        slice.piece(i, v);
#pragma unroll
        for (int k = 0; k < kPiece; ++k) sum += exp_fast(v[k], r);
        whole += fixed_of(sum, r);
      }
    } else {
      slice.each([&](float v, uint32_t) { whole += exp_fixed(v, r, sh.table); });
    }
  }
  if (greedy) {
    for (uint32_t i = threadIdx.x; i < slice.pieces && first == 0xFFFFFFFFu; i += kThreads) {
      float v[kPiece];
      slice.piece(i, v);
#pragma unroll
      for (int k = kPiece - 1; k >= 0; --k) first = v[k] == r.top ? slice.token(i) + k : first;
    }
  }
  uint64_t front_of;
  if (greedy) {
    first = ~max_of(~first, sh);
    if (threadIdx.x < 32) cluster.post(sh.firsts, first);
    sums_of<false>(whole, 0, sh, cluster, &whole, nullptr, &front_of);
    if (ctas > 1) first = __reduce_min_sync(0xFFFFFFFFu, lane < ctas ? sh.firsts[lane] : 0xFFFFFFFFu);
    if (cluster.rank == 0 && threadIdx.x == 0) finish(first, r.top, whole);
    return;
  }
  float apart = 0.0f;         // bins of a unit of the logits
  uint32_t b1 = 0, b2 = kBins;  // the bins in which the nucleus ends
  bool crowded = false;         // more tokens up to there than a list holds
  auto bin_of = [&](float v) { return min(uint32_t(kBins - 1), __float2uint_rz(__fmul_rn(__fsub_rn(r.top, v), apart))); };
  if (!cuts) {  // what lies below weighs less than 1 - p of the row, even if it were the whole vocabulary
    sums_of<false>(whole, 0, sh, cluster, &whole, nullptr, &front_of);
    // FP32: as draw_spread has it, and 2^-22 and 2^-24 for the unit; 2^-18 covers it
    const float mass = __fmul_rd(__ull2float_rd(whole - (whole >> 18)), __int_as_float((127 - r.scale) << 23));
    const float left = __fmul_rd(__fsub_rd(1.0f, fmaxf(s.p, 0.0f)), __fdiv_rd(mass, __uint2float_ru(a.vocab)));
    const float down = fmaxf(0.0f, -__fmul_rn(s.t, logf(left)));  // off by 2^-22 at most
    const float bar = plain(r.top - down * (1.0f + 0x1p-18f) - s.t * 0x1p-18f - fabsf(r.top) * 0x1p-22f);
    bound = min(high, key_of(bar));
    // masses of the tokens from there on by their distance from the top, in multiples of 2^-31 of the row's: off by half
    // a multiple a token, 2^17 of them for 2^18 tokens, and by 2^-18 of the row's, 2^13, for FP32: 2^18 is more than both
    uint32_t* hist = sh.low[1];  // the first search clears it
    apart = __fdiv_rn(float(kBins), fmaxf(r.top - bar, 1e-20f));
    const float grain = __fdividef(__fmul_rn(0x1p31f, r.unit), __ull2float_rn(whole));
    if (r.plain && a.vocab <= (1u << 18)) {
      for (uint32_t i = threadIdx.x; i < slice.pieces; i += kThreads) {
        float v[kPiece];
        slice.piece(i, v);
#pragma unroll
        for (int k = 0; k < kPiece; ++k)
          if (v[k] >= bar) atomicAdd(&hist[bin_of(v[k])], __float2uint_rn(__fmul_rn(exp_fast(v[k], r), grain)));
      }
      cluster.sync();
      const uint32_t bin = 2 * threadIdx.x;
      uint64_t m[2] = {0, 0};
      for (uint32_t c = 0; c < ctas; c += 8) {
        uint64_t w[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) w[j] = c + j < ctas ? cluster.load(reinterpret_cast<const unsigned long long*>(&hist[bin]), c + j) : 0;
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) m[0] += uint32_t(w[j]), m[1] += w[j] >> 32;
      }
      const uint64_t up = warp_up(m[0] + m[1]);
      if ((threadIdx.x & 31u) == 31u) sh.part[threadIdx.x >> 5] = up;
      if (threadIdx.x == 0) sh.bin = sh.end = kBins - 1;
      __syncthreads();
      uint64_t at = up - m[0] - m[1];
      for (uint32_t k = 0; k < (threadIdx.x >> 5); ++k) at += sh.part[k];
      const float goal = fmaxf(s.p, 0.0f) * 0x1p31f;
      const uint64_t from = __float2ull_rd(fmaxf(goal - 0x1p18f, 0.0f)), to = __float2ull_ru(goal + 0x1p18f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (at <= from && from < at + m[j]) sh.bin = bin + j;
        if (at < to && to <= at + m[j]) sh.end = bin + j;
        at += m[j];
      }
      __syncthreads();
      b1 = sh.bin, b2 = sh.end;
      // so many tokens at least lie there, each at most as heavy as its bin's upper end: too many for a list? Only the way
      // hangs on it, so no quotient is rounded with care.
      uint32_t n = 0;
      const float step = (r.top - bar) * (1.0f / kBins), part = __fmul_rn(__ull2float_rn(whole), 0x1p-31f) * ex2(-__log2f(r.unit));
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (bin + j <= b2)
          n += __float2uint_rd(fminf(1e6f, __ull2float_rn(m[j]) * part * ex2(fminf(-__fmaf_rn(r.top - float(bin + j) * step, r.ch, r.c0), 100.0f))));
      n = __reduce_add_sync(0xFFFFFFFFu, n);
      if (lane == 0) atomicAdd(&sh.crowd, n);
      __syncthreads();
      crowded = sh.crowd > kList;
    }
  }
  // the tokens at or above the bound: a list in each CTA
  if (bound && !crowded) {
    const float bar = of_key(max(bound, key_of(lowest()) + 1));
    constexpr uint32_t kSet = 64 / kPiece;  // pieces whose comparisons fit into 64 bits
    for (uint32_t i0 = threadIdx.x; i0 < slice.pieces; i0 += kThreads * kSet) {
      uint64_t mine = 0;
#pragma unroll
      for (uint32_t j = 0; j < kSet; ++j) {
        const uint32_t i = i0 + j * kThreads;
        if (i >= slice.pieces) break;
        float v[kPiece];
        slice.piece(i, v);
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kPiece; ++k) m |= (v[k] >= bar ? 1u : 0u) << k;
        mine |= uint64_t(m) << (j * kPiece);
      }
      for (; mine; mine &= mine - 1) {
        const uint32_t b = __ffsll(static_cast<long long>(mine)) - 1, j = (i0 + b / kPiece * kThreads) * kPiece + b % kPiece - slice.lead;
        const float v = slice.logit(j);
        if (!cuts && bin_of(v) > b2) continue;
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kList) sh.keys[at] = Keys<T>::of(v), sh.tokens[at] = slice.begin + j;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) cluster.post(sh.counts, crowded ? kList + 1 : sh.listed);
  if (cuts)
    sums_of<false>(whole, 0, sh, cluster, &whole, nullptr, &front_of);
  else
    cluster.sync();
  const uint32_t own_count = lane < ctas ? sh.counts[lane] : 0u;
  const bool fits = __all_sync(0xFFFFFFFFu, own_count <= kList);
  const uint32_t listed = fits ? __reduce_add_sync(0xFFFFFFFFu, own_count) : kList + 1;
  // The lists of all CTAs behind the first one's, in its memory, after the next sync().
  auto push = [&](const uint32_t* counts) {
    if (cluster.rank == 0) return;
    const uint32_t at = __reduce_add_sync(0xFFFFFFFFu, lane < cluster.rank ? counts[lane] : 0u);
    for (uint32_t i = threadIdx.x; i < counts[cluster.rank]; i += kThreads) {
      cluster.store(&sh.keys[at + i], 0, sh.keys[i]);
      cluster.store(&sh.tokens[at + i], 0, sh.tokens[i]);
    }
  };
  // The whole row's sum with exp_fixed where the first CTA wants it (`need`), by all of them; else 0. The other CTAs wait
  // here for what it wants: alone it would take 75 us for a row of 2^17.
  auto settle = [&](bool need) {
    if (cluster.rank == 0 && threadIdx.x < ctas) cluster.store(&sh.sure, threadIdx.x, need ? 1u : 0u);
    cluster.sync();
    uint64_t mass = 0;
    if (sh.sure) {
      slice.each([&](float v, uint32_t) { mass += exp_fixed(v, r, sh.table); });
      sums_of<false>(mass, 0, sh, cluster, &mass, nullptr, &front_of);
    }
    return mass;
  };
  // A list of a token a thread in the order of falling logits, by comparing all with all. In the histograms' room.
  auto* pairs = reinterpret_cast<unsigned long long*>(sh.low);
  auto* weights = pairs + kThreads;
  uint32_t *keys = sh.high[0], *tokens = sh.high[0] + kThreads;
  auto pair = [&](uint32_t k, uint32_t t) { return static_cast<unsigned long long>(uint64_t(k) << 32 | ~t); };  // not 0
  auto order = [&](uint32_t n, uint64_t mine) {  // of pairs[0] .. pairs[n - 1], 0 behind them; this thread's
    uint32_t place = 0;
    for (uint32_t j = 0; j < n; j += 2) {
      const ulonglong2 two = reinterpret_cast<const ulonglong2*>(pairs)[j / 2];
      place += (two.x > mine ? 1u : 0u) + (two.y > mine ? 1u : 0u);
    }
    if (threadIdx.x < n) {
      keys[place] = uint32_t(mine >> 32);
      tokens[place] = ~uint32_t(mine);
      weights[place] = exp_fixed(Keys<T>::value(uint32_t(mine >> 32)), r, sh.table);
    }
    __syncthreads();
  };
  auto order_list = [&](uint32_t n) {
    const uint64_t mine = threadIdx.x < n ? pair(sh.keys[threadIdx.x], sh.tokens[threadIdx.x]) : 0;
    pairs[threadIdx.x] = mine;
    __syncthreads();
    order(n, mine);
  };
  // Running sums over such a list, and the sums of the kept tokens in front of each in the order of tokens.
  auto end_small = [&](uint32_t n) {
    const uint32_t i = threadIdx.x;
    order_list(n);
    const uint32_t c = cuts ? min(uint32_t(s.k), n) : n;
    const uint64_t w = i < c ? weights[i] : 0;
    uint64_t before = warp_up(w) - w;
    if (lane == 31) sh.part[i >> 5] = before + w;
    __syncthreads();
    uint64_t mass = 0;
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) {
      if (k < (i >> 5)) before += sh.part[k];
      mass += sh.part[k];
    }
    bool kept = i < c;
    if (nucleus) {
      const uint64_t off = !cuts && r.plain ? whole >> 18 : 0;
      if (!cuts) mass = whole;
      uint64_t share = s.p > 0.0f ? part_of(s.p, mass - off, true) : 0;
      if (off) {
        const bool open = __syncthreads_or(kept && i > 0 && s.p > 0.0f && before >= share && before < part_of(s.p, mass + off, true));
        mass = settle(open);  // the sum in FP32 leaves the last token open
        if (open) share = part_of(s.p, mass, true);
      }
      kept = kept && (i == 0 || before < share);
    }
    const float v = kept ? Keys<T>::value(keys[i]) : 0.0f;
    kept = kept && s.keeps(v, r, sh.table);
    const uint32_t last = __syncthreads_count(kept);  // the kept ones are the first of the order
    mass = sum_of(kept ? w : 0, sh);
    const uint64_t under = place_of(s.u, mass);
    if (kept) {
      const uint32_t t = tokens[i];
      uint64_t front = 0;
      for (uint32_t j = 0; j < last; ++j) front += tokens[j] < t ? weights[j] : 0;
      if (front <= under && under < front + w) finish(t, v, whole);
    }
  };
  // The end of the nucleus in such a list of n, ordered, as nucleus_of finds it.
  enum { kFound, kOpen, kElsewhere };
  auto nucleus_small = [&](uint32_t n, uint64_t mass, uint64_t off, uint64_t front, Cut* cut) {
    const uint32_t i = threadIdx.x;
    const uint64_t w = i < n ? weights[i] : 0, share = max(1ull, static_cast<unsigned long long>(s.p > 0.0f ? part_of(s.p, mass - off, true) : 0));
    uint64_t before = front + warp_up(w) - w;
    __syncthreads();
    if (lane == 31) sh.part[warp] = before + w - front;
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k)
      if (k < warp) before += sh.part[k];
    const uint32_t last = __syncthreads_count(i < n && before < share);  // the first ones of the order
    const uint64_t most = off && s.p > 0.0f ? part_of(s.p, mass + off, true) : share;
    if (__syncthreads_or(i < n && before >= share && before < most)) return kOpen;
    const bool ends = __syncthreads_or(last != 0 && i + 1 == last && before + w >= most);
    if (ends) *cut = Cut{keys[last - 1], tokens[last - 1]};
    return ends ? kFound : kElsewhere;
  };
  const uint32_t low = Keys<T>::of(of_key(max(bound, key_of(lowest()))));
  high = Keys<T>::of(r.top);
  Cut cut;
  if (bound != 0 && listed <= kList) {
    push(sh.counts);
    cluster.sync();
    if (cluster.rank != 0) {  // the first CTA ends the row
      if (nucleus && !cuts && r.plain) settle(false);
      return;
    }
    if (listed <= kThreads) {
      end_small(listed);
    } else {
      auto each = [&](auto f) {
        for (uint32_t i = threadIdx.x; i < listed; i += kThreads) f(sh.keys[i], sh.tokens[i]);
      };
      if (cuts) cut = top_k_of<T>(sh, alone, s, a.vocab, low, high, each);
      if (nucleus) {
        uint64_t mass = whole, off = r.plain ? whole >> 18 : 0;
        if (cuts) {
          mass = off = 0;
          each([&](uint32_t k, uint32_t i) { if (cut.keeps(k, i)) mass += exp_fixed(Keys<T>::value(k), r, sh.table); });
          mass = sum_of(mass, sh);
        }
        int state = kElsewhere;
        if (off) {  // the bins in which it ends hold few tokens, as a rule; those in front of them belong to it
          __syncthreads();
          pairs[threadIdx.x] = 0;
          if (threadIdx.x == 0) sh.listed = 0;
          __syncthreads();
          uint64_t front = 0;
          each([&](uint32_t k, uint32_t i) {
            const float v = Keys<T>::value(k);
            if (bin_of(v) < b1) {
              front += exp_fixed(v, r, sh.table);
            } else {
              const uint32_t at = atomicAdd(&sh.listed, 1u);
              if (at < kThreads) pairs[at] = pair(k, i);
            }
          });
          front = sum_of(front, sh);
          const uint32_t few = sh.listed;
          if (few <= kThreads) {
            order(few, pairs[threadIdx.x]);
            state = nucleus_small(few, mass, off, front, &cut);
            mass = settle(state != kFound);  // exact where the sum in FP32 leaves the last token open
            off = 0;
            if (state == kOpen) state = nucleus_small(few, mass, 0, front, &cut);
          }
          __syncthreads();
          for (uint32_t i = threadIdx.x; i < 2 * kBins; i += kThreads) sh.low[0][i] = 0, sh.high[0][i] = 0;
          __syncthreads();
        }
        if (state != kFound) {
          const bool open = !nucleus_of<T>(sh, alone, s, r, a.vocab, low, high, mass, off, 0, &cut, each);
          if (off) {
            mass = settle(open);
            if (open) nucleus_of<T>(sh, alone, s, r, a.vocab, low, high, mass, 0, 0, &cut, each);
          }
        }
      }
      auto kept = [&](auto add) {
        each([&](uint32_t k, uint32_t i) {
          const float v = Keys<T>::value(k);
          if (cut.keeps(k, i) && s.keeps(v, r, sh.table)) add(~i, [&] { return exp_fixed(v, r, sh.table); });
        });
      };
      uint64_t mass = 0;
      kept([&](uint32_t, auto w) { mass += w(); });
      mass = sum_of(mass, sh);
      Found f;
      const uint32_t token = ~search<false>(sh, alone, ~(a.vocab - 1), ~0u, 0, place_of(s.u, mass) + 1, &f, kept);
      each([&](uint32_t k, uint32_t i) { if (i == token) finish(token, Keys<T>::value(k), whole); });
    }
    return;
  }
  auto each = [&](auto f) {
    slice.each([&](float v, uint32_t t) {
      const uint32_t k = Keys<T>::of(v);
      if (k >= low && v > lowest()) f(k, t);
    });
  };
  if (cuts) cut = top_k_of<T>(sh, cluster, s, a.vocab, low, high, each);
  if (nucleus && cuts) {
    uint64_t mass = 0;
    slice.each([&](float v, uint32_t t) { if (v > lowest() && cut.keeps(Keys<T>::of(v), t)) mass += exp_fixed(v, r, sh.table); });
    sums_of<false>(mass, 0, sh, cluster, &mass, nullptr, &front_of);
    nucleus_of<T>(sh, cluster, s, r, a.vocab, low, high, mass, 0, 0, &cut, each);
  } else if (nucleus) {
    // exact sums of the row and of what surely comes before the cut, and a new list: of the bins where it falls
    const float bar = of_key(bound);
    uint64_t mass = 0, front = 0;
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    slice.each([&](float v, uint32_t t) {
      const uint64_t w = exp_fixed(v, r, sh.table);
      mass += w;
      if (v >= bar && v > lowest()) {
        const uint32_t b = bin_of(v);
        if (b < b1) {
          front += w;
        } else if (b <= b2) {
          const uint32_t at = atomicAdd(&sh.listed, 1u);
          if (at < kList) sh.keys[at] = Keys<T>::of(v), sh.tokens[at] = t;
        }
      }
    });
    __syncthreads();
    if (threadIdx.x < 32) cluster.post(sh.firsts, sh.listed);
    sums_of<true>(mass, front, sh, cluster, &mass, &front, &front_of);
    const uint32_t own_listed = lane < ctas ? sh.firsts[lane] : 0u;
    bool found = false;
    if (__all_sync(0xFFFFFFFFu, own_listed <= kList) && __reduce_add_sync(0xFFFFFFFFu, own_listed) <= kList) {
      push(sh.firsts);
      cluster.sync();
      if (cluster.rank == 0) {
        const uint32_t n = __reduce_add_sync(0xFFFFFFFFu, own_listed);
        if (n <= kThreads) {
          order_list(n);
          found = nucleus_small(n, mass, 0, front, &cut) == kFound;
        } else {
          found = nucleus_of<T>(sh, alone, s, r, a.vocab, low, high, mass, 0, front, &cut, [&](auto f) {
            for (uint32_t i = threadIdx.x; i < n; i += kThreads) f(sh.keys[i], sh.tokens[i]);
          });
        }
        if (threadIdx.x < ctas) {
          cluster.store(&sh.cut[0], threadIdx.x, cut.key);
          cluster.store(&sh.cut[1], threadIdx.x, cut.token);
          cluster.store(&sh.cut[2], threadIdx.x, found ? 1u : 0u);
        }
      }
      cluster.sync();
      cut.key = sh.cut[0], cut.token = sh.cut[1];
      found = sh.cut[2] != 0;
    }
    if (!found) {
      cut = Cut{};
      __syncthreads();
      for (uint32_t i = threadIdx.x; i < 2 * kBins; i += kThreads) sh.low[0][i] = 0, sh.high[0][i] = 0;
      __syncthreads();
      nucleus_of<T>(sh, cluster, s, r, a.vocab, low, high, mass, 0, 0, &cut, each);
    }
  }
  draw(cut, std::true_type{});
}

template <typename T>
cudaError_t sample_of(const SampleArgs& a, int sms, cudaStream_t stream) {
  constexpr uint32_t kPiece = 16 / sizeof(T);
  // as few CTAs as hold the row in slices of the wanted size, more where there are fewer rows than SMs
  uint32_t ctas = 1;
  while (ctas < kCtas && uint64_t(a.vocab) * sizeof(T) > uint64_t(ctas) * kSliceBytes) ctas *= 2;
  while (ctas < kCtas && uint64_t(a.rows) * ctas * 2 <= uint64_t(sms) && a.vocab >= ctas * 4096) ctas *= 2;
  const uint32_t per = ((a.vocab + ctas - 1) / ctas + kPiece - 1) / kPiece * kPiece;
  uint64_t bytes = (uint64_t(per) / kPiece + 1) * 16;
  const bool resident = bytes <= kSliceMost;
  if (!resident) bytes = 0;
  const auto kernel = resident ? sample_kernel<T, true> : sample_kernel<T, false>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernels may use their shared memory and clusters
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    for (const auto k : {sample_kernel<T, true>, sample_kernel<T, false>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSliceMost));
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(a.rows * ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = size_t(bytes);
  c.stream = stream;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, a, ctas, per);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, bool bf16, int sms, cudaStream_t stream) {
  return bf16 ? sample_of<uint16_t>(a, sms, stream) : sample_of<float>(a, sms, stream);
}

}  // namespace pulse
