// Tokens from logits on sm_103a: temperature, top-k, top-p and min-p filters and one given random
// number per row.
//
//   order the row by (logit descending, index ascending); z = (l - max l) / T, w = e^z
//   keep the first top_k; of those, the shortest prefix whose mass reaches top_p of their mass;
//   of those, w >= min_p (of the largest token's 1); the first token always stays
//   S = sum of the kept w; token = lowest index whose kept mass so far exceeds u S; prob = w / S
// NaN counts as -inf, which has no mass. Every filter cuts the order at one place, so the kept set
// is {l > cut, or l == cut and index <= tie}.
//
// The answer is a whole number, and it is the one of the definition: a mass is a sum of integers (w
// in units of a power of two, so the order of summation does not matter). Two weights are used. The
// exact one (weight_pair) is good to about 2^-37 without 64-bit floats, of which this machine has
// few. The quick one is a single special-function exponential, and a mass of quick weights comes
// with a bound on its error; where a decision (a border of top-p, the token itself) lies within
// that bound, the mass is taken again from exact weights. The unit of an exact mass is 2^-60 to 2^-61
// of it, as a quick pass before has told (refine), or 2^-50 of the largest weight in a list of 2048:
// what rounding n weights to whole units drops, n / 2 units, is below 2^-37 of the mass for any n up
// to 2^24. (In units that fit any row of 2^24 tokens it would be 2^-14 of a heavy token's.)
//
// One row a cluster of up to 8 CTAs, each with a contiguous share of the vocabulary in its shared
// memory, read from memory once (rows too long for that are read again in each pass). Each warp
// has a contiguous part of the share and each thread re-reads its own loads only. The threads'
// maxima give a bound that at least `want` tokens reach and not many more; those go to the first
// CTA's list, which sorts them and settles top-k <= want, or a nucleus of less than that (with the
// row's mass from the same pass), there. What the list cannot settle (a larger top-k, a flat
// nucleus, too many ties, a border within the error bound) is cut by narrowing an interval around
// the cut with passes over the row, three pivots each, until the list holds what is in it.
//
// With many rows a row is one CTA's (which needs no exchange between CTAs) and reads its logits
// twice; rows that this leaves open (a large top-k, a flat nucleus, a border within the error bound)
// are marked and taken by larger clusters in a second launch (ds_head_sample.cu).
//
// Bound: the floor is one read of the logits, 20 us at 256 x 262144 bf16 and 40 us at 2048 x 32749
// fp32; the first launches there take 56 (top-k and top-p) to 86 us (nucleus) and 97 (token by mass)
// to 143 us (nucleus). At the first size two reads from memory are 40 us of it; beyond that it is issue slots
// (26 instructions a token) and a row's last steps, over a list of some tens to two thousand tokens,
// which keep a CTA waiting on barriers and shuffles. 64-bit floats cost thousands of cycles a row here
// and are not used. One row over eight CTAs takes 8 (greedy) to 15 us (filters), of which each exchange
// between the CTAs is about 2 us; a flat nucleus of 130000 tokens takes 100 to 160 us.
#pragma once

#include <climits>

#include "ds_head.h"

namespace ds {

namespace sample {

constexpr int kMaxCluster = 8;  // CTAs a row, at most

struct SampleArgs {
  const void* logits;
  const float *temperature, *top_p, *min_p, *u;
  const int32_t* top_k;
  const uint8_t* done;
  int32_t* token;
  float* prob;
  int64_t stride;
  int64_t rows;
  int vocab;
  int chunk;   // vocabulary entries per CTA (a multiple of 16 bytes of them), from the aligned-down
               // start of the row
  float unit;  // weights are counted in units of 1 / unit (a power of two; a sum of as many as the
               // vocabulary has fits 62 bits) before their mass is known
  int list_fine;  // units of a list are so many bits finer (kListUnit, or `unit` if that is finer)
};

// What a launch does with rows that quick passes do not settle: all of it, or leave them (token
// kLater and, where nothing is to be cut, how many bits finer the units that fit the kept mass are),
// or only what was left.
enum { kWhole = 0, kQuick = 1, kRest = 2 };
constexpr int kLater = INT_MIN;

constexpr int kListCap = 2048;  // tokens the first CTA's list holds
// Bits of a weight of 1 in the units of a whole that fits 62: of all tokens of a vocabulary, of a list.
constexpr int kMassBits = 61, kListBits = kMassBits - 11;
constexpr float kListUnit = 1ull << kListBits;
static_assert(kListCap <= 1 << 11, "the list's mass has to fit 62 bits");

// `clusters` clusters of C CTAs over the rows of q, and what a device needs for that once; one unit
// of this directory for each logit type and mode.
template <typename T, int MODE>
cudaError_t launch_rows(SampleArgs q, int C, int64_t clusters, int sms, cudaStream_t st);
template <typename T, int MODE>
cudaError_t prepare_rows();

#ifdef DS_SAMPLE_KERNELS
namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kPer = 4;              // entries of the first CTA's list a thread takes
static_assert(kListCap == kPer * kSampleThreads, "the list is one round of the CTA");
constexpr int kResidentMax = 160 * 1024;  // bytes of a row a CTA keeps


// 2^(j / 32), j = -16 .. 16, as the nearest float and the nearest float to the rest.
__device__ const float2 kExp2Table[33] = {
    {0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f}, {0x1.71f75e0000000p-1f, 0x1.1d8bee0000000p-26f}, {0x1.7a11480000000p-1f, -0x1.829fd00000000p-26f},
    {0x1.82589a0000000p-1f, -0x1.accc7c0000000p-27f}, {0x1.8ace540000000p-1f, 0x1.15506e0000000p-28f}, {0x1.93737c0000000p-1f, -0x1.e647440000000p-26f},
    {0x1.9c49180000000p-1f, 0x1.51f8480000000p-28f}, {0x1.a5503c0000000p-1f, -0x1.b83b540000000p-26f}, {0x1.ae89fa0000000p-1f, -0x1.a94b140000000p-27f},
    {0x1.b7f7700000000p-1f, -0x1.a094380000000p-26f}, {0x1.c199be0000000p-1f, -0x1.3d56b20000000p-28f}, {0x1.cb720e0000000p-1f, -0x1.8837cc0000000p-28f},
    {0x1.d5818e0000000p-1f, -0x1.822dbc0000000p-28f}, {0x1.dfc9740000000p-1f, -0x1.908c940000000p-26f}, {0x1.ea4afa0000000p-1f, 0x1.52486c0000000p-28f},
    {0x1.f507660000000p-1f, -0x1.246eb00000000p-27f}, {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}};

// The row's map from logits to weights: w = 2^((l - m) log2(e) / T) with the factor as a float
// pair.
struct WeightMap {
  float m, c_hi, c_lo;
  const float2* table;
};

DS_DEV WeightMap weight_map(float m, float T, const float2* table) {
  // log2(e) = hi + lo; c_hi = rnd(hi / T), and what it misses of the quotient over T again
  constexpr float kLog2eHi = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;
  const float c = fminf(kLog2eHi / T, 3e38f);  // (finite for the least T too)
  const float rest = __fmaf_rn(-c, T, kLog2eHi) + kLog2eLo;
  return WeightMap{m, c, c >= 3e38f || c == 0.f ? 0.f : rest / T, table};
}

// e^((l - m) / T) as a float pair, for l <= m; relative error about 2^-37. The table-driven method of
// P. T. P. Tang (ACM Transactions on Mathematical Software 15, 1989) in pairs of floats: sums with
// their rounding errors by Knuth's two-sum and, where the larger term is known, Dekker's; products
// with theirs by a fused multiply-add. 2^t splits into a power of two, a table entry and e^z with
// |z| < 0.011, whose series stops at z^5 / 120 (the next term is below 2^-48) and is below 2^-14 from
// its second-order term on, so that part needs single precision only.
DS_DEV float2 weight_pair(const WeightMap& w, float l) {
  const float d = __fsub_rn(l, w.m);
  const float t0 = __fmul_rn(d, w.c_hi), t = fmaxf(t0, -64.f);
  const float b1 = __fadd_rn(d, w.m), a1 = __fsub_rn(d, b1);
  const float dl = __fsub_rn(__fsub_rn(l, b1), __fadd_rn(w.m, a1));
  float tl = __fmaf_rn(d, w.c_hi, -t);
  tl = __fmaf_rn(d, w.c_lo, tl);
  tl = __fmaf_rn(dl, w.c_hi, tl);
  // nearest integers by way of a large number's last bits
  constexpr float kBig = 12582912.f;  // 1.5 2^23
  const float tn = __fadd_rn(t, kBig), n = __fsub_rn(tn, kBig), f = __fsub_rn(t, n);
  const float fj = __fmaf_rn(f, 32.f, kBig), j = __fsub_rn(fj, kBig);
  const float r = __fmaf_rn(j, -0.03125f, f);
  const float a = __fadd_rn(r, tl), al = __fsub_rn(tl, __fsub_rn(a, r));
  constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
  const float zh = __fmul_rn(a, kLn2Hi);
  const float zl = __fmaf_rn(a, kLn2Lo, __fmaf_rn(al, kLn2Hi, __fmaf_rn(a, kLn2Hi, -zh)));
  const float s = __fmaf_rn(zh, __fmaf_rn(zh, __fmaf_rn(zh, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
  const float e = __fmaf_rn(__fmul_rn(zh, zh), s, zl);
  const float p = __fadd_rn(zh, e), pl = __fsub_rn(e, __fsub_rn(p, zh));
  const float2 tb = w.table[__float_as_int(fj) - (__float_as_int(kBig) - 16)];
  const float h = __fmul_rn(tb.x, p);
  const float hl = __fadd_rn(__fmaf_rn(tb.x, p, -h), __fmaf_rn(tb.x, pl, tb.y));
  const float sum = __fadd_rn(tb.x, h), rest = __fadd_rn(__fsub_rn(h, __fsub_rn(sum, tb.x)), hl);
  const float scale = __int_as_float((__float_as_int(tn) - (__float_as_int(kBig) - 127)) << 23);
  // 0 below every unit (and for -inf, and NaN from it); 1 at the maximum, +inf too
  const float k = l == w.m ? 1.f : (t0 > -64.f ? sum * scale : 0.f);
  return make_float2(k, l == w.m || !(t0 > -64.f) ? 0.f : rest * scale);
}

// The exact weight in units. A call in the kernels for rows left, whose passes are mostly these
// (256 x 262144 mixed: 224 us in all, 243 with copies in every pass, which spilled, as measured when
// that was chosen); inlined in the others (one row: 14.0 us, 14.6 with calls).
#ifdef DS_SAMPLE_WEIGHTS_CALLED
#define DS_WEIGHT_FN __device__ __noinline__
#else
#define DS_WEIGHT_FN DS_DEV
#endif
DS_WEIGHT_FN uint64_t weight_units_of(float m, float c_hi, float c_lo, const float2* table,
                                                 float l, float unit) {
  const float2 p = weight_pair(WeightMap{m, c_hi, c_lo, table}, l);
  return (uint64_t)(__float2ll_rn(p.x * unit) + __float2ll_rn(p.y * unit));
}
DS_DEV uint64_t weight_units(const WeightMap& w, float l, float unit) {
  return weight_units_of(w.m, w.c_hi, w.c_lo, w.table, l, unit);
}
// The exact weight to single precision.
DS_WEIGHT_FN float weight_of(float m, float c_hi, float c_lo, const float2* table, float l) {
  return weight_pair(WeightMap{m, c_hi, c_lo, table}, l).x;
}

// A quick weight is 2^t, t = l c - m c as one fused multiply-add with a rounded m c; what that
// rounding costs is the same factor for the whole row, known exactly and put back into the sums. A
// mass of quick weights is then off by no more than mass 2^-20 (the special-function unit's own 2^-22
// and the fp32 additions of a thread's sum, compensated: a few 2^-24) and sum w |t| 2 2^-24 ln 2 (the
// roundings of t and of c); and sum w |t| is no more than mass log2(n / mass) for n tokens with the
// largest weight 1, since the entropy of n tokens is no more than log2 n. prob is a weight over such a
// mass where the token needed no other: that is its 2^-20, and why its last bits follow the row's
// alignment. Exact masses everywhere would take 708 us where these take 102 (256 x 262144 bf16).
constexpr float kQuickRel = 9.6e-7f, kQuickArg = 1e-7f;

// ceil(x whole) and floor(x whole) for x in (0, 1): 64-bit floats cost this machine more than the
// 88-bit product.
DS_DEV uint64_t scale_mass(float x, uint64_t whole, bool up) {
  int e;
  const uint64_t f = (uint64_t)(frexpf(x, &e) * 16777216.f);  // x = f 2^(e - 24), exactly
  const int sh = 24 - e;                                     // at least 24
  const uint64_t hi = __umul64hi(f, whole), lo = f * whole;  // hi < 2^24
  if (sh >= 64) {
    const int h = sh - 64;
    const uint64_t q = h < 64 ? hi >> h : 0;
    const bool more = lo || (h < 64 ? (hi & ((1ull << h) - 1)) : hi);
    return q + (up && more);
  }
  return (lo >> sh | hi << (64 - sh)) + (up && (lo & ((1ull << sh) - 1)));
}

DS_DEV float to_f32(float v) { return v; }
DS_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// What stays of the row: l above `cut`, and at `cut` the indices up to `tie`.
struct Kept {
  float cut;
  int tie;
};
DS_DEV bool kept(const Kept& k, float l, int i) { return l > k.cut || (l == k.cut && i <= k.tie); }

DS_DEV uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Key of a list entry: larger means earlier in the order.
DS_DEV uint64_t list_key(float l, int i) {
  return ((uint64_t)float_key(l) << 32) | (uint32_t)~(uint32_t)i;
}
DS_DEV float key_logit(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
DS_DEV int key_index(uint64_t key) { return (int)~(uint32_t)key; }

// What the CTAs of a cluster tell one another.
struct Word {
  uint64_t a[3];
  uint64_t n[3];
  float f, g;
};

struct Found {
  uint64_t key, before, w;  // an entry of the list, what lies before it in some order, its own weight
};

struct Shared {
  Word in[2][kMaxCluster];  // by turns
  uint64_t wsum[3][kSampleWarps];
  float wf[kSampleWarps], wg[kSampleWarps];
  uint32_t wn[3][kSampleWarps];
  uint32_t hist[256];
  float2 table[33];
  uint32_t n_list;   // entries of this CTA's list (the first CTA's: of all)
  uint32_t n_local;
  int pick;
  uint32_t base;
  // the first CTA's findings, told to all
  int state;
  Kept cut;
  uint64_t list[kListCap];
  uint64_t extra[kListCap];  // a CTA's own finds; then the weights of the list
  uint16_t at[kListCap];     // places in the list of the entries of one bin
  uint64_t bin[256];
  uint4 edge[2];
  Found found;
  float4 map;  // m, c_hi, c_lo of the row's map, for put()
};

constexpr size_t kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;

DS_DEV uint32_t remote(const void* p, uint32_t rank) { return mapa_shared(smem_u32(p), rank); }
DS_DEV void st_remote_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
DS_DEV void st_remote_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
DS_DEV uint32_t add_remote_u32(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

enum { kOpen = 0, kDone = 1, kCut = 2 };

// The row's share of one CTA. T: type of the logits; RES: the share is in shared memory.
template <typename T, bool RES>
struct Row {
  static constexpr int E = 16 / (int)sizeof(T);  // entries of one 16-byte group
  static constexpr int STEP = 32 * E;            // entries a warp takes at a time
  const T* base;   // the row's start, aligned down to 16 bytes
  uint4* smem;     // groups of this CTA
  int lead;        // entries before the row's own first
  int first, last; // groups [first, last) of this warp, counted from `base`
  int g0, g1;      // groups [g0, g1) of this CTA,
  int wper;        // this many a warp
  int end;         // lead + vocab
  uint4* edge;     // [2] (shared): the row's first and last group where it fills them in part
  int full0, full1;  // groups [full0, full1) are filled whole

  DS_DEV uint4 fetch(int g) const {
    const int i = g * E;
    if (i >= lead && i + E <= end) return __ldg(reinterpret_cast<const uint4*>(base) + g);
    union {
      uint4 q;
      T v[E];
    } x;
#pragma unroll
    for (int e = 0; e < E; ++e)
      x.v[e] = i + e >= lead && i + e < end ? base[i + e] : static_cast<T>(-INFINITY);
    return x.q;
  }
  // NaN becomes -inf: the largest of a NaN and another value is the other
  DS_DEV static uint4 clean(uint4 q) {
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(fmaxf(__uint_as_float(w[i]), -INFINITY));
      } else {
        __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&w[i]);
        v = __hmax2(v, __nv_bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80)));
        w[i] = *reinterpret_cast<uint32_t*>(&v);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  DS_DEV static void unpack(uint4 q, float (&v)[E]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  DS_DEV void get(int g, float (&v)[E]) const {
    if constexpr (RES) unpack(smem[g - g0], v);
    else unpack(clean(*(g >= full0 && g < full1 ? reinterpret_cast<const uint4*>(base) + g : edge + (g >= full1))), v);
  }
  // f(values, group, largest value) for each of this thread's groups, a few fetched at a time.
  template <typename F>
  DS_DEV void each(F f) const {
    constexpr int U = RES ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const uint4* src = reinterpret_cast<const uint4*>(base);
    for (int b = first + lane; b < last; b += 32 * U) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int g = b + 32 * i;
        if (g < last) q[i] = RES ? smem[g - g0] : *(g >= full0 && g < full1 ? src + g : edge + (g >= full1));
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (b + 32 * i < last) {
          const uint4 x = RES ? q[i] : clean(q[i]);
          float v[E];
          unpack(x, v);
          f(v, b + 32 * i, most(x));
        }
    }
  }
  // The largest entry of a group as it lies in memory (NaN already -inf).
  DS_DEV static float most(uint4 q) {
    if constexpr (sizeof(T) == 4) {
      return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                   fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    } else {  // in pairs
      const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&q);
      const __nv_bfloat162 x = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
      return fmaxf(__low2float(x), __high2float(x));
    }
  }
  DS_DEV int index(int g) const { return g * E - lead; }  // vocabulary index of a group's first
};

template <typename T, bool RES, int MODE>
struct Sampler {
  using R = Row<T, RES>;
  static constexpr int E = R::E;
  Shared& sh;
  R row;
  int C;          // CTAs in the cluster
  uint32_t rank;
  int turn = 0;
  float m = 0.f, T_r = 1.f, unit0;
  int fine = 0;
  WeightMap map;
  float c_quick = 0.f, b_quick = 0.f, fix_quick = 0.f;  // log2(e) / T, -m of it, the row's factor
  bool odd = false;  // the maximum is +inf, or |m| / T past what quick weights take
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  DS_DEV Sampler(Shared& s) : sh(s) {}

  DS_DEV void sync() {
    if (C > 1) cluster_sync();
    else __syncthreads();
  }
  // Tell every CTA this CTA's word (the first C threads have it) and learn all of theirs.
  DS_DEV const Word* tell(const Word& w) {
    const int t = turn;
    turn ^= 1;
    if ((int)threadIdx.x < C) {
      const uint32_t at = C > 1 ? remote(&sh.in[t][rank], threadIdx.x) : smem_u32(&sh.in[t][rank]);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        st_remote_u64(at + 8 * i, w.a[i]);
        st_remote_u64(at + 24 + 8 * i, w.n[i]);
      }
      st_remote_u32(at + 48, __float_as_uint(w.f));
      st_remote_u32(at + 52, __float_as_uint(w.g));
    }
    sync();
    return sh.in[t];
  }

  // Quick weight of l but for the row's factor, fix_quick. Not for `odd` rows.
  DS_DEV float quick(float l) const { return exp2_approx(fmaf(l, c_quick, b_quick)); }

  // What masses are counted in: units of 1 / unit(), `fine` bits finer than those that fit any row.
  DS_DEV static float finer(float unit, int bits) { return unit * __int_as_float((127 + bits) << 23); }
  DS_DEV float unit() const { return finer(unit0, fine); }
  struct Sums {
    uint64_t mass[3];
    uint64_t pre[3];  // of it, in the CTAs before this one
    uint64_t n[3];
    uint64_t err;  // bound on the error of any of them (0 for exact weights)
  };
  // Over the kept tokens: for each pivot p_j (-inf: all), the mass, or else the number, of those
  // with l > p_j. p_0 >= p_1 >= p_2. J pivots are used. Per-warp sums stay in sh.wsum.
  // ALL: every token is kept. FIND: tokens from `reach` up go to the first CTA's list on the way.
  template <bool EXACT, bool MASS, int J, bool ALL = false, bool FIND = false>
  DS_DEV Sums pass(const Kept keep, const float (&piv)[3], float reach = 0.f) {
    if constexpr (FIND) {
      if (threadIdx.x == 0) sh.n_local = 0;
      __syncthreads();
    }
    float s[J], comp[J];
    uint64_t x[J];
    uint32_t n[J];
#pragma unroll
    for (int j = 0; j < J; ++j) s[j] = comp[j] = 0.f, x[j] = 0, n[j] = 0;
    const float least = fmaxf(keep.cut, piv[J - 1]);
    row.each([&](float (&v)[E], int g, float top) {
      float part[J];
      if (!FIND && top < least) return;
#pragma unroll
      for (int j = 0; j < J; ++j) part[j] = 0.f;
      const int i0 = row.index(g);
      if constexpr (FIND) {
        if (top >= reach) {
          uint32_t hits = 0;
#pragma unroll
          for (int e = 0; e < E; ++e) hits |= (uint32_t)(v[e] >= reach && v[e] > -INFINITY) << e;
          note(v, hits, i0);
        }
      }
      if constexpr (!ALL) {  // what does not stay counts as -inf
#pragma unroll
        for (int e = 0; e < E; ++e)
          v[e] = (v[e] > keep.cut) | ((v[e] == keep.cut) & (i0 + e <= keep.tie)) ? v[e] : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if constexpr (!MASS) {
#pragma unroll
          for (int j = 0; j < J; ++j) n[j] += v[e] > piv[j];
        } else if constexpr (EXACT) {
          const uint64_t w = weight_units(map, v[e], unit());
#pragma unroll
          for (int j = 0; j < J; ++j) x[j] += v[e] > piv[j] ? w : 0;
        } else {
          const float w = quick(v[e]);
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (FIND || v[e] > piv[j]) part[j] += w;
        }
      }
      if constexpr (MASS && !EXACT) {
#pragma unroll
        for (int j = 0; j < J; ++j) {  // running sum, compensated as by W. Kahan (1965)
          const float y = part[j] - comp[j], z = s[j] + y;
          comp[j] = (z - s[j]) - y;
          s[j] = z;
        }
      }
    });
    if constexpr (FIND) {
      __syncthreads();
      send_finds();
    }
    if constexpr (MASS && !EXACT) {
      const float uq = unit() * fix_quick;
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] = __float2ull_rn(s[j] * uq);
    }
    __syncthreads();  // the sums of the pass before have been read
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint64_t xs = warp_sum_u64(x[j]);
      const uint32_t ns = __reduce_add_sync(0xffffffffu, n[j]);
      if (lane == 0) sh.wsum[j][warp] = xs, sh.wn[j][warp] = ns;
    }
    __syncthreads();
    Word w{};
    if (warp == 0) {
      for (int q = 0; q < kSampleWarps; ++q) {
#pragma unroll
        for (int j = 0; j < J; ++j) w.a[j] += sh.wsum[j][q], w.n[j] += sh.wn[j][q];
      }
    }
    const Word* in = tell(w);
    Sums r{};
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        r.mass[j] += in[c].a[j], r.n[j] += in[c].n[j];
        if (c < (int)rank) r.pre[j] += in[c].a[j];
      }
    }
    if constexpr (!EXACT && MASS) {
      const float mass = __ull2float_rn(r.mass[J - 1]);
      const float bits = mass > 0.f ? log2f((float)(row.end - row.lead) * unit() / mass) : 0.f;
      r.err = __float2ull_ru(mass * (kQuickRel + kQuickArg * fmaxf(bits, 0.f)));
    }
    return r;
  }
  // Units of 2^-61 to 2^-60 of a quick mass, from units that fit any row; the mass in them.
  DS_DEV void refine(Sums& z) {
    const int up = max(0, __clzll((long long)(z.mass[0] + z.err)) - 3);
    fine += up;
    z.mass[0] <<= up, z.pre[0] <<= up, z.err <<= up;
  }
  // The kept tokens' quick mass, in units that fit any row.
  DS_DEV Sums quick_mass(const Kept keep) {
    const float p[3] = {-INFINITY, -INFINITY, -INFINITY};
    fine = 0;
    return pass<false, true, 1>(keep, p);
  }
  // Units that fit the kept tokens' mass, from exact weights.
  DS_DEV void exact_units(const Kept keep) {
    const float p[3] = {-INFINITY, -INFINITY, -INFINITY};
    fine = 0;
    Sums z = pass<true, true, 1>(keep, p);
    z.err = (uint64_t)(row.end - row.lead);
    refine(z);
  }

  // The n-th lowest index (n >= 1) with this logit, among all CTAs.
  DS_DEV int nth_index(float value, uint64_t n) {
    uint32_t c = 0;
    row.each([&](const float (&v)[E], int, float) {
#pragma unroll
      for (int e = 0; e < E; ++e) c += v[e] == value;
    });
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) sh.wn[0][warp] = c;
    if (threadIdx.x == 0) sh.pick = -1;
    __syncthreads();
    Word w{};
    if (warp == 0)
      for (int q = 0; q < kSampleWarps; ++q) w.n[0] += sh.wn[0][q];
    const Word* in = tell(w);
    uint64_t pre = 0;
    for (int q = 0; q < (int)rank; ++q) pre += in[q].n[0];
    for (int q = 0; q < warp; ++q) pre += sh.wn[0][q];
    if (pre < n && pre + sh.wn[0][warp] >= n) {  // in this warp's part
      uint32_t left = (uint32_t)(n - pre);
      for (int b = row.first; b < row.last && left; b += 32) {
        float v[E];
        uint32_t hits = 0;
        if (b + lane < row.last) {
          row.get(b + lane, v);
#pragma unroll
          for (int e = 0; e < E; ++e) hits |= (uint32_t)(v[e] == value) << e;
        }
        uint32_t cnt = __popc(hits), incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        if (all >= left) {
          if (incl >= left && incl - cnt < left) {
            uint32_t k = left - (incl - cnt);
            for (int e = 0; e < E; ++e)
              if ((hits >> e & 1) && --k == 0) sh.pick = row.index(b + lane) + e;
          }
          break;
        }
        left -= all;
      }
    }
    __syncthreads();
    Word p{};
    p.f = __int_as_float(sh.pick);
    in = tell(p);
    int at = -1;
    for (int q = 0; q < C; ++q) at = max(at, __float_as_int(in[q].f));
    return at;
  }

  // This CTA's tokens with lo < l <= hi (kept ones) into sh.extra; n_local counts them all.
  DS_DEV void find(float lo, float hi, const Kept keep) {
    if (threadIdx.x == 0) sh.n_local = 0;
    __syncthreads();
    row.each([&](const float (&v)[E], int g, float top) {
      if (!(top > lo)) return;
      uint32_t hits = 0;
      const int i0 = row.index(g);
#pragma unroll
      for (int e = 0; e < E; ++e)
        hits |= (uint32_t)(v[e] > lo && v[e] <= hi && kept(keep, v[e], i0 + e)) << e;
      note(v, hits, i0);
    });
    __syncthreads();
  }
  DS_DEV void note(const float (&v)[E], uint32_t hits, int i0) {
    if (!hits) return;
    uint32_t at = atomicAdd(&sh.n_local, (uint32_t)__popc(hits));
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (hits >> e & 1) {
        if (at < kListCap) sh.extra[at] = list_key(v[e], i0 + e);
        ++at;
      }
  }
  // All CTAs' finds to the first one's list; sh.n_list there counts them all (which may be more
  // than it holds). Ends before the cluster has met: the caller's next tell() or sync() does.
  DS_DEV void send_finds() {
    const uint32_t n = sh.n_local;
    if (threadIdx.x == 0) sh.base = C > 1 ? add_remote_u32(remote(&sh.n_list, 0), n) : atomicAdd(&sh.n_list, n);
    __syncthreads();
    const uint32_t b = sh.base;
    const uint32_t at = C > 1 ? remote(sh.list, 0) : smem_u32(sh.list);
    for (uint32_t i = threadIdx.x; i < n && i < kListCap; i += kSampleThreads)
      if (b + i < kListCap) st_remote_u64(at + 8 * (b + i), sh.extra[i]);
  }

  // The first CTA's list, a few entries a thread: keys, and exact weights in units.
  struct Entries {
    uint64_t key[kPer], w[kPer];  // key 0: none
    int n;
    float high, low;  // the largest logit and the least, but not so low that it weighs nothing
  };
  DS_DEV void take_list(Entries& t, float unit) {
    t.n = (int)min(sh.n_list, (uint32_t)kListCap);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = (int)threadIdx.x + q * kSampleThreads;
      t.key[q] = i < t.n ? sh.list[i] : 0;
      t.w[q] = t.key[q] ? weight_units(map, key_logit(t.key[q]), unit) : 0;
      if (i < t.n) sh.extra[i] = t.w[q];
    }
    float low = INFINITY, high = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (t.key[q]) {
        low = fminf(low, key_logit(t.key[q]));
        high = fmaxf(high, key_logit(t.key[q]));
      }
    low = warp_min(low);
    high = -warp_min(-high);
    __syncthreads();
    if (lane == 0) sh.wf[warp] = low, sh.wg[warp] = high;
    __syncthreads();
    for (int q = 0; q < kSampleWarps; ++q) low = fminf(low, sh.wf[q]), high = fmaxf(high, sh.wg[q]);
    t.low = fmaxf(low, m - 50.f * T_r);
    t.high = high;
  }
  // Mass of the entries whose key is at least `cut` (all threads of the CTA).
  DS_DEV uint64_t list_mass(const Entries& t, uint64_t cut) {
    uint64_t x = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) x += t.key[q] >= cut ? t.w[q] : 0;
    return total(x);
  }
  // The first entry, in the order (or in index order), at which the running sum of weights (or of
  // entries) over those with key >= cut reaches `need` (1 .. the whole sum). 256 bins along the
  // order; while the bin holds many, again over its own range (of indices, if it is a tie); then the
  // entries of the bin against one another.
  template <bool BY_INDEX, bool BY_MASS>
  DS_DEV Found select(const Entries& t, uint64_t cut, uint64_t need) {
    uint32_t cand = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (t.key[q] && t.key[q] >= cut && (!BY_MASS || t.w[q])) cand |= 1u << q;
    uint64_t before = 0;
    float vlo = t.low, vhi = t.high;
    int ilo = 0, ihi = row.end - row.lead - 1;
    int nb;
    for (int level = 0;; ++level) {
      const bool by_index = BY_INDEX || vlo == vhi;
      const float scale = 256.f / (by_index ? (float)(ihi - ilo) + 1.f : vhi - vlo);
      auto bin_of = [&](uint64_t key) {
        // (monotone in the order; anything odd, such as infinities, lands in bin 0)
        const float x = by_index ? (float)(key_index(key) - ilo) * scale : (vhi - key_logit(key)) * scale;
        return x > 0.f ? (int)fminf(x, 255.f) : 0;
      };
      if (threadIdx.x < 256) sh.bin[threadIdx.x] = 0;
      if (threadIdx.x == 0) sh.n_local = 0, sh.pick = 255;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (cand >> q & 1)
          atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bin[bin_of(t.key[q])]),
                    BY_MASS ? (unsigned long long)t.w[q] : 1ull);
      __syncthreads();
      if (warp == 0) {  // 8 bins a lane
        uint64_t c[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += c[e] = sh.bin[8 * lane + e];
        uint64_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        uint64_t run = before + incl - sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (run < need && run + c[e] >= need) {
            sh.pick = 8 * lane + e;
            sh.found.before = run;
          }
          run += c[e];
        }
      }
      __syncthreads();
      const int pick = sh.pick;
      before = sh.found.before;
      float l = INFINITY, h = -INFINITY;
      int il = INT_MAX, ih = -1;
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (cand >> q & 1) {
          if (bin_of(t.key[q]) == pick) {
            sh.at[atomicAdd(&sh.n_local, 1u)] = (uint16_t)(threadIdx.x + q * kSampleThreads);
            l = fminf(l, key_logit(t.key[q])), h = fmaxf(h, key_logit(t.key[q]));
            il = min(il, key_index(t.key[q])), ih = max(ih, key_index(t.key[q]));
          } else {
            cand &= ~(1u << q);
          }
        }
      __syncthreads();
      nb = (int)sh.n_local;
      if (nb <= 96 || level == 5) break;
      // the bin's own range
      l = warp_min(l), h = -warp_min(-h);
      il = __reduce_min_sync(0xffffffffu, il), ih = __reduce_max_sync(0xffffffffu, ih);
      if (lane == 0) {
        sh.wf[warp] = l, sh.wg[warp] = h;
        sh.wn[0][warp] = (uint32_t)il, sh.wn[1][warp] = (uint32_t)ih;
      }
      __syncthreads();
      vlo = INFINITY, vhi = -INFINITY, ilo = INT_MAX, ihi = -1;
      for (int q = 0; q < kSampleWarps; ++q) {
        vlo = fminf(vlo, sh.wf[q]), vhi = fmaxf(vhi, sh.wg[q]);
        ilo = min(ilo, (int)sh.wn[0][q]), ihi = max(ihi, (int)sh.wn[1][q]);
      }
    }
    for (int i = threadIdx.x; i < nb; i += kSampleThreads) {
      const uint64_t key = sh.list[sh.at[i]], w = sh.extra[sh.at[i]];
      uint64_t b = before;
      for (int j = 0; j < nb; ++j) {
        const uint64_t o = sh.list[sh.at[j]];
        const bool first = BY_INDEX ? (uint32_t)o > (uint32_t)key : o > key;  // (~index descends)
        if (first) b += BY_MASS ? sh.extra[sh.at[j]] : 1;
      }
      if (b < need && b + (BY_MASS ? w : 1) >= need) sh.found = Found{key, b, w};
    }
    __syncthreads();
    const Found f = sh.found;
    __syncthreads();
    return f;
  }
  // Sum over the CTA.
  DS_DEV uint64_t total(uint64_t x) {
    x = warp_sum_u64(x);
    __syncthreads();
    if (lane == 0) sh.wsum[0][warp] = x;
    __syncthreads();
    x = 0;
    for (int q = 0; q < kSampleWarps; ++q) x += sh.wsum[0][q];
    return x;
  }
  // A list of at most one entry a thread, settled by comparing all pairs: its top-k, top-p (of its
  // own mass, or of `row_mass`, in units that fit any row and known to within `err`), min-p (logits
  // from floor_l up; all_min_p: the list holds all of them) and token. False if `err` leaves the
  // border of top-p open, or the nucleus reaches past the list.
  DS_DEV bool settle_small(const SampleArgs& a, int64_t r, const Entries& t, int k, float top_p,
                           bool own, uint64_t row_mass, uint64_t err, float floor_l, bool all_min_p,
                           float u) {
    // each entry is compared by `parts` neighbouring threads
    int parts = 1;
    while (parts < 32 && t.n * parts * 2 <= kSampleThreads) parts *= 2;
    const int i = threadIdx.x / parts, first = threadIdx.x & (parts - 1);
    const bool live = i < t.n, lead = live && first == 0;
    const uint64_t key = live ? sh.list[i] : ~0ull, w = live ? sh.extra[i] : 0;
    uint64_t above = 0;
    uint32_t rank_of = 0;
    for (int j = first; j < t.n; j += parts) {
      const bool up = sh.list[j] > key;
      above += up ? sh.extra[j] : 0;
      rank_of += up;
    }
    for (int o = parts >> 1; o; o >>= 1) {
      above += __shfl_xor_sync(0xffffffffu, above, o);
      rank_of += __shfl_xor_sync(0xffffffffu, rank_of, o);
    }
    const bool high = live && key_logit(key) >= floor_l;
    bool in = live && rank_of < (uint32_t)k;
    if (top_p < 1.f) {
      const uint64_t mine = total(lead && in ? w : 0);
      const uint64_t need = own ? reach_of(top_p, mine) : in_list_units(reach_of(top_p, row_mass), a);
      const uint64_t slack = own ? 0 : ((err + 1) << a.list_fine) + kListCap;
      if (!own && mine <= need + slack) {
        // the nucleus reaches past the list, but may hold all that min_p keeps
        const uint64_t some = total(lead && high ? w : 0);
        if (!all_min_p || some + slack > need) return false;
      }
      // the border's entry is the one that reaches `need`
      const bool open = !own && need > 1 && lead && in && above < need && above + w >= need &&
                        (need - above <= slack || above + w - need <= slack);
      if (__syncthreads_or(open)) return false;
      in = in && above < need;
    }
    in = in && high;
    const uint64_t S = total(lead && in ? w : 0), need = past(u, S);  // (all have read sh.extra)
    if (lead && !in) sh.extra[i] = 0;
    __syncthreads();
    uint64_t before = 0;
    for (int j = first; j < t.n; j += parts)
      before += (uint32_t)sh.list[j] > (uint32_t)key ? sh.extra[j] : 0;  // (lower indices)
    for (int o = parts >> 1; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if (lead && in && before < need && before + w >= need) put(a, r, key_index(key), key_logit(key), S, finer(a.unit, a.list_fine));
    return true;
  }
  // The same for a longer list, by bins.
  DS_DEV bool settle_large(const SampleArgs& a, int64_t r, Entries& t, int k, float top_p, bool own,
                           uint64_t row_mass, uint64_t err, float floor_l, bool all_min_p, float u) {
    uint32_t high = 0;  // entries that min-p keeps
#pragma unroll
    for (int q = 0; q < kPer; ++q) high |= (uint32_t)(t.key[q] && key_logit(t.key[q]) >= floor_l) << q;
    uint64_t from = 1;  // the least key that stays
    if (t.n > k) from = select<false, false>(t, 1, (uint64_t)k).key;
    if (top_p < 1.f) {
      const uint64_t mine = list_mass(t, from);
      const uint64_t need = own ? reach_of(top_p, mine) : in_list_units(reach_of(top_p, row_mass), a);
      const uint64_t slack = own ? 0 : ((err + 1) << a.list_fine) + kListCap;
      if (!own && mine <= need + slack) {
        // the nucleus reaches past the list, but may hold all that min_p keeps
        uint64_t some = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) some += high >> q & 1 ? t.w[q] : 0;
        some = total(some);
        if (!all_min_p || some + slack > need) return false;
      } else {
        const Found f = select<false, true>(t, from, need);
        from = f.key;
        if (!own && need > 1 && (need - f.before <= slack || f.before + f.w - need <= slack))
          return false;
      }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (!(high >> q & 1)) t.w[q] = 0;
    const uint64_t S = list_mass(t, from);
    const Found f = select<true, true>(t, from, past(u, S));
    if (threadIdx.x == 0) put(a, r, key_index(f.key), key_logit(f.key), S, finer(a.unit, a.list_fine));
    return true;
  }
  // A mass of the row in units of the list; more than all of a list where it is that.
  DS_DEV static uint64_t in_list_units(uint64_t x, const SampleArgs& a) {
    return x >> (62 - a.list_fine) ? 1ull << 62 : x << a.list_fine;
  }
  // The running sum at which a share top_p of a whole is reached: at least 1, at most all of it.
  DS_DEV static uint64_t reach_of(float top_p, uint64_t whole) {
    if (!(top_p > 0.f)) return 1;
    return top_p < 1.f ? max(scale_mass(top_p, whole, true), (uint64_t)1) : whole;
  }
  // The running sum that the token's has to reach to exceed u S: u below 0 gives the first, 1 and
  // above (and NaN) the last.
  DS_DEV static uint64_t past(float u, uint64_t S) {
    if (u <= 0.f) return 1;
    return u < 1.f ? min(scale_mass(u, S, false) + 1, S) : S;
  }

  // The lowest logit that weighs at least min_p: 32 candidates at a time (every warp alike).
  DS_DEV float min_p_cut(float min_p) const {
    const uint64_t least = (uint64_t)(fminf(min_p, 1.f) * kListUnit);
    uint32_t lo = float_key(-INFINITY), hi = float_key(m);  // lo is too low, hi is not
    while (hi - lo > 1) {
      const uint32_t step = max((hi - lo) / 33, 1u), k = min(lo + step * (lane + 1), hi);
      const uint32_t ok = __ballot_sync(0xffffffffu, weight_units(map, key_logit((uint64_t)k << 32), kListUnit) >= least);
      const int f = ok ? __ffs(ok) - 1 : 32;
      const uint32_t a = lo + step * f;
      if (f < 32) hi = min(lo + step * (f + 1), hi);
      lo = min(a, hi - 1);
    }
    return key_logit((uint64_t)hi << 32);
  }

  // The token, its logit l, and the kept mass S in units of 1 / unit.
  DS_DEV void put(const SampleArgs& a, int64_t r, int token, float l, uint64_t S, float unit) const {
    a.token[r] = token;
    if (a.prob) {
      const float4 c = sh.map;
      a.prob[r] = weight_of(c.x, c.y, c.z, sh.table, l) * unit / __ull2float_rn(S);
    }
  }

  // The first CTA's state and cut to all.
  DS_DEV void announce(int state, Kept cut) {
    if (rank == 0 && (int)threadIdx.x < C) {
      const uint32_t at = C > 1 ? remote(&sh.state, threadIdx.x) : smem_u32(&sh.state);
      const uint32_t kc = C > 1 ? remote(&sh.cut, threadIdx.x) : smem_u32(&sh.cut);
      st_remote_u32(at, (uint32_t)state);
      st_remote_u32(kc, __float_as_uint(cut.cut));
      st_remote_u32(kc + 4, (uint32_t)cut.tie);
      if (threadIdx.x == 0) sh.n_list = 0;
    }
    sync();
  }

  // An interval (lo, hi] of logits around a cut of the order: of the kept tokens, fewer than `need`
  // (by number, or by quick mass known to within `err`) lie above hi, at least that many above lo.
  // It ends as one float wide, or with no more tokens in it than the list holds.
  struct Interval {
    float lo, hi;
    uint64_t n_hi;  // kept tokens (or their mass) above hi
    bool all;       // no cut: every token above -inf is needed
    bool ok;        // it has ended (quick masses may leave it open)
    DS_DEV bool one() const { return nextafterf(lo, INFINITY) >= hi; }
  };
  template <bool BY_MASS>
  DS_DEV Interval narrow(const Kept keep, uint64_t need, uint64_t err) {
    // g(x) = number (mass) of kept tokens above x; the cut's logit is the least x with g(x) below
    // the target. g(hi) < target <= g(lo) throughout.
    Interval v{-INFINITY, m, 0, false, false};
    uint64_t g_hi = 0, g_lo = ~0ull;  // g at hi and lo (~0: not known)
    float span = T_r, side = 0.2f;
    for (int round = 0; round < 64; ++round) {
      // how many tokens are in it: by number, or at most its mass over the least weight there
      bool few = false;
      if (g_lo != ~0ull) {
        const uint64_t in = g_lo - g_hi;
        few = BY_MASS ? (float)kListCap * __ull2float_rn(weight_units(map, v.lo, unit())) >
                            1.001f * __ull2float_rn(in + 2 * err)
                      : in <= (uint64_t)kListCap;
      }
      v.ok = few || v.one();
      if (v.ok) break;
      float p[3];
      const uint32_t kl = float_key(v.lo), kh = float_key(v.hi);
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        float x;
        if (v.lo == -INFINITY && round < 4) {
          x = v.hi - span * (j == 0 ? 4.f : (j == 1 ? 10.f : 22.f));
        } else if (v.lo > -INFINITY && round < 10) {
          // where g would meet the target if it were straight in between, and `side` to each side
          const float at = __ull2float_rn(need - min(need, g_hi)) / __ull2float_rn(g_lo - g_hi);
          x = v.hi - (v.hi - v.lo) * fminf(fmaxf(fminf(at, 1.f) + side * (float)(j - 1), 0.f), 1.f);
        } else {  // quarters of the floats between
          const uint32_t k = kh - (uint32_t)(((uint64_t)(kh - kl) * (j + 1)) >> 2);
          x = key_logit((uint64_t)k << 32);
        }
        if (!(x < v.hi)) x = nextafterf(v.hi, -INFINITY);
        if (!(x > v.lo)) x = v.lo;
        p[j] = x;
      }
      if (p[1] > p[0]) p[1] = p[0];
      if (p[2] > p[1]) p[2] = p[1];
      span *= 8.f;
      Sums s{};
      bool close = BY_MASS && odd;
      const float lo0 = v.lo;
      auto open = [&](int j) {
        const uint64_t x = s.mass[j];
        return (x > need ? x - need : need - x) <= s.err + err;
      };
      if (!close) s = keep.cut == -INFINITY ? pass<false, BY_MASS, 3, true>(keep, p)
                                            : pass<false, BY_MASS, 3>(keep, p);
      if (BY_MASS) {
        for (int j = 0; j < 3; ++j) close |= open(j);
        if (close) s = pass<true, true, 3>(keep, p);
      }
#pragma unroll
      for (int j = 0; j < 3; ++j) {  // descending pivots
        if (BY_MASS && err && open(j)) continue;  // (says nothing)
        if (BY_MASS ? s.mass[j] < need : s.n[j] < need) {
          v.hi = p[j];
          g_hi = BY_MASS ? s.mass[j] : s.n[j];
        } else {
          if (p[j] > v.lo || (p[j] == v.lo && g_lo == ~0ull)) {
            v.lo = p[j];
            g_lo = BY_MASS ? s.mass[j] : s.n[j];
          }
          break;
        }
      }
      // the straighter the shorter: sides shrink as long as they hold the target
      if (lo0 > -INFINITY) side = v.lo >= p[2] && v.hi <= p[0] ? side * 0.25f : 0.25f;
      if (v.hi == -INFINITY) {
        v.all = v.ok = true;
        break;
      }
    }
    v.n_hi = g_hi;
    return v;
  }

  // The tokens that share the logit hi (all there is in the interval): those of them that stay, to
  // take `left` tokens (or mass).
  template <bool BY_MASS>
  DS_DEV Kept cut_tie(const Interval& v, const Kept keep, uint64_t left) {
    const float p[3] = {v.hi, v.lo, v.lo};
    const Sums s = pass<false, false, 2>(keep, p);
    const uint64_t n_tie = s.n[1] - s.n[0];
    uint64_t n = left;
    if (BY_MASS) {
      const uint64_t w = weight_units(map, v.hi, unit());
      n = w ? (left + w - 1) / w : n_tie;
    }
    if (n >= n_tie) return Kept{v.hi, v.hi == keep.cut ? keep.tie : INT_MAX};
    return Kept{v.hi, nth_index(v.hi, n)};
  }

  // The cut after `left` tokens (or that mass) of the interval, by the first CTA's list.
  template <bool BY_MASS>
  DS_DEV Kept cut_list(const Interval& v, const Kept keep, uint64_t left) {
    find(v.lo, v.hi, keep);
    send_finds();
    sync();
    Kept cut{v.hi, INT_MAX};
    if (rank == 0) {
      Entries t;
      take_list(t, unit());
      Found f;
      if (BY_MASS) f = select<false, true>(t, 1, min(left, list_mass(t, 1)));
      else f = select<false, false>(t, 1, left);
      cut = Kept{key_logit(f.key), key_index(f.key)};
    }
    announce(kCut, cut);
    cut = sh.cut;
    return cut;
  }

  // After the first `need` kept tokens.
  DS_DEV Kept cut_by_number(const Kept keep, uint64_t need) {
    const Interval v = narrow<false>(keep, need, 0);
    if (v.all) return keep;
    return v.one() ? cut_tie<false>(v, keep, need - v.n_hi)
                   : cut_list<false>(v, keep, need - v.n_hi);
  }

  // After the first token at which the kept mass reaches top_p of all of it; and, since one exact
  // pass then has nearly all that it takes, the token. True: done; false: *cut is the cut.
  DS_DEV bool cut_by_mass(const SampleArgs& a, int64_t r, const Kept keep, float top_p, const Sums& z,
                          float floor_l, float u, Kept* cut) {
    const float lowest = -INFINITY;
    Interval v;
    uint64_t above_hi, need;
    // the interval by quick masses; if it turns out off by exact ones, by these
    for (int exact = odd; ; exact = 1) {
      if (exact) {
        const float p[3] = {lowest, lowest, lowest};
        need = reach_of(top_p, pass<true, true, 1>(keep, p).mass[0]);
        v = narrow<true>(keep, need, 0);
      } else {
        v = narrow<true>(keep, reach_of(top_p, z.mass[0]), z.err + 1);
      }
      if (!v.ok && !exact) continue;
      if (v.all) {
        *cut = keep;
        return false;
      }
      const float p[3] = {v.hi, v.lo, lowest};
      const Sums s = keep.cut == -INFINITY ? pass<true, true, 3, true>(keep, p) : pass<true, true, 3>(keep, p);
      need = reach_of(top_p, s.mass[2]);
      above_hi = s.mass[0];
      if (exact || (above_hi < need && need <= s.mass[1])) {
        above_hi = min(above_hi, need - 1);
        break;
      }
    }
    const uint64_t w_hi = sh.wsum[0][warp];  // this warp's part of above_hi
    const uint64_t left = need - above_hi;
    *cut = v.one() ? cut_tie<true>(v, keep, left) : cut_list<true>(v, keep, left);
    if (floor_l > cut->cut) return false;  // min_p cuts higher
    // per-warp masses of what stays: that above hi, and what the cut leaves of the interval
    uint64_t x = 0;
    row.each([&](const float (&l)[E], int g, float top) {
      if (top < cut->cut) return;
      const int i0 = row.index(g);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (l[e] <= v.hi && kept(*cut, l[e], i0 + e)) x += weight_units(map, l[e], unit());
    });
    x = warp_sum_u64(x) + w_hi;
    __syncthreads();
    if (lane == 0) sh.wsum[0][warp] = x;
    __syncthreads();
    Word w{};
    if (warp == 0)
      for (int q = 0; q < kSampleWarps; ++q) w.a[0] += sh.wsum[0][q];
    const Word* in = tell(w);
    uint64_t before = 0, all = 0;
    for (int c = 0; c < C; ++c) {
      if (c < (int)rank) before += in[c].a[0];
      all += in[c].a[0];
    }
    finish<true>(a, r, *cut, before, all, 0, u);
    return true;
  }

  // The token of a row whose kept set is known, by a pass: quick weights (false: too close to a
  // border; the units fit the kept mass from then on) or exact ones, in the present units.
  template <bool EXACT>
  DS_DEV bool locate(const SampleArgs& a, int64_t r, const Kept keep, float u) {
    const float p[3] = {-INFINITY, -INFINITY, -INFINITY};
    if (!EXACT) fine = 0;
    Sums s = keep.cut == -INFINITY ? pass<EXACT, true, 1, true>(keep, p) : pass<EXACT, true, 1>(keep, p);
    // (quick weights are rounded to these units one by one when the token is looked for)
    if (!EXACT) s.err += (uint64_t)(row.end - row.lead);
    if (finish<EXACT>(a, r, keep, s.pre[0], s.mass[0], s.err, u)) return true;
    refine(s);
    return false;
  }
  // The same from the kept mass S, known to within err, that of the CTAs before this one, and its
  // warps' (sh.wsum[0]).
  template <bool EXACT>
  DS_DEV bool finish(const SampleArgs& a, int64_t r, const Kept keep, uint64_t before, uint64_t S,
                     uint64_t err, float u) {
    const uint64_t need = past(u, S);
    const uint64_t slack = 2 * err + 1;  // the borders and u S are each off by no more than err
    if (!EXACT && (need <= slack || S - need <= slack)) return false;  // (also u out of range)
    // the warp's part that holds the token (if it is in this CTA), and of this its sixteenth
    int part = -1;
    for (int q = 0; q < kSampleWarps; ++q) {
      const uint64_t x = sh.wsum[0][q];
      if (before < need && before + x >= need) {
        part = q;
        break;
      }
      before += x;
    }
    bool here = false;
    int from = 0, to = 0;
    const float uq = unit() * fix_quick;
    auto units_of = [&](float l, int i) -> uint64_t {
      if (!(l > -INFINITY) || !kept(keep, l, i)) return 0;
      if (EXACT) return weight_units(map, l, unit());
      return __float2ull_rn(quick(l) * uq);
    };
    if (part >= 0) {
      const int f = min(row.g1, row.g0 + part * row.wper), l = min(row.g1, f + row.wper);
      const int sub = ((l - f + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
      from = min(l, f + warp * sub);
      to = min(l, from + sub);
      uint64_t x = 0;
      for (int g = from + lane; g < to; g += 32) {
        float v[E];
        row.get(g, v);
        const int i0 = row.index(g);
#pragma unroll
        for (int e = 0; e < E; ++e) x += units_of(v[e], i0 + e);
      }
      x = warp_sum_u64(x);
      __syncthreads();
      if (lane == 0) sh.wsum[1][warp] = x;
      __syncthreads();
      for (int q = 0; q < warp; ++q) before += sh.wsum[1][q];
      here = before < need && before + x >= need;
    }
    int verdict = 0;
    if (here) {
      int token = -1;
      uint64_t cum = before;
      bool sure = false;
      for (int b = from; b < to; b += 32) {
        float v[E];
        uint64_t x[E], run = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = -INFINITY;
        if (b + lane < to) row.get(b + lane, v);
        const int i0 = row.index(b + lane);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[e] = units_of(v[e], i0 + e);
          run += x[e];
        }
        uint64_t incl = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, cum + incl >= need);
        if (hit) {
          const int src = __ffs(hit) - 1;
          uint64_t c = cum + incl - run;
          if (lane == src) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              if (token < 0 && c + x[e] >= need) {
                token = i0 + e;
                sure = need - c > slack && c + x[e] - need > slack;
              }
              c += x[e];
            }
          }
          token = __shfl_sync(0xffffffffu, token, src);
          sure = __shfl_sync(0xffffffffu, (int)sure, src) != 0;
          break;
        }
        cum += __shfl_sync(0xffffffffu, incl, 31);
      }
      if ((EXACT || sure) && token >= 0) {
        verdict = 1;
        // (a quick S is good to 2^-20)
        if (lane == 0) put(a, r, token, to_f32(row.base[row.lead + token]), S, unit());
      }
    }
    if (EXACT) return true;
    const int any = __syncthreads_or(verdict);
    Word w{};
    w.f = any ? 1.f : 0.f;
    const Word* in = tell(w);
    bool done = false;
    for (int c = 0; c < C; ++c) done |= in[c].f != 0.f;
    return done;
  }

  DS_DEV void run(const SampleArgs& a, int64_t r, uint4* share, int cluster, uint32_t rk) {
    C = cluster;
    rank = rk;
    unit0 = a.unit;
    const int V = a.vocab;
    const T* start = static_cast<const T*>(a.logits) + r * a.stride;
    row.lead = (int)((reinterpret_cast<uintptr_t>(start) & 15) / sizeof(T));
    row.base = start - row.lead;
    row.end = row.lead + V;
    row.smem = share;
    const int groups = (row.end + E - 1) / E, per = a.chunk / E;
    row.g0 = min(groups, (int)rank * per);
    row.g1 = min(groups, row.g0 + per);
    row.wper = ((row.g1 - row.g0 + kSampleWarps - 1) / kSampleWarps + 31) / 32 * 32;
    row.first = min(row.g1, row.g0 + warp * row.wper);
    row.last = min(row.g1, row.first + row.wper);
    row.edge = sh.edge;
    row.full0 = row.lead ? 1 : 0;
    row.full1 = row.end / E;
    // (before the cluster meets: only then is the row's token written)
    const int left = MODE == kRest ? a.token[r] - kLater : 0;
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.n_list = 0;
    // no CTA writes into another's shared memory before that one runs (waited for below)
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    T_r = a.temperature ? a.temperature[r] : 1.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    const float top_p = a.top_p ? a.top_p[r] : 1.f, min_p = a.min_p ? a.min_p[r] : 0.f;
    const float u = a.u[r];
    const bool greedy = !(T_r > 0.f), by_k = !greedy && k > 0 && k < V, by_p = !greedy && top_p < 1.f;
    const int most = C == 1 ? 448 : (C == 2 ? 768 : 1024);
    const bool list = MODE != kRest && ((by_k && k <= most) || (!by_k && by_p));
    const int want = by_k ? k : most;

    // the one read of the row: a thread's maximum on the way
    float tmax = -INFINITY;
    auto take = [&](uint4 q, int g) {
      q = R::clean(q);
      if constexpr (RES) row.smem[g - row.g0] = q;
      tmax = fmaxf(tmax, R::most(q));
    };
    // eight loads a thread in flight, with no branch between them (groups that the row fills; its
    // first and last may be partly filled: those by element, by the thread that reads them later)
    constexpr int U = 8;
    const int full0 = row.full0, full1 = row.full1;
    const uint4* src = reinterpret_cast<const uint4*>(row.base);
    for (int b = row.first + lane; b < row.last; b += 32 * U) {
      uint4 q[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int g = b + 32 * i;
        if (g >= full0 && g < full1 && g < row.last) q[i] = __ldg(src + g);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int g = b + 32 * i;
        if (g >= full0 && g < full1 && g < row.last) take(q[i], g);
      }
    }
    for (int e = 0; e < 2; ++e) {
      const int g = e ? full1 : 0;
      if ((e || full0) && (!e || g >= full0) && g >= row.first && g < row.last &&
          lane == ((g - row.first) & 31)) {
        const uint4 q = row.fetch(g);
        sh.edge[e] = q;
        if (full1 == 0) sh.edge[1] = q;  // (both ends)
        take(q, g);
      }
    }
    if (threadIdx.x < 33) sh.table[threadIdx.x] = kExp2Table[threadIdx.x];
    // this CTA's maximum, and a logit that at least want / C of its tokens reach: the threads'
    // maxima in 256 bins between the least and the largest
    float hi = tmax, lo = tmax == -INFINITY ? INFINITY : tmax;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane == 0) sh.wf[warp] = hi, sh.wg[warp] = lo;
    __syncthreads();
    for (int q = 0; q < kSampleWarps; ++q) hi = fmaxf(hi, sh.wf[q]), lo = fminf(lo, sh.wg[q]);
    float reach = -INFINITY;
    if (list) {
      const uint32_t need = (uint32_t)((want + C - 1) / C);
      int bin = -1;
      const float scale = 255.f / (hi - lo);  // (0 / 0 and infinities fall to bin 0 below)
      if (tmax > -INFINITY) {
        const float x = (tmax - lo) * scale;
        bin = x > 0.f ? min(255, (int)x) : 0;
        atomicAdd(&sh.hist[bin], 1u);
      }
      if (threadIdx.x == 0) sh.pick = -1;
      __syncthreads();
      if (warp == 0) {  // the highest bin with `need` threads in it and above: 8 bins a lane
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += c[e] = sh.hist[255 - (8 * lane + e)];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        uint32_t run = incl - sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (run < need && run + c[e] >= need) sh.pick = 255 - (8 * lane + e);
          run += c[e];
        }
      }
      __syncthreads();
      const int pick = sh.pick;  // -1: fewer threads than that have a token at all
      float x = pick >= 0 && bin >= pick ? tmax : INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, o));
      __syncthreads();
      if (lane == 0) sh.wf[warp] = x;
      __syncthreads();
      reach = INFINITY;
      for (int q = 0; q < kSampleWarps; ++q) reach = fminf(reach, sh.wf[q]);
      if (pick < 0) reach = -INFINITY;
    }
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    {
      Word w{};
      w.f = hi;
      w.g = reach;
      const Word* in = tell(w);
      for (int c = 0; c < C; ++c) hi = fmaxf(hi, in[c].f), reach = fminf(reach, in[c].g);
    }
    m = hi;
    if (m == -INFINITY) {  // nothing to choose from
      if (rank == 0 && threadIdx.x == 0) {
        a.token[r] = -1;
        if (a.prob) a.prob[r] = 0.f;
      }
      return;
    }
    if (greedy) {
      const int at = nth_index(m, 1);
      if (rank == 0 && threadIdx.x == 0) {
        a.token[r] = at;
        if (a.prob) a.prob[r] = 1.f;
      }
      return;
    }
    map = weight_map(m, T_r, sh.table);
    if (threadIdx.x == 0) sh.map = make_float4(map.m, map.c_hi, map.c_lo, 0.f);
    {
      const float mc = m * map.c_hi;
      odd = !(fabsf(mc) < 4194304.f);  // 2^22: the rounding below is 2^-3 at most
      c_quick = fmaxf(map.c_hi, 1e-37f);
      b_quick = -mc;
      fix_quick = exp2f(-__fmaf_rn(m, map.c_hi, b_quick));
    }
    const Kept all{-INFINITY, INT_MAX};
    Kept keep = all;
    Sums z{};  // the row's quick mass
    const float floor_l = min_p > 0.f ? min_p_cut(min_p) : -INFINITY;
    if (MODE != kRest && list) {
      // with top-p alone, what min_p drops need not be in the list: its mass is in the row's
      if (!by_k) reach = fmaxf(reach, floor_l);
      const bool all_min_p = min_p > 0.f && floor_l >= reach;
      // tokens from `reach` up to the first CTA; for top-p alone, the row's mass in the same pass
      if (by_k) {
        find(reach == -INFINITY ? reach : nextafterf(reach, -INFINITY), INFINITY, all);
        send_finds();
        sync();
      } else {
        const float p[3] = {-INFINITY, -INFINITY, -INFINITY};
        z = pass<false, true, 1, true, true>(all, p, reach);
      }
      int state = kOpen;
      Kept cut = all;
      const uint32_t found = sh.n_list;
      __syncthreads();  // (announce() clears it)
      if (rank == 0 && found <= (uint32_t)kListCap) {
        Entries t;
        take_list(t, finer(a.unit, a.list_fine));
        // the mass that top_p is a share of is known exactly if it is the list's: that of its first
        // k tokens, or of the whole row if that is what the list holds
        const bool own = by_k || reach == -INFINITY;
        const int kk = by_k ? k : t.n;
        if (own || !odd) {
          const bool ok = t.n <= kSampleThreads
                              ? settle_small(a, r, t, kk, top_p, own, z.mass[0], z.err, floor_l, all_min_p, u)
                              : settle_large(a, r, t, kk, top_p, own, z.mass[0], z.err, floor_l, all_min_p, u);
          if (ok) state = kDone;
        }
      }
      announce(state, cut);
      if (sh.state == kDone) return;
    }
    if constexpr (MODE == kQuick) {
      if (floor_l > keep.cut) keep = Kept{floor_l, INT_MAX};
      if (!by_k && !by_p && !odd && locate<false>(a, r, keep, u)) return;
      if (rank == 0 && threadIdx.x == 0) a.token[r] = kLater + fine;
      return;
    } else {
      if (by_k) keep = cut_by_number(keep, (uint64_t)k);
      if (by_p) {
        if (odd) {
          exact_units(keep);
        } else {
          if (!list || by_k) z = quick_mass(keep);  // (else taken with the list)
          refine(z);
        }
        bool within = false;  // all that min_p keeps has less than top_p of the mass
        if (floor_l > keep.cut && !odd) {
          const float p[3] = {-INFINITY, -INFINITY, -INFINITY};
          const Sums s = pass<false, true, 1>(Kept{floor_l, INT_MAX}, p);
          const uint64_t need = reach_of(top_p, z.mass[0]);
          within = s.mass[0] + s.err + z.err + 1 < need;
        }
        if (!within && cut_by_mass(a, r, keep, top_p, z, floor_l, u, &keep)) return;
      }
      if (floor_l > keep.cut) keep = Kept{floor_l, INT_MAX};
      if (odd) exact_units(keep);
      // (a row without a cut was left because quick weights leave its token open)
      else if (MODE == kRest && !by_k && !by_p) fine = left;
      else if (locate<false>(a, r, keep, u)) return;
      locate<true>(a, r, keep, u);
    }
  }
};

template <typename T, bool RES, int MODE>
__global__ void __launch_bounds__(kSampleThreads, MODE == kQuick ? 2 : 1) k_sample_logits(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  pdl_wait();
  uint32_t size;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
  const uint32_t rank = size > 1 ? cluster_ctarank() : 0u;
  uint4* share = reinterpret_cast<uint4*>(dyn + kSharedBytes);
  int64_t r = blockIdx.x / size;
  if constexpr (MODE != kRest) {
    if (a.done && a.done[r]) return;  // the whole cluster
    Sampler<T, RES, MODE> s(sh);
    s.run(a, r, share, (int)size, rank);
  } else {
    // every cluster takes the rows left among its own, one in gridDim / size: only it writes their
    // tokens, and not before all its CTAs have looked at them
    __shared__ uint32_t left[kSampleWarps];
    const int64_t step = gridDim.x / size;
    for (int64_t r0 = r; r0 < a.rows; r0 += step * kSampleThreads) {
      const int64_t mine = r0 + step * threadIdx.x;
      const bool is = mine < a.rows && !(a.done && a.done[mine]) && a.token[mine] <= kLater + kMassBits;
      const uint32_t set = __ballot_sync(0xffffffffu, is);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) left[threadIdx.x >> 5] = set;
      __syncthreads();
#pragma unroll 1
      for (int w = 0; w < kSampleWarps; ++w)
#pragma unroll 1
        for (uint32_t m = left[w]; m; m &= m - 1) {
          Sampler<T, RES, MODE> s(sh);
          s.run(a, r0 + step * (32 * w + __ffs(m) - 1), share, (int)size, rank);
          s.sync();
        }
    }
  }
}

}  // namespace

template <typename T, int MODE>
cudaError_t prepare_rows() {
  cudaError_t e = cudaFuncSetAttribute(k_sample_logits<T, true, MODE>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSharedBytes + kResidentMax);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_sample_logits<T, false, MODE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedBytes);
  return e;
}

// Shares stay in shared memory where two CTAs an SM hold theirs (64 KB each), or one does and there
// is one; else they are read again from L2 in each pass.
template <typename T, int MODE>
cudaError_t launch_rows(SampleArgs q, int C, int64_t clusters, int sms, cudaStream_t st) {
  constexpr int es = (int)sizeof(T), per16 = 16 / es;
  const int64_t groups = ((int64_t)q.vocab + 2 * per16 - 2) / per16;  // with the longest lead
  q.chunk = (int)((groups + C - 1) / C) * per16;
  const int64_t share = (int64_t)q.chunk * es;
  const bool res = share <= 65536 + 512 || (share <= kResidentMax && clusters * C <= sms);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSampleThreads);
  cfg.gridDim = dim3((unsigned)(clusters * C));
  cfg.dynamicSmemBytes = kSharedBytes + (res ? (size_t)share : 0);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = (unsigned)C;
  attr[n].val.clusterDim.y = 1;
  attr[n++].val.clusterDim.z = 1;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return res ? cudaLaunchKernelEx(&cfg, k_sample_logits<T, true, MODE>, q)
             : cudaLaunchKernelEx(&cfg, k_sample_logits<T, false, MODE>, q);
}
#endif  // DS_SAMPLE_KERNELS

}  // namespace sample
}  // namespace ds
