// The row and table sides of the 8-bit output head on sm_103a: a root-mean-square norm that adds
// the residual and writes its rows in 8 bits, and the 8-bit form of a matrix.
//
//   h = rnd(x + residual)            rnd: to the tensors' own type, so that the norm sees exactly
//                                    what the residual stream carries on
//   y = h / sqrt(mean(h^2) + eps) (offset + w)
//   per block: s = max(max |y|, 2^-100) / F,  q = rnd8(y / s),  F = 448 (e4m3) or 57344 (e5m2)
// Sums and products in fp32; q to nearest even, saturating. bf16 values often lie halfway between
// two codes, and any rounding on the way tips them: y / s is formed as y F / max with F / max as a
// float pair, so that what is rounded to a code is the quotient rounded to fp32 once. In the norm
// 1 / sqrt(mean + eps) divides out of it but for a power of two, so the codes do not see its rounding
// either (only that of h (offset + w)). The floor of 2^-100 keeps s and 1/s finite for blocks of zeros.
//
// Both kernels touch each byte once. The table's quantisation is bound by memory (262144 x 2816 bf16:
// 322 us, 6.9 TB/s). The norm is too where a row is a warp's (65536 x 256 fp32: 36 us, 6.1 TB/s);
// longer rows pay for the sum across warps and about 30 instructions a value (65536 x 2816 bf16 with
// a residual: 256 us, 5.0 TB/s; 16001 x 5000: 117 us, 4.8 TB/s; one row: 2.4 us).
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "ds_head.h"

namespace ds {
namespace {

constexpr float kTinyMax = 7.888609052210118e-31f;  // 2^-100

// Eight consecutive values of a row as they lie in memory.
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};

// Columns c .. c + 7 of a row of n (zeros past its end); VEC: the row is 16-byte aligned. (At the end
// of the longest row c + 8 passes 2^31; n - c and n - 8 stay below.)
template <typename T, bool VEC>
DS_DEV Raw8<T> load8(const T* row, int c, int n) {
  Raw8<T> t;
  if (VEC && c <= n - 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(row + c)[i];
      t.w[4 * i] = q.x, t.w[4 * i + 1] = q.y, t.w[4 * i + 2] = q.z, t.w[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) {
        t.w[i] = i < n - c ? __float_as_uint(row[c + i]) : 0u;
      } else {
        const uint32_t v =
            i < n - c ? (uint32_t)reinterpret_cast<const unsigned short*>(row)[c + i] : 0u;
        t.w[i >> 1] = i & 1 ? t.w[i >> 1] | v << 16 : v;
      }
    }
  }
  return t;
}

template <typename T, bool VEC>
DS_DEV void store8(T* row, int c, int n, const Raw8<T>& t) {
  if (VEC && c <= n - 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(row + c)[i] =
          make_uint4(t.w[4 * i], t.w[4 * i + 1], t.w[4 * i + 2], t.w[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n - c) {
        if constexpr (sizeof(T) == 4) row[c + i] = __uint_as_float(t.w[i]);
        else reinterpret_cast<unsigned short*>(row)[c + i] = (unsigned short)(t.w[i >> 1] >> (16 * (i & 1)));
      }
  }
}

template <typename T>
DS_DEV void unpack8(const Raw8<T>& t, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(t.w[i]);
    else f[i] = __uint_as_float(i & 1 ? t.w[i >> 1] & 0xffff0000u : t.w[i >> 1] << 16);
  }
}

// Rounds f to T, in place, and packs it.
template <typename T>
DS_DEV Raw8<T> round8(float (&f)[8]) {
  Raw8<T> t;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      t.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    unpack8(t, f);
  }
  return t;
}

// F / m as a float pair: good to 2^-44 of itself, which is the remainder's own rounding.
struct Factor {
  float hi, lo;
};
DS_DEV Factor block_factor(float m, float top) {
  const float r = __frcp_rn(m), hi = top * r;
  return Factor{hi, isinf(m) ? 0.f : __fmaf_rn(-hi, m, top) * r};
}

// Two products, or two multiply-adds, in one instruction: what issues is what these kernels wait for.
DS_DEV float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
DS_DEV float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Codes of y * f in columns c .. c + 7 of a row of n codes; VEC: the row is 8-byte aligned.
template <bool VEC, bool E5M2>
DS_DEV void store_codes(uint8_t* row, int c, int n, const float (&y)[8], const Factor f) {
  constexpr __nv_fp8_interpretation_t kind = E5M2 ? __NV_E5M2 : __NV_E4M3;
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(y[2 * i], y[2 * i + 1]);
    const float2 v = fma2(x, make_float2(f.hi, f.hi), mul2(x, make_float2(f.lo, f.lo)));
    p[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, kind);
  }
  const uint32_t w[2] = {p[0] | (p[1] << 16), p[2] | (p[3] << 16)};
  if (VEC && c <= n - 8) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n - c) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Largest |y| over the 16 threads that hold a block's 128 columns.
DS_DEV float amax16(const float (&y)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));  // fmaxf passes over NaN
#pragma unroll
  for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

struct NormArgs {
  const void *x, *residual, *weight;
  void* h;
  uint8_t* q;
  float* scales;
  int64_t rows, x_stride, r_stride, h_stride, q_stride, s_stride;
  int d;
  float eps, offset, top, rtop, rd;  // rtop = 1 / top, rd = 1 / d
  int e5m2;
};

// One row per blockDim.x threads (a multiple of 32, so that a 128-column block is 16 neighbouring
// lanes), blockDim.y rows a CTA at a time. A row stays in registers between the sum of squares and
// the output, NV groups of 8 columns a thread, all of whose loads are in flight at once; the weight
// stays there over all rows of the CTA, and the next row is fetched meanwhile (NV <= 2).
template <typename T, bool VEC, int NV, bool E5M2>
__global__ void __launch_bounds__(NV == 1 ? 1024 : (NV == 2 ? 384 : 512), NV == 2 ? 2 : 1)
    k_rmsnorm_fp8(const NormArgs a) {
  __shared__ float part[2][32];
  pdl_wait();
  const int tpr = blockDim.x, d = a.d, wpr = tpr >> 5, w0 = threadIdx.y * wpr;
  const int lane = threadIdx.x & 31;
  auto col = [&](int j) { return 8 * ((int)threadIdx.x + j * tpr); };
  constexpr bool KEEP = NV <= 2;
  float g[KEEP ? NV : 1][8];
  auto weight = [&](int j, float (&w)[8]) {
    unpack8(load8<T, VEC>(static_cast<const T*>(a.weight), col(j), d), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = col(j) + i < d ? w[i] + a.offset : 0.f;
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < NV; ++j) weight(j, g[j]);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t r0 = (int64_t)blockIdx.x * blockDim.y;
  Raw8<T> t[NV], res[NV];
  auto fetch = [&](int64_t r) {
    if (r >= a.rows) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      t[j] = load8<T, VEC>(static_cast<const T*>(a.x) + r * a.x_stride, col(j), d);
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        res[j] = load8<T, VEC>(static_cast<const T*>(a.residual) + r * a.r_stride, col(j), d);
    }
  };
  if constexpr (KEEP) fetch(r0 + threadIdx.y);
  // all threads of a CTA stay for its barriers while any of its rows is left
  for (int turn = 0; r0 < a.rows; ++turn, r0 += step) {
    const int64_t r = r0 + threadIdx.y;
    const bool live = r < a.rows;
    float h[NV][8];
    float ss = 0.f;
    if (live) {
      if constexpr (!KEEP) fetch(r);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        unpack8(t[j], h[j]);
        if (a.residual) {
          float f[8];
          unpack8(res[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] += f[i];
          t[j] = round8<T>(h[j]);
        }
        if (a.h) store8<T, VEC>(static_cast<T*>(a.h) + r * a.h_stride, col(j), d, t[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
      }
    }
    if constexpr (KEEP) fetch(r + step);  // the next row is on its way from here
    ss = warp_sum(ss);
    if (wpr > 1) {
      if (lane == 0) part[turn & 1][w0 + (threadIdx.x >> 5)] = ss;
      __syncthreads();
      ss = warp_sum(lane < wpr ? part[turn & 1][w0 + lane] : 0.f);
    }
    if (!live) continue;
    // 1 / sqrt(mean + eps) = r2 t, r2 a power of two (or 0, inf or NaN, with t = 1)
    const float rinv = 1.0f / sqrtf(ss * a.rd + a.eps);
    const uint32_t rb = __float_as_uint(rinv);
    const float r2 = isnan(rinv) ? rinv : __uint_as_float(rb & 0x7f800000u);
    const float t1 = __uint_as_float((rb & 0x007fffffu) | 0x3f800000u);
    const float least = __fdividef(kTinyMax, t1);  // the floor of max |y|, over t
    uint8_t* q = a.q + r * a.q_stride;
    float* scales = a.scales + r * a.s_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j);
      if constexpr (!KEEP) weight(j, g[0]);
      float (&w)[8] = g[KEEP ? j : 0];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {  // y / t1
        const float2 v = mul2(mul2(make_float2(h[j][i], h[j][i + 1]), make_float2(r2, r2)),
                              make_float2(w[i], w[i + 1]));
        h[j][i] = v.x, h[j][i + 1] = v.y;
      }
      const float m = amax16(h[j]);
      if ((threadIdx.x & 15) == 0 && c < d) scales[c / kScaleBlock] = fmaxf(m * t1, kTinyMax) * a.rtop;
      if (c < d) store_codes<VEC, E5M2>(q, c, d, h[j], block_factor(fmaxf(m, least), a.top));
    }
  }
}

struct QuantArgs {
  const void* x;
  uint8_t* q;
  float* scales;
  int64_t rows, x_stride, q_stride, s_stride;
  int cols;
  float top;
  int e5m2;
};

template <typename T>
DS_DEV float amax8(const Raw8<T>& t) {
  float m = 0.f;
  if constexpr (sizeof(T) == 2) {  // in pairs; the maximum of a NaN and a number is the number
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(t.w);
    const __nv_bfloat162 x = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])),
                                     __hmax2(__habs2(p[2]), __habs2(p[3])));
    m = fmaxf(fmaxf(__low2float(x), __high2float(x)), m);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(__uint_as_float(t.w[i])));
  }
  return m;
}

// One 128 x 128 block a CTA of 256 threads: 16 threads across, 16 rows at a time, 8 loads of 8
// columns in flight a thread, four CTAs an SM for bf16 (262144 x 2816: 324 us; three, 354). ROWS:
// each row of the block has its own scale. Blocks go to CTAs along the rows of x, so that the CTAs
// that run together read whole rows.
template <typename T, bool VEC, bool ROWS, bool E5M2>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) k_quantize_fp8(const QuantArgs a) {
  __shared__ float part[8];
  pdl_wait();
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int64_t ncb = ((int64_t)a.cols + kScaleBlock - 1) / kScaleBlock;
  const int64_t n = ncb * ((a.rows + kScaleBlock - 1) / kScaleBlock);
  for (int64_t blk = blockIdx.x; blk < n; blk += gridDim.x) {
    const int64_t rb = blk / ncb, r0 = rb * kScaleBlock;
    const int cb = (int)(blk - rb * ncb);
    const int c = cb * kScaleBlock + 8 * cx;
    Raw8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + ry + 16 * i;
      v[i] = load8<T, VEC>(static_cast<const T*>(a.x) + r * a.x_stride, r < a.rows ? c : a.cols, a.cols);
    }
    Factor f{};
    if constexpr (!ROWS) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      __syncthreads();  // the maxima of the block before have been read
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, part[w]);
      m = fmaxf(m, kTinyMax);
      f = block_factor(m, a.top);
      if (threadIdx.x == 0) a.scales[rb * a.s_stride + cb] = __fdiv_rn(m, a.top);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + ry + 16 * i;
      if constexpr (ROWS) {
        float m = amax8(v[i]);
#pragma unroll
        for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = fmaxf(m, kTinyMax);
        f = block_factor(m, a.top);
        if (cx == 0 && r < a.rows) a.scales[r * a.s_stride + cb] = __fdiv_rn(m, a.top);
      }
      if (r < a.rows && c < a.cols) {
        float y[8];
        unpack8(v[i], y);
        store_codes<VEC, E5M2>(a.q + r * a.q_stride, c, a.cols, y, f);
      }
    }
  }
}

bool on16(const void* p, int64_t stride_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride_bytes % 16 == 0;
}
bool on8(const void* p, int64_t stride_bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 7) == 0 && stride_bytes % 8 == 0;
}
float top_of(int fp8) { return fp8 == DS_FP8_E5M2 ? 57344.f : 448.f; }

template <typename T, bool VEC>
cudaError_t norm_nv(int nv, dim3 grid, dim3 block, cudaStream_t st, const NormArgs& n) {
  auto go = [&](auto e4m3, auto e5m2) {
    return launch_k(n.e5m2 ? e5m2 : e4m3, grid, block, 0, st, n);
  };
  if (nv == 1) return go(k_rmsnorm_fp8<T, VEC, 1, false>, k_rmsnorm_fp8<T, VEC, 1, true>);
  if (nv == 2) return go(k_rmsnorm_fp8<T, VEC, 2, false>, k_rmsnorm_fp8<T, VEC, 2, true>);
  if (nv == 4) return go(k_rmsnorm_fp8<T, VEC, 4, false>, k_rmsnorm_fp8<T, VEC, 4, true>);
  return go(k_rmsnorm_fp8<T, VEC, 8, false>, k_rmsnorm_fp8<T, VEC, 8, true>);
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const ds_rmsnorm_fp8_args& a, cudaStream_t st) {
  const int es = a.dtype == DS_DTYPE_FP32 ? 4 : 2;
  NormArgs n{a.x, a.residual, a.weight, a.h, a.q, a.scales, a.rows, a.x_stride, a.residual_stride,
             a.h_stride, a.q_stride, a.scales_stride, a.d, a.eps, a.weight_offset, top_of(a.fp8),
             1.f / top_of(a.fp8), 1.f / (float)a.d, a.fp8 == DS_FP8_E5M2};
  const bool vec = on16(a.x, a.x_stride * es) && (!a.residual || on16(a.residual, a.residual_stride * es)) &&
                   (!a.h || on16(a.h, a.h_stride * es)) && on16(a.weight, 0) && on8(a.q, a.q_stride);
  const int groups = (a.d + 7) / 8;
  // Groups of 8 columns a thread: one, unless a row then takes 513 to 768 threads, of which an SM
  // holds one row only (at 64 registers a thread): two then, and two rows (at 80). Measured, bf16
  // with a residual, one group: 65536 x 2816 257 us, 16384 x 8192 169 us, 16001 x 5000 187 us; two:
  // 16001 x 5000 117 us (one row an SM, 128 registers: 140). More where a row has more than 8192
  // columns.
  int nv = groups > 512 && groups <= 768 ? 2 : 1;
  if (groups > 1024)
    for (nv = 4; nv * 512 < groups;) nv *= 2;
  const int tpr = ((groups + nv - 1) / nv + 31) / 32 * 32;
  const int rpc = std::max(1, 256 / tpr);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // CTAs that fit the GPU at once, each over its share of the rows
  const int64_t fit = (int64_t)sms * std::max(1, (nv == 1 ? 1024 : (nv == 2 ? 768 : 2048)) / (tpr * rpc));
  const dim3 block(tpr, rpc), grid((unsigned)std::min<int64_t>((a.rows + rpc - 1) / rpc, fit));
  if (es == 4)
    return vec ? norm_nv<float, true>(nv, grid, block, st, n)
               : norm_nv<float, false>(nv, grid, block, st, n);
  return vec ? norm_nv<__nv_bfloat16, true>(nv, grid, block, st, n)
             : norm_nv<__nv_bfloat16, false>(nv, grid, block, st, n);
}

cudaError_t launch_quantize_fp8(const ds_quantize_fp8_args& a, cudaStream_t st) {
  const int es = a.dtype == DS_DTYPE_FP32 ? 4 : 2;
  QuantArgs n{a.x, a.q, a.scales, a.rows, a.x_stride, a.q_stride, a.scales_stride, a.cols,
              top_of(a.fp8), a.fp8 == DS_FP8_E5M2};
  const bool vec = on16(a.x, a.x_stride * es) && on8(a.q, a.q_stride);
  const int64_t blocks = ((int64_t)a.cols + kScaleBlock - 1) / kScaleBlock *
                         ((a.rows + kScaleBlock - 1) / kScaleBlock);
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 30));
  auto go = [&](auto e4m3, auto e5m2) {
    return launch_k(n.e5m2 ? e5m2 : e4m3, grid, dim3(256), 0, st, n);
  };
  auto pick = [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value;
    return a.block_rows == 1 ? go(k_quantize_fp8<T, V, true, false>, k_quantize_fp8<T, V, true, true>)
                             : go(k_quantize_fp8<T, V, false, false>, k_quantize_fp8<T, V, false, true>);
  };
  if (es == 4) return vec ? pick(float{}, std::true_type{}) : pick(float{}, std::false_type{});
  return vec ? pick(__nv_bfloat16{}, std::true_type{}) : pick(__nv_bfloat16{}, std::false_type{});
}

}  // namespace ds
