// Product of two 8-bit matrices with a scale for each block of 128, on sm_103a:
//   C[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in block b} A[m, k] B[n, k]
// A [M, K] and B [N, K] in e4m3 or e5m2, one fp32 scale per row and 128 columns of A and per
// 128 x 128 block of B, C [M, N] in bf16 or fp32. The products inside a block are summed by the
// tensor core; the blocks' sums are scaled and added in fp32 registers, rounding to nearest.
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "ds_head.h"
#include "ds_tc_common.cuh"

namespace ds {
namespace {

using namespace tcpipe;

// Error bits of this device's products (kErrTimeout), and those that ds_head_status took from it last:
// one exchange reads and clears, so that a bit set by a product on another stream meanwhile is not lost.
__device__ uint32_t g_matmul_fp8_err = 0, g_matmul_fp8_taken = 0;
__global__ void k_take_matmul_fp8_errors() {
  pdl_wait();
  g_matmul_fp8_taken = atomicExch(&g_matmul_fp8_err, 0u);
}

// ------------------------------------------------------------------------------------------
// CUDA cores: any strides and bases
// ------------------------------------------------------------------------------------------
struct MatmulArgs {
  const uint8_t *a, *b;
  const float *sa, *sb;
  void* out;
  int64_t lda, ldb, lsa, lsb, ldo;
  int m, n, k;
  int a_e5m2, b_e5m2;
};

DS_DEV float fp8_to_f32(uint8_t v, bool e5m2) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, e5m2 ? __NV_E5M2 : __NV_E4M3)));
}

DS_DEV void put(float* p, float v) { *p = v; }
DS_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 64 x 64 tile of C a CTA, 4 x 4 a thread, 32 columns of K at a time.
template <typename O>
__global__ void __launch_bounds__(256) k_matmul_fp8_simt(const MatmulArgs p) {
  __shared__ float as[32][65], bs[32][65];
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < p.k; k0 += 32) {
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * 32; e += 256) {
      const int row = e >> 5, col = e & 31;
      const bool in = k0 + col < p.k;
      as[col][row] =
          in && m0 + row < p.m ? fp8_to_f32(p.a[(m0 + row) * p.lda + k0 + col], p.a_e5m2) : 0.f;
      bs[col][row] =
          in && n0 + row < p.n ? fp8_to_f32(p.b[(n0 + row) * p.ldb + k0 + col], p.b_e5m2) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int kk = 0; kk < 32; ++kk) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) av[i] = as[kk][ty + 16 * i];
#pragma unroll
      for (int j = 0; j < 4; ++j) bv[j] = bs[kk][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], bv[j], part[i][j]);
    }
    if ((k0 + 32) % kScaleBlock == 0 || k0 + 32 >= p.k) {
      const int kb = k0 / kScaleBlock;
      const float sb = p.sb[(n0 / kScaleBlock) * p.lsb + kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t row = m0 + ty + 16 * i;
        const float s = row < p.m ? p.sa[row * p.lsa + kb] * sb : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = m0 + ty + 16 * i, col = n0 + tx + 16 * j;
      if (row < p.m && col < p.n) put(static_cast<O*>(p.out) + row * p.ldo + col, acc[i][j]);
    }
}

// ------------------------------------------------------------------------------------------
// tensor cores
// ------------------------------------------------------------------------------------------
// The pipeline of ds_tc_common.cuh: one persistent CTA per SM, a warp that issues tiled copies, one
// that issues MMAs, and eight that drain. A k-block is 128 columns = 128 bytes a row = one scale
// block: four MMAs fill one TMEM buffer, and the drain adds it to its fp32 registers times
// sa[row] sb[128 columns], one factor per thread, since a thread holds one row and its columns lie
// in one block of B. A drain (TMEM read and one multiply-add an element) takes about half the time
// of the k-block's MMAs, so it hides behind the next one.
//
// PAIR: clusters of two CTAs and M = 256 MMAs, each CTA staging its 128 rows of A and half of the
// tile's rows of B: 2/3 of the bytes per product that a lone CTA takes in (2048 x 131072 x 2816:
// 618 us, lone CTAs 773).
//
// Bound, measured with parts left out of a copy: the MMAs of a k-block take 626 cycles when nothing
// waits for them (512 by the tensor core's nominal rate; an MMA is issued when the one before it
// starts, so what the issuing thread does between k-blocks shows). The two TMEM buffers make a chain
// of it: last MMA - commit - drain - release - next MMA into that buffer, about 1000 to 1200 cycles
// beside the MMAs, of which the drain's multiply-adds are 260 (two at a time; one at a time the
// kernel takes 677 us) and the handshake between the CTAs most of the rest; a k-block so takes about
// 1050 cycles, with the tile's output (12%). Tiles of 128 columns would have four buffers, but their
// MMAs read A twice as often and the kernel takes 779 us. Few rows are bound by B's bytes: 1 x 262144
// x 2816 runs in 107 to 113 us, 6.5 to 6.9 TB/s.
template <int BN, bool PAIR>
struct Tile {
  static constexpr int kBRows = PAIR ? BN / 2 : BN;  // rows of B a CTA stages
  static constexpr uint32_t kABytes = 128 * 128, kBBytes = kBRows * 128;
  static constexpr uint32_t kStage = kABytes + kBBytes;
  static constexpr int kStages = BN == 64 ? 8 : (BN == 256 && !PAIR ? 4 : 6);
  static constexpr int kBufs = BN == 256 ? 2 : 4;  // TMEM accumulators of BN columns
  static constexpr uint32_t kTmem = kBufs * BN;
  static constexpr uint32_t kStg = 4096;  // output boxes of an epilogue warp
  static constexpr size_t kSmem = (size_t)kStages * kStage + kEpiWarps * kStg + 1024;
};

// Warps 0-3 (copies, MMAs, two idle) give registers to warps 4-11, the drain, whose accumulators
// take 128 each: 128 x 40 + 256 x 232 registers are those of the launch, 384 x 168.
constexpr int kMmThreads = 128 + 32 * kEpiWarps;
DS_DEV void regs_control() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
DS_DEV void regs_drain() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }

// Columns that a tile's fixed costs (its first loads, its output) are worth, in the choice of width.
constexpr int kTileCost = 48;

struct MmCtl {
  uint64_t full[8], empty[8], tfull[4], tempty[4], mma_done;
  uint32_t tmem_base;
  int abort;
};

// a += b * s, two lanes of fp32 at a time.
DS_DEV void fma2(uint64_t& a, uint32_t b0, uint32_t b1, uint64_t s) {
  asm("{\n .reg .b64 t;\n mov.b64 t, {%1, %2};\n fma.rn.f32x2 %0, t, %3, %0;\n}\n"
      : "+l"(a)
      : "r"(b0), "r"(b1), "l"(s));
}

// acc[i] += scale * TMEM columns 2i, 2i + 1 of this warp's lanes, COLS (32, 64 or 128) columns from
// taddr; columns are on their way while others are added. `release` is called once all have
// been read.
template <int COLS, typename F>
DS_DEV void drain_scaled(uint32_t taddr, uint64_t (&acc)[COLS / 2], float scale, F release) {
  uint64_t s2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(scale));
  uint32_t r[2][32];
  auto add = [&](int c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) fma2(acc[16 * c + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], s2);
  };
  tmem_ld_32cols(taddr, r[0]);
  if constexpr (COLS > 32) tmem_ld_32cols(taddr + 32, r[1]);
  tmem_ld_wait();
  if constexpr (COLS <= 64) release();
  add(0);
  if constexpr (COLS > 64) tmem_ld_32cols(taddr + 64, r[0]);
  if constexpr (COLS > 32) add(1);
  if constexpr (COLS > 64) {
    tmem_ld_32cols(taddr + 96, r[1]);
    tmem_ld_wait();
    release();
    add(2);
    add(3);
  }
}

DS_DEV float lane0(uint64_t v) { return __uint_as_float((uint32_t)v); }
DS_DEV float lane1(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

template <int BN, bool PAIR, typename O>
__global__ void __launch_bounds__(kMmThreads, 1)
    k_matmul_fp8_tc(const __grid_constant__ CUtensorMap map_a,
                    const __grid_constant__ CUtensorMap map_b,
                    const __grid_constant__ CUtensorMap map_c, const MatmulArgs p,
                    const uint32_t a_bytes, const int tma_out) {
  using T = Tile<BN, PAIR>;
  constexpr int COLS = BN / 2;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ MmCtl ctl;
  uint8_t* smem = align1024(dyn_smem);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int n_units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int n_it = (p.m + (PAIR ? 255 : 127)) / (PAIR ? 256 : 128);
  const int n_tiles = n_it * ((p.n + BN - 1) / BN);  // (2^31 tiles would be 35 TB of output)
  const int nk = (p.k + 127) / 128;
  uint32_t* err = &g_matmul_fp8_err;
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(smem_u32(&ctl.full[s]), 1);
      mbar_init(smem_u32(&ctl.empty[s]), 1);
    }
    for (int b = 0; b < T::kBufs; ++b) {
      mbar_init(smem_u32(&ctl.tfull[b]), 1);
      mbar_init(smem_u32(&ctl.tempty[b]), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(smem_u32(&ctl.mma_done), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
    if (tma_out) tma_prefetch_desc(&map_c);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&ctl.tmem_base), T::kTmem);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&ctl.tmem_base), T::kTmem);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers initialised before any remote use
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort_flag = &ctl.abort;
  pdl_wait();

  if (warp < 4) {
    regs_control();
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_first();
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = unit; tile < n_tiles && ok; tile += n_units) {
          const int it = tile % n_it, ct = tile / n_it;
          const int row0 = (PAIR ? 2 * it + (int)rank : it) * 128;
          const int col0 = ct * BN + (PAIR ? (int)rank * T::kBRows : 0);
          for (int kb = 0; kb < nk; ++kb) {
            if (!mbar_wait(smem_u32(&ctl.empty[stage]), phase ^ 1, abort_flag, err)) {
              ok = false;
              break;
            }
            const uint32_t sa = sbase + stage * T::kStage, sb = sa + T::kABytes;
            const uint32_t fb = smem_u32(&ctl.full[stage]);
            if constexpr (PAIR) {
              // both CTAs' copies complete on the even CTA's barrier, which expects all of them
              if (rank == 0) mbar_arrive_expect_tx(fb, 2 * T::kStage);
              const uint32_t fb0 = mapa_shared(fb, 0);
              tma_load_2d_pair(sa, &map_a, fb0, kb * 128, row0, pol_a);
              tma_load_2d_pair(sb, &map_b, fb0, kb * 128, col0, pol_b);
            } else {
              // (a_bytes: fewer than 128 rows of A are copied when there are none; the rest of the
              // stage holds whatever was there, in rows of the product that are not stored)
              mbar_arrive_expect_tx(fb, a_bytes + T::kBBytes);
              tma_load_2d(sa, &map_a, fb, kb * 128, row0, pol_a);
              tma_load_2d(sb, &map_b, fb, kb * 128, col0, pol_b);
            }
            ++issued;
            if (++stage == T::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        // after an abort: wait for the copies still in flight, the last ones into each stage (pair:
        // the odd CTA's copies complete on the even CTA's barriers, where its producer waits)
        if (!ok && rank == 0) {
          for (int i = max(0, issued - T::kStages); i < issued; ++i)
            mbar_wait_quiet(smem_u32(&ctl.full[i % T::kStages]), (uint32_t)((i / T::kStages) & 1));
        }
      }
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        const uint32_t idesc = idesc_fp8_f32(PAIR ? 256 : 128, BN, p.a_e5m2, p.b_e5m2);
        const uint64_t adesc0 = sdesc_sw128(sbase, 16, 1024);
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        const int my_tiles = unit < n_tiles ? (n_tiles - 1 - unit) / n_units + 1 : 0;
        const int64_t total = (int64_t)my_tiles * nk;
        bool have = false, free = true;  // next stage filled, next buffer drained (seen so already)
        for (int64_t i = 0; i < total; ++i) {
          const uint32_t fb = smem_u32(&ctl.full[stage]), te = smem_u32(&ctl.tempty[buf]);
          if ((!free && !mbar_wait(te, bphase ^ 1, abort_flag, err)) ||
              (!have && !mbar_wait(fb, phase, abort_flag, err)))
            break;
          tc_fence_after();
          const uint32_t dt = tmem + (uint32_t)(buf * BN);
          const uint64_t ad = adesc0 + (uint64_t)(stage * (T::kStage >> 4));
          const uint64_t bd = ad + (T::kABytes >> 4);
          const uint32_t eb = smem_u32(&ctl.empty[stage]), tf = smem_u32(&ctl.tfull[buf]);
          if (++stage == T::kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++buf == T::kBufs) {
            buf = 0;
            bphase ^= 1;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 32 columns on: two 16-byte units of the address field
            if constexpr (PAIR) umma_fp8_pair(dt, ad + 2 * k, bd + 2 * k, idesc, k != 0);
            else umma_fp8(dt, ad + 2 * k, bd + 2 * k, idesc, k != 0);
            // an MMA is issued when the one before it starts, so what stands between the last MMA
            // of a k-block and the first of the next is what can leave the tensor core idle: the
            // next k-block's barriers are looked at here instead
            if (k == 1) have = mbar_test<false>(smem_u32(&ctl.full[stage]), phase);
            if (k == 2) free = mbar_test<false>(smem_u32(&ctl.tempty[buf]), bphase ^ 1);
          }
          if constexpr (PAIR) {
            umma_commit_pair(tf, 0x3);
            umma_commit_pair(eb, 0x3);
          } else {
            umma_commit(tf);
            umma_commit(eb);
          }
        }
        if constexpr (PAIR) umma_commit_pair(smem_u32(&ctl.mma_done), 0x1);
        else umma_commit(smem_u32(&ctl.mma_done));
        mbar_wait_quiet(smem_u32(&ctl.mma_done), 0);
      }
    }
  } else {
    regs_drain();
    const int q = warp & 3;            // TMEM lane quadrant this warp may access
    const int half = (warp - 4) >> 2;  // column half of the tile
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    const uint32_t stg0 = sbase + T::kStages * T::kStage + (uint32_t)(warp - 4) * T::kStg;
    int buf = 0, box = 0;  // box: of the output boxes, the next one
    uint32_t bphase = 0;
    bool ok = true;
    for (int tile = unit; tile < n_tiles && ok; tile += n_units) {
      const int it = tile % n_it, ct = tile / n_it;
      const int row0 = (PAIR ? 2 * it + (int)rank : it) * 128 + q * 32;
      const int col0 = ct * BN + half * COLS;
      const bool live = row0 < p.m && col0 < p.n;  // else nothing of this box is stored
      const float* sa = p.sa + (int64_t)min(row0 + lane, p.m - 1) * p.lsa;
      const float* sb = p.sb + (int64_t)(min(col0, p.n - 1) / kScaleBlock) * p.lsb;
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0;
      float scale = sa[0] * sb[0];
      for (int kb = 0; kb < nk; ++kb) {
        const int nx = min(kb + 1, nk - 1);
        const float next_a = sa[nx], next_b = sb[nx];
        if (!mbar_wait(smem_u32(&ctl.tfull[buf]), bphase, abort_flag, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl.tempty[buf]), 0));
            else mbar_arrive(smem_u32(&ctl.tempty[buf]));
          }
        };
        if (live)
          drain_scaled<COLS>(tmem + (uint32_t)(buf * BN + half * COLS) + lane_base, acc, scale, release);
        else
          release();
        scale = next_a * next_b;
        if (++buf == T::kBufs) {
          buf = 0;
          bphase ^= 1;
        }
      }
      if (!ok) break;
      if (!live) continue;
#pragma unroll
      for (int bx = 0; bx < COLS / 32; ++bx) {
        if (tma_out) {
          // boxes are used in turn, over all tiles of this warp (a tile of 64 columns has one a warp):
          // the one before last has been read when all but the last have
          constexpr uint32_t kBox = sizeof(O) * 1024;
          constexpr int kBoxes = T::kStg / kBox;
          static_assert(kBoxes == 1 || kBoxes == 2, "the wait below is for one or two boxes");
          const uint32_t stg = stg0 + (COLS / 32 % kBoxes == 0 ? bx % kBoxes : box) * kBox;
          box = (box + 1) % kBoxes;
          if (lane == 0) {
            if constexpr (kBoxes == 2) bulk_wait_read_le1();
            else bulk_wait_read_all();
          }
          __syncwarp();
          if constexpr (sizeof(O) == 4) {
            // row `lane` of the box, 16-byte chunk c at its 128-byte-swizzled position
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_f4(stg + lane * 128 + ((c ^ (lane & 7)) << 4), lane0(acc[bx * 16 + 2 * c]),
                           lane1(acc[bx * 16 + 2 * c]), lane0(acc[bx * 16 + 2 * c + 1]),
                           lane1(acc[bx * 16 + 2 * c + 1]));
          } else {
            // rows of 64 bytes in the 64-byte swizzle
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint64_t v = acc[bx * 16 + 4 * c + e];
                const __nv_bfloat162 h = __floats2bfloat162_rn(lane0(v), lane1(v));
                w[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
              st_shared_u4(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&map_c, stg, (int32_t)(col0 + bx * 32), row0);
            bulk_commit();
          }
        } else {
          // rows of C on any boundary: the box turns in shared memory (word (r, c) at column c ^ r,
          // so neither side has bank conflicts) and leaves a row of 32 columns at a time
          const uint32_t stg = stg0;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            st_shared_f32(stg + lane * 128 + (((2 * i) ^ lane) << 2), lane0(acc[bx * 16 + i]));
            st_shared_f32(stg + lane * 128 + (((2 * i + 1) ^ lane) << 2), lane1(acc[bx * 16 + i]));
          }
          __syncwarp();
          const int col = col0 + bx * 32 + lane;
          const int rows = min(32, p.m - row0);
          O* out = static_cast<O*>(p.out) + (int64_t)row0 * p.ldo + col;
          if (col < p.n)
            for (int r = 0; r < rows; ++r, out += p.ldo)
              put(out, ld_shared_f32(stg + r * 128 + ((lane ^ r) << 2)));
        }
      }
    }
    if (tma_out && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  // pair: neither CTA frees its TMEM or exits while the other may still use its barriers,
  // shared memory or TMEM
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, T::kTmem);
    else tmem_dealloc(tmem, T::kTmem);
  }
}

// What launches need to know of a device, read once for each: the SMs, and how many CTA pairs can
// be resident at once (a TPC with one SM holds none).
struct DeviceInfo {
  int sms, pairs;
};
std::once_flag g_device_once[kMaxHeadDevices];
DeviceInfo g_device[kMaxHeadDevices];
cudaError_t g_device_error[kMaxHeadDevices];

template <int BN, bool PAIR, typename O>
void prepare(cudaError_t* e) {
  if (*e == cudaSuccess)
    *e = cudaFuncSetAttribute(k_matmul_fp8_tc<BN, PAIR, O>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Tile<BN, PAIR>::kSmem);
}

cudaError_t device_info(DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxHeadDevices) return cudaErrorInvalidDevice;
  std::call_once(g_device_once[dev], [dev] {
    DeviceInfo& d = g_device[dev];
    cudaError_t& s = g_device_error[dev];
    s = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    prepare<256, true, float>(&s);
    prepare<256, false, float>(&s);
    prepare<128, false, float>(&s);
    prepare<64, false, float>(&s);
    prepare<256, true, __nv_bfloat16>(&s);
    prepare<256, false, __nv_bfloat16>(&s);
    prepare<128, false, __nv_bfloat16>(&s);
    prepare<64, false, __nv_bfloat16>(&s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(2, d.sms / 2 * 2));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = Tile<256, true>::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (s == cudaSuccess)
      s = cudaOccupancyMaxActiveClusters(&d.pairs, k_matmul_fp8_tc<256, true, float>, &cfg);
    d.pairs = std::max(1, d.pairs);
  });
  *out = g_device[dev];
  return g_device_error[dev];
}

MatmulArgs pack(const ds_matmul_fp8_args& a) {
  return MatmulArgs{a.a, a.b, a.a_scales, a.b_scales, a.out, a.a_stride, a.b_stride,
                    a.a_scales_stride, a.b_scales_stride, a.out_stride, (int)a.m, (int)a.n, (int)a.k,
                    a.a_type == DS_FP8_E5M2, a.b_type == DS_FP8_E5M2};
}

}  // namespace

cudaError_t launch_matmul_fp8_simt(const ds_matmul_fp8_args& a, cudaStream_t st) {
  const MatmulArgs p = pack(a);
  // tiles of rows go to grid.y in slices of its largest extent
  for (int64_t m0 = 0; m0 < a.m; m0 += 65535ll * 64) {
    MatmulArgs q = p;
    q.a += m0 * q.lda;
    q.sa += m0 * q.lsa;
    q.m = (int)std::min<int64_t>(a.m - m0, 65535ll * 64);
    const int es = a.out_dtype == DS_DTYPE_FP32 ? 4 : 2;
    q.out = static_cast<uint8_t*>(p.out) + m0 * q.ldo * es;
    const dim3 grid((unsigned)((a.n + 63) / 64), (unsigned)((q.m + 63) / 64));
    const cudaError_t e =
        es == 4 ? launch_k(k_matmul_fp8_simt<float>, grid, dim3(256), 0, st, q)
                : launch_k(k_matmul_fp8_simt<__nv_bfloat16>, grid, dim3(256), 0, st, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

bool matmul_fp8_tensor_ok(const ds_matmul_fp8_args& a) {
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return tc_available() && on16(a.a) && on16(a.b) && a.a_stride % 16 == 0 && a.b_stride % 16 == 0;
}

cudaError_t launch_matmul_fp8_tc(const ds_matmul_fp8_args& a, cudaStream_t st) {
  DeviceInfo di;
  cudaError_t e = device_info(&di);
  if (e != cudaSuccess) return e;
  const MatmulArgs p = pack(a);
  const int es = a.out_dtype == DS_DTYPE_FP32 ? 4 : 2;
  // Tile width and pairing: the least of (rounds of tiles over the SMs) x (columns a tile takes,
  // plus what a tile costs whatever its width). A pair works on 256 rows, a lone CTA on 128.
  const int64_t mt = (p.m + 127) / 128, mt2 = (p.m + 255) / 256;
  auto rounds = [](int64_t tiles, int units) { return (tiles + units - 1) / units; };
  int bn = 256;
  bool pair = false;
  double best = 0;
  for (int w : {256, 128, 64}) {
    const double c = (double)rounds(mt * ((p.n + w - 1) / w), di.sms) * (w + kTileCost);
    if (w == 256 || c < best) {
      best = c;
      bn = w;
    }
  }
  if (p.m > 128) {
    const double c = (double)rounds(mt2 * ((p.n + 255) / 256), di.pairs) * (256 + kTileCost);
    if (c <= best) {
      bn = 256;
      pair = true;
    }
  }
  CUtensorMap ma, mb, mc;
  const int abox = pair ? 128 : (int)std::min<int64_t>(128, (p.m + 7) / 8 * 8);
  const bool tma_out = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && a.out_stride * es % 16 == 0;
  if (!tc_make_map_strided(&ma, 0, p.a, p.m, p.k, p.lda, abox, 128, false) ||
      !tc_make_map_strided(&mb, 0, p.b, p.n, p.k, p.ldb, pair ? 128 : bn, 128, false))
    return cudaErrorInvalidValue;
  mc = ma;  // not used without tma_out
  if (tma_out && !tc_make_map_strided(&mc, es == 4 ? 2 : 1, p.out, p.m, p.n, p.ldo * es, 32, 32, es == 2))
    return cudaErrorInvalidValue;
  const int64_t tiles = pair ? mt2 * ((p.n + 255) / 256) : mt * ((p.n + bn - 1) / bn);
  auto go = [&](auto kernel, int smem, bool pr) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pr) {
      attr[n].id = cudaLaunchAttributeClusterDimension;
      attr[n].val.clusterDim.x = 2;
      attr[n].val.clusterDim.y = 1;
      attr[n++].val.clusterDim.z = 1;
    }
    if (pdl_enabled()) {
      attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const int64_t units = std::min<int64_t>(tiles, pr ? di.pairs : di.sms);
    cfg.gridDim = dim3((unsigned)(pr ? 2 * units : units));
    return cudaLaunchKernelEx(&cfg, kernel, ma, mb, mc, p, (uint32_t)abox * 128u, tma_out ? 1 : 0);
  };
  auto pick = [&](auto o) {
    using O = decltype(o);
    if (pair) return go(k_matmul_fp8_tc<256, true, O>, (int)Tile<256, true>::kSmem, true);
    if (bn == 256) return go(k_matmul_fp8_tc<256, false, O>, (int)Tile<256, false>::kSmem, false);
    if (bn == 128) return go(k_matmul_fp8_tc<128, false, O>, (int)Tile<128, false>::kSmem, false);
    return go(k_matmul_fp8_tc<64, false, O>, (int)Tile<64, false>::kSmem, false);
  };
  return es == 4 ? pick(float{}) : pick(__nv_bfloat16{});
}

cudaError_t read_matmul_fp8_errors(uint32_t* word, cudaStream_t st) {
  static std::mutex m;  // one reader at a time has g_matmul_fp8_taken
  std::lock_guard<std::mutex> lock(m);
  cudaError_t e = launch_k(k_take_matmul_fp8_errors, dim3(1), dim3(1), 0, st);
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(word, g_matmul_fp8_taken, sizeof(*word), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e;
}

}  // namespace ds
