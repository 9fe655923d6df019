// fp8_gemm.cu -- products of e4m3 codes with one fp32 scale per block of 128,
// dense or grouped by expert, on the 5th-generation tensor cores.
//
//   c[m][n] = sum_b sa[m][b] sw[n/128][b] * (sum_{k in block b} a[m][k] w[n][k])
//
// The scales are arbitrary fp32 numbers, so they cannot ride on the MMA's own
// power-of-two block scales: each block of 128 columns is one MMA group (four
// tcgen05.mma kind::f8f6f4 of K = 32) into a TMEM accumulator of its own, and
// the epilogue warps read it back and add scale * partial to a sum in
// registers.  One scale product per thread and block suffices, because a thread
// owns one row and columns of a single 128-row weight block.
//
// A tile is 128 rows x BN columns.  Warp 0 loads the A and W tiles of each
// block by TMA (128-byte swizzle: a row of a block is exactly one 128-byte
// atom), one lane of warp 1 issues the MMAs, warps 2-9 promote: two warps per
// TMEM lane quarter, each with half of the columns.  TMEM holds 512 / BN
// accumulators (two at BN = 256), so the MMAs of the next block run while one
// is promoted.  Blocks are persistent over tiles.
//
// BN = 256 keeps the tensor cores busiest per byte of shared memory; narrow
// tiles (down to 16) spread few rows over all SMs, which then stream the
// weights at HBM rate.  The rule is in launch_fp8_gemm.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "ops.h"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int FG_BM = 128;
constexpr int FG_BK = kBlock128;                 // bytes = codes
constexpr int FG_EPI_WARPS = 8;
constexpr int FG_THREADS = 32 * (2 + FG_EPI_WARPS);
constexpr int FG_A_BYTES = FG_BM * FG_BK;

template <int BN>
struct FgCfg {
  static constexpr int kStage = FG_A_BYTES + BN * FG_BK;
  static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 5 : 8;
  static constexpr int kAcc = BN >= 256 ? 2 : BN >= 128 ? 4 : 8;      // TMEM accumulators
  static constexpr int kAccCols = BN < 32 ? 32 : BN;                  // TMEM column pitch
  static constexpr int kCols = BN / 2;                                // columns of one warp
  // output staging of an epilogue warp: 32 rows x kOutCols bf16 (the four
  // stages of BN = 256 leave room for 32 columns)
  static constexpr int kOutCols = BN >= 256 ? 32 : kCols;
  static constexpr int kOutBytes = FG_EPI_WARPS * 32 * kOutCols * 2;
  static constexpr size_t smem(int G) {
    return 1024 + (size_t)kStages * kStage + kOutBytes + (2 * kStages + 2 * kAcc) * 8 + 16 +
           (size_t)(2 * G + 2) * 4;
  }
};

struct alignas(64) FgMaps {
  CUtensorMap a, w;
};

__device__ __forceinline__ void fg_tma_2d(void* dst, const CUtensorMap* map, int c0, int c1,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T over 32 e4m3 columns, issued by one thread.
__device__ __forceinline__ void fg_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void fg_tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "columns per load");
  if constexpr (N == 32) {
    tmem_ld_32x32b_x32(taddr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
  }
}

// acc += s * p on a pair of floats.
__device__ __forceinline__ void fma2(float2& acc, float2 p, float2 s) {
  unsigned long long a = *reinterpret_cast<unsigned long long*>(&acc);
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(a)
      : "l"(*reinterpret_cast<unsigned long long*>(&p)),
        "l"(*reinterpret_cast<unsigned long long*>(&s)));
  acc = *reinterpret_cast<float2*>(&a);
}

// Where a tile lies.
struct FgTile {
  int g;         // group
  int m0, m_end; // first row, end of the group's rows
  int n0;        // first column
};

// Tiles run along the rows of one column stripe first inside a group, so that
// neighbouring blocks share the weights of the stripe.
__device__ __forceinline__ bool fg_tile(long long t, const GemmArgs& a, int bn, const int* rows,
                                        const int* first, FgTile* o) {
  const int nt = (a.N + bn - 1) / bn;
  if (t >= (long long)first[a.G] * nt) return false;
  // the last group g with first[g] * nt <= t
  int lo = 0, hi = a.G;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)first[mid] * nt <= t) lo = mid; else hi = mid;
  }
  // empty groups share their start with the next one: lo is the last of them,
  // and the only one that holds tiles
  const int mt = first[lo + 1] - first[lo];
  const int q = (int)(t - (long long)first[lo] * nt);
  o->g = lo;
  o->m0 = rows[lo] + (q % mt) * FG_BM;
  o->m_end = rows[lo + 1];
  o->n0 = (q / mt) * bn;
  return true;
}

template <int BN>
__global__ void __launch_bounds__(FG_THREADS, 1) fp8_gemm_kernel(
    GemmArgs a, const __grid_constant__ FgMaps mp) {
  using C = FgCfg<BN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* out_s = smem + C::kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_s + C::kOutBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* accf = empty + C::kStages;
  uint64_t* acce = accf + C::kAcc;
  uint32_t* holder = reinterpret_cast<uint32_t*>(acce + C::kAcc);
  int* rows = reinterpret_cast<int*>(holder + 4);    // [G+1] first row of each group
  int* first = rows + a.G + 1;                       // [G+1] first row tile of each group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KB = blocks128(a.K);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kAcc; ++s) {
      mbar_init(&accf[s], 1);
      mbar_init(&acce[s], FG_EPI_WARPS);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(holder, C::kAcc * C::kAccCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<uint64_t>(lane == 0 ? &mp.a : &mp.w))
                 : "memory");
  pdl_wait();
  pdl_launch_dependents();
  // row range and row-tile count of each group
  if (!a.offsets) {
    if (tid == 0) {
      rows[0] = 0;
      rows[1] = a.M;
      first[0] = 0;
      first[1] = (a.M + FG_BM - 1) / FG_BM;
    }
  } else if (warp == 0) {
    // one warp scans the offsets: a running maximum clamps them to 0..M and to
    // non-decreasing order, a running sum counts the tiles
    int top = 0, tiles = 0;
    bool bad = false;
    for (int g0 = 0; g0 <= a.G; g0 += 32) {
      const int g = g0 + lane;
      const int raw = g <= a.G ? a.offsets[g] : 0;
      int v = g <= a.G ? min(max(raw, 0), a.M) : 0;
      v = max(v, top);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, u);
      }
      bad |= g <= a.G && v != raw;
      int prev = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) prev = top;
      // tiles of group g - 1 end at offset g
      int n = (g >= 1 && g <= a.G) ? (v - prev + FG_BM - 1) / FG_BM : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += u;
      }
      if (g <= a.G) {
        rows[g] = v;
        first[g] = tiles + n;
      }
      top = __shfl_sync(0xffffffffu, v, 31);
      tiles += __shfl_sync(0xffffffffu, n, 31);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0)
      record_error(a.ctl, kErrRange, 0x400);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long long fills = 0;
      bool ok = true;
      FgTile tl;
      for (long long t = blockIdx.x; ok && fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
        const int wrow = tl.g * a.N + tl.n0;
        for (int kb = 0; kb < KB; ++kb) {
          if (fills >= C::kStages && !mbar_wait(&empty[s], ph ^ 1u, a.ctl, 0x401)) {
            ok = false;
            break;
          }
          unsigned char* st = smem + s * C::kStage;
          mbar_arrive_expect_tx(&full[s], C::kStage);
          fg_tma_2d(st, &mp.a, kb * FG_BK, tl.m0, &full[s]);
          fg_tma_2d(st + FG_A_BYTES, &mp.w, kb * FG_BK, wrow, &full[s]);
          ++fills;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // the newest phase of each stage may be unconsumed: its copies land first
      for (long long j = fills > C::kStages ? fills - C::kStages : 0; j < fills; ++j)
        mbar_wait(&full[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, a.ctl, 0x402);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // kind::f8f6f4: e4m3 A and B (format 0), fp32 D, both K-major
      const uint32_t idesc = idesc_f16_f32(FG_BM, BN);
      const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
      int s = 0, as = 0;
      uint32_t ph = 0, aph = 0;
      long long issued = 0;
      bool ok = true;
      FgTile tl;
      for (long long t = blockIdx.x; ok && fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb) {
          if ((issued >= C::kAcc && !mbar_wait(&acce[as], aph ^ 1u, a.ctl, 0x403)) ||
              !mbar_wait(&full[s], ph, a.ctl, 0x404)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + (uint64_t)(s * (C::kStage >> 4));
          const uint64_t bd = ad + (FG_A_BYTES >> 4);
          const uint32_t d = tmem + (uint32_t)(as * C::kAccCols);
#pragma unroll
          for (int j = 0; j < 4; ++j) fg_mma(d, ad + 2 * j, bd + 2 * j, idesc, j > 0 ? 1u : 0u);
          tc_commit(&empty[s]);
          tc_commit(&accf[as]);
          ++issued;
          if (++s == C::kStages) {
            s = 0;
            ph ^= 1u;
          }
          if (++as == C::kAcc) {
            as = 0;
            aph ^= 1u;
          }
        }
      }
      // every MMA issued has completed before this warp frees the TMEM: the
      // last phase of each accumulator
      for (long long j = issued > C::kAcc ? issued - C::kAcc : 0; j < issued; ++j)
        mbar_wait(&accf[j % C::kAcc], (uint32_t)(j / C::kAcc) & 1u, a.ctl, 0x405);
    }
  } else {
    const int ew = warp - 2, q = warp & 3, half = ew >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * C::kCols);
    uint32_t* stage = reinterpret_cast<uint32_t*>(out_s + ew * (32 * C::kOutCols * 2));
    constexpr int LD = C::kCols < 16 ? C::kCols : 16;    // columns of one TMEM load
    int as = 0;
    uint32_t aph = 0;
    bool ok = true;
    FgTile tl;
    for (long long t = blockIdx.x; ok && fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
      const int row0 = tl.m0 + 32 * q, row = row0 + lane;
      const int col0 = tl.n0 + half * C::kCols;
      const bool idle = row0 >= tl.m_end || col0 >= a.N;   // nothing of this warp's part is stored
      const float* sa = a.a_scales + (long long)min(row, a.M - 1) * KB;
      const float* sw = a.w_scales +
                        ((long long)tl.g * blocks128(a.N) + min(col0, a.N - 1) / kBlock128) * KB;
      float2 acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      float sa_n = idle ? 0.f : sa[0], sw_n = idle ? 0.f : sw[0];
      for (int kb = 0; kb < KB; ++kb) {
        const float sc = sa_n * sw_n;
        if (!idle && kb + 1 < KB) {
          sa_n = sa[kb + 1];
          sw_n = sw[kb + 1];
        }
        ok = mbar_wait(&accf[as], aph, a.ctl, 0x406);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!idle) {
          tc_fence_after();
          const float2 sc2 = make_float2(sc, sc);
#pragma unroll
          for (int c = 0; c < C::kCols; c += LD) {
            uint32_t v[LD];
            fg_tmem_ld<LD>(lane_base + (uint32_t)(as * C::kAccCols + c), v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < LD; j += 2)
              fma2(acc[(c + j) / 2], make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])),
                   sc2);
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[as]);
        if (++as == C::kAcc) {
          as = 0;
          aph ^= 1u;
        }
      }
      if (!ok || idle) continue;
      // rows of this warp to bf16 through its staging buffer (16-byte pieces,
      // rotated by the row so that neither side conflicts), then rows of
      // kOutCols columns to global memory
      constexpr int PIECES = C::kOutCols / 8;     // 16-byte pieces of a staged row
      const int nrow = min(32, tl.m_end - row0);
      const bool vec = (a.N & 7) == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
#pragma unroll
      for (int c = 0; c < C::kCols; c += C::kOutCols) {
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = acc[(c + 8 * p) / 2 + j];
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          const int at = p ^ (lane & (PIECES - 1));
          *reinterpret_cast<uint4*>(stage + (lane * PIECES + at) * 4) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int cols = min(C::kOutCols, a.N - (col0 + c));
        if (vec) {
#pragma unroll 4
          for (int i = lane; i < 32 * PIECES; i += 32) {
            const int r = i / PIECES, p = i % PIECES;
            if (r < nrow && 8 * p < cols)
              *reinterpret_cast<uint4*>(a.c + (long long)(row0 + r) * a.N + col0 + c + 8 * p) =
                  *reinterpret_cast<const uint4*>(stage + (r * PIECES + (p ^ (r & (PIECES - 1)))) * 4);
          }
        } else {
          const uint16_t* s16 = reinterpret_cast<const uint16_t*>(stage);
          for (int i = lane; i < 32 * C::kOutCols; i += 32) {
            const int r = i / C::kOutCols, n = i % C::kOutCols, p = n >> 3;
            if (r < nrow && n < cols)
              a.c[(long long)(row0 + r) * a.N + col0 + c + n] =
                  s16[(r * PIECES + (p ^ (r & (PIECES - 1)))) * 8 + (n & 7)];
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kAcc * C::kAccCols);
}

PFN_cuTensorMapEncodeTiled_v12000 fg_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// 2-D byte tensor [rows][inner], box [box_rows][128], 128-byte swizzle; rows
// and columns outside read as zero.
bool fg_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
  auto fn = fg_encode();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {inner};
  cuuint32_t box[2] = {FG_BK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
cudaError_t fg_launch(const GemmArgs& a, long long tiles, cudaStream_t st) {
  FgMaps mp;
  if (!fg_map(&mp.a, a.a, (uint64_t)a.K, (uint64_t)a.M, FG_BM) ||
      !fg_map(&mp.w, a.w, (uint64_t)a.K, (uint64_t)a.N * a.G, BN))
    return cudaErrorInvalidValue;
  const size_t sm = FgCfg<BN>::smem(a.G);
  cudaError_t e = cudaFuncSetAttribute(fp8_gemm_kernel<BN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  const long long grid = tiles < sm_count() ? tiles : sm_count();
  return launch_pdl(fp8_gemm_kernel<BN>, dim3((unsigned)grid), dim3(FG_THREADS), sm, st, a, mp);
}

}  // namespace

// Narrower tiles while there are fewer of them than SMs: a tile's time is then
// the latency of its own chain of blocks, and more SMs share the weight stream.
cudaError_t launch_fp8_gemm(const GemmArgs& a, cudaStream_t st) {
  // row tiles: the groups hold M rows in all, each at most one partial tile
  const long long mt = a.offsets ? a.M / FG_BM + (a.G < a.M ? a.G : a.M)
                                 : (a.M + FG_BM - 1) / FG_BM;
  const int sms = sm_count();
  auto tiles = [&](int bn) { return mt * ((a.N + bn - 1) / bn); };
  if (tiles(256) >= sms) return fg_launch<256>(a, tiles(256), st);
  if (tiles(128) >= sms) return fg_launch<128>(a, tiles(128), st);
  if (tiles(64) >= sms) return fg_launch<64>(a, tiles(64), st);
  if (tiles(32) >= sms) return fg_launch<32>(a, tiles(32), st);
  return fg_launch<16>(a, tiles(16), st);
}

}  // namespace moe
