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
// k-block by TMA (128-byte swizzle: a row of a k-block is exactly one 128-byte
// atom), one lane of warp 1 issues the MMAs, eight other warps promote, two per
// TMEM lane quarter, each with half of the columns.  TMEM holds several
// accumulators (two at BN = 256), so the MMAs of the next k-blocks run while one
// is promoted.  Blocks are persistent over tiles.
//
// Two kernels: fp8_gemm_kernel for BN = 16 .. 128, where few rows are spread over
// all SMs, which then stream the weights; fp8_gemm_wide_kernel for BN = 256, which
// moves the fewest operand bytes per product.  The rule is in launch_fp8_gemm.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "ops.h"
#include "pipe.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int FG_BM = 128;
constexpr int FG_BK = kBlock128;                 // bytes = codes
constexpr int FG_EPI_WARPS = 8;
constexpr int FG_THREADS = 32 * (2 + FG_EPI_WARPS);

// One tile shape: BN columns; AR rows of A staged (32: every tile has at most
// 32 rows, and what the MMA reads as rows 32..127 is whatever follows in shared
// memory, which only reaches accumulator rows that are never stored); KBS
// k-blocks per stage of the ring and per group of accumulators.  A hand-over
// between two roles costs about 200 cycles of barrier operations whatever it
// hands over, so narrow tiles, whose k-block takes less than that, hand over
// several at a time.
template <int BN, int AR>
struct FgCfg {
  static constexpr int kKbs = BN == 128 ? 2 : AR == 32 ? 4 : 2;
  static constexpr int kABytes = AR * FG_BK;
  static constexpr int kBlockBytes = kABytes + BN * FG_BK;            // one k-block
  static constexpr int kStage = kKbs * kBlockBytes;
  // the MMA reads 128 rows from the base of a short A tile: the ring's tail
  // keeps the last k-block's reads inside it
  static constexpr int kTail = FG_BM * FG_BK > kBlockBytes ? FG_BM * FG_BK - kBlockBytes : 0;
  static constexpr int kStages = (192 * 1024 - kTail) / kStage;
  static constexpr int kGroups = 512 / (kKbs * BN) > 4 ? 4 : 512 / (kKbs * BN);
  static constexpr int kTmemCols = kGroups * kKbs * BN;
  static constexpr int kCols = BN / 2;                                // columns of one epilogue warp
  static constexpr int kLd = kCols < 32 ? kCols : 32;                 // columns of one TMEM load
  // output staging of an epilogue warp: 32 rows x kOutCols bf16
  static constexpr int kOutCols = kCols < 32 ? kCols : 32;
  static constexpr int kOutBytes = FG_EPI_WARPS * 32 * kOutCols * 2;
  static constexpr int kRingEnd = kStages * kStage + kTail;
  static constexpr size_t smem(int G) {
    return 1024 + (size_t)kRingEnd + kOutBytes + (2 * kStages + 2 * kGroups + 1) * 8 + 16 +
           (size_t)(2 * G + 2) * 4;
  }
};

// A by tiles of 128 rows, and by pieces of 32 rows for tiles with few.
struct alignas(64) FgMaps {
  CUtensorMap a, a32, w, c;     // c: output by 32 rows x 64 columns (wide tiles only)
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

// Wait for this thread's TMEM loads; v passes through, so that nothing that
// uses it can move ahead of the wait.
template <int N>
__device__ __forceinline__ void fg_tmem_wait(uint32_t (&v)[N]) {
  if constexpr (N == 32) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])::"memory");
  } else if constexpr (N == 16) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
  } else {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7])::"memory");
  }
}

// Hand an accumulator back.  Relaxed: the TMEM loads are complete (wait::ld)
// and nothing else is handed over, while a release would first wait for the
// scale loads in flight (about 1,000 cycles at cluster scope).
__device__ __forceinline__ void fg_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Test switch: the role `who` of block 0 issues nothing, so that the others' waits
// for it run out.
constexpr uint32_t kHoldMma = 1u, kHoldLoads = 2u;
__device__ __forceinline__ bool fg_held(const Control* ctl, uint32_t who) {
  return ctl && blockIdx.x == 0 &&
         *reinterpret_cast<const volatile uint32_t*>(&ctl->withhold_ops) == who;
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

// The block's tile t, by a whole warp; o->g starts at 0 and goes along with t, which
// only grows.  Tiles run along the rows of one column stripe first inside a group,
// so that neighbouring blocks share the weights of the stripe.  The group is
// looked for 32 at a time from the last one on (a binary search by each lane took
// about 800 cycles, as long as two k-blocks).
__device__ __forceinline__ bool fg_tile(long long t, const GemmArgs& a, int bn, const int* rows,
                                        const int* first, FgTile* o) {
  const int nt = (a.N + bn - 1) / bn;
  if (t >= (long long)first[a.G] * nt) return false;
  // the last group g with first[g] * nt <= t: empty groups share their start with
  // the next one, so it is the one that holds tile t
  int g = o->g;
  if (a.G > 1) {
    for (;;) {
      const int i = g + 1 + (int)(threadIdx.x & 31);
      const uint32_t m = __ballot_sync(0xffffffffu, i <= a.G && (long long)first[i] * nt <= t);
      g += __popc(m);
      if (m != 0xffffffffu) break;
    }
  }
  const int mt = first[g + 1] - first[g];
  const int q = (int)(t - (long long)first[g] * nt), n = q / mt;
  o->g = g;
  o->m0 = rows[g] + (q - n * mt) * FG_BM;
  o->m_end = rows[g + 1];
  o->n0 = n * bn;
  return true;
}

// Row range and row-tile count of each group, into shared memory; the caller's
// barrier follows.
__device__ __forceinline__ void fg_groups(const GemmArgs& a, int* rows, int* first) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
}

// One epilogue warp's 32 rows x COLS columns to bf16 and to global memory,
// through its staging buffer of OUT columns at a time (16-byte pieces, rotated
// by the row so that neither side conflicts), so that stores cover whole runs
// of a row.
template <int COLS, int OUT>
__device__ __forceinline__ void fg_store(const GemmArgs& a, const float2 (&acc)[COLS / 2],
                                         uint32_t* stage, int row0, int nrow, int col0, int lane) {
  constexpr int PIECES = OUT / 8;     // 16-byte pieces of a staged row
  constexpr int RPI = 32 / PIECES;    // rows of one store instruction
  const bool vec = (a.N & 7) == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
#pragma unroll
  for (int c = 0; c < COLS; c += OUT) {
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
    const int cols = min(OUT, a.N - (col0 + c));
    if (vec) {
      const int p = lane % PIECES, r0 = lane / PIECES;
      uint16_t* o = a.c + (long long)(row0 + r0) * a.N + col0 + c + 8 * p;
      const long long step = (long long)RPI * a.N;
#pragma unroll
      for (int i = 0; i < PIECES; ++i, o += step) {
        const int r = r0 + i * RPI;
        if (r < nrow && 8 * p < cols)
          *reinterpret_cast<uint4*>(o) =
              *reinterpret_cast<const uint4*>(stage + (r * PIECES + (p ^ (r & (PIECES - 1)))) * 4);
      }
    } else {
      const uint16_t* s16 = reinterpret_cast<const uint16_t*>(stage);
      for (int i = lane; i < 32 * OUT; i += 32) {
        const int r = i / OUT, n = i % OUT, p = n >> 3;
        if (r < nrow && n < cols)
          a.c[(long long)(row0 + r) * a.N + col0 + c + n] =
              s16[(r * PIECES + (p ^ (r & (PIECES - 1)))) * 8 + (n & 7)];
      }
    }
  }
}

template <int BN, int AR>
__global__ void __launch_bounds__(FG_THREADS, 1) fp8_gemm_kernel(
    GemmArgs a, const __grid_constant__ FgMaps mp) {
  using C = FgCfg<BN, AR>;
  constexpr int KBS = C::kKbs;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* out_s = smem + C::kRingEnd;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_s + C::kOutBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* accf = empty + C::kStages;
  uint64_t* acce = accf + C::kGroups;
  uint64_t* done = acce + C::kGroups;                // every MMA has completed
  uint32_t* holder = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* gave_up = holder + 1;
  int* rows = reinterpret_cast<int*>(holder + 4);    // [G+1] first row of each group
  int* first = rows + a.G + 1;                       // [G+1] first row tile of each group
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KB = blocks128(a.K);

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kGroups; ++s) {
      mbar_init(&accf[s], 1);
      mbar_init(&acce[s], FG_EPI_WARPS);
    }
    mbar_init(done, 1);
    *gave_up = 0u;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane < 3 && (AR == FG_BM || lane > 0))
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<uint64_t>(lane == 0 ? &mp.a : lane == 1 ? &mp.a32 : &mp.w))
                 : "memory");
  pdl_wait();
  fg_groups(a, rows, first);
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();   // the TMEM is allocated: no block of the next kernel can take it first
  tc_fence_after();
  const uint32_t tmem = *holder;
  const bool elected = elect_one();

  // The loader and the MMA warp walk their loops whole, with one lane, elected
  // once, issuing, so that the loop's values stay warp-uniform (a loop under
  // lane == 0 spent twice the cycles on issuing).
  if (warp == 0) {
    int s = 0;
    uint32_t ph = 0;
    int fills = 0;          // capped at kStages
    long long n = 0;        // fills issued
    bool live = !fg_held(a.ctl, kHoldLoads);   // until a wait runs out
    FgTile tl = {};
    for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl);
         t += gridDim.x) {
      const int wrow = tl.g * a.N + tl.n0;
      // Rows past the tile's last are not loaded, by pieces of 32.
      const int nrow = min(FG_BM, tl.m_end - tl.m0), pieces = nrow > 96 ? 0 : (nrow + 31) / 32;
      const uint32_t bytes = ((pieces ? pieces * 32 : FG_BM) + BN) * FG_BK;
      for (int kb = 0; kb < KB; kb += KBS) {
        if (fills == C::kStages) {
          live &= pipe_wait(&empty[s], ph ^ 1u, a.ctl, 0x401, gave_up);
        } else {
          ++fills;
        }
        if (elected && live) {
          ++n;
          unsigned char* st = smem + s * C::kStage;
          const int nk = min(KBS, KB - kb);
          mbar_arrive_expect_tx(&full[s], nk * bytes);
#pragma unroll
          for (int j = 0; j < KBS; ++j) {
            if (j < nk) {
              unsigned char* b = st + j * C::kBlockBytes;
              if (AR == FG_BM && pieces == 0) {
                fg_tma_2d(b, &mp.a, (kb + j) * FG_BK, tl.m0, &full[s]);
              } else {
                for (int p = 0; p < (AR == 32 ? 1 : pieces); ++p)
                  fg_tma_2d(b + p * 32 * FG_BK, &mp.a32, (kb + j) * FG_BK, tl.m0 + 32 * p, &full[s]);
              }
              fg_tma_2d(b + C::kABytes, &mp.w, (kb + j) * FG_BK, wrow, &full[s]);
            }
          }
        }
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (elected) pipe_drain(full, C::kStages, n, a.ctl, 0x402);
  } else if (warp == 1) {
    // kind::f8f6f4: e4m3 A and B (format 0), fp32 D, both K-major
    const uint32_t idesc = idesc_f16_f32(FG_BM, BN);
    const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
    int s = 0, as = 0, used = 0;     // used: accumulator groups handed out, capped at kGroups
    uint32_t ph = 0, aph = 0;
    bool live = !fg_held(a.ctl, kHoldMma);   // until a wait runs out
    FgTile tl = {};
    for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl);
         t += gridDim.x) {
      for (int kb = 0; kb < KB; kb += KBS) {
        if (used == C::kGroups) {
          live &= pipe_wait(&acce[as], aph ^ 1u, a.ctl, 0x403, gave_up);
        } else {
          ++used;
        }
        live &= pipe_wait(&full[s], ph, a.ctl, 0x404, gave_up);
        tc_fence_after();
        if (elected && live) {
          const uint64_t st = desc0 + (uint64_t)(s * (C::kStage >> 4));
          const uint32_t d = tmem + (uint32_t)(as * KBS * BN);
          const int nk = min(KBS, KB - kb);
#pragma unroll
          for (int j = 0; j < KBS; ++j) {
            if (j < nk) {
              const uint64_t ad = st + (uint64_t)(j * (C::kBlockBytes >> 4));
              const uint64_t bd = ad + (C::kABytes >> 4);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                fg_mma(d + (uint32_t)(j * BN), ad + 2 * i, bd + 2 * i, idesc, i > 0 ? 1u : 0u);
            }
          }
          tc_commit(&empty[s]);
          tc_commit(&accf[as]);
        }
        if (++s == C::kStages) {
          s = 0;
          ph ^= 1u;
        }
        if (++as == C::kGroups) {
          as = 0;
          aph ^= 1u;
        }
      }
    }
    // every MMA issued has completed before this warp frees the TMEM
    if (elected) tc_commit(done);
    mbar_wait(done, 0, a.ctl, 0x405);
  } else {
    const int ew = warp - 2, q = warp & 3, part = ew >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(part * C::kCols);
    uint32_t* stage = reinterpret_cast<uint32_t*>(out_s + ew * (32 * C::kOutCols * 2));
    constexpr int LD = C::kLd, CH = C::kCols / LD;     // loads per k-block
    int as = 0;
    uint32_t aph = 0;
    FgTile tl = {};
    for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl);
         t += gridDim.x) {
      const int row0 = tl.m0 + 32 * q, row = row0 + lane;
      const int col0 = tl.n0 + part * C::kCols;
      const bool idle = row0 >= tl.m_end || col0 >= a.N;   // nothing of this warp's part is stored
      const float* sa = a.a_scales + (long long)min(row, a.M - 1) * KB;
      const float* sw = a.w_scales +
                        ((long long)tl.g * blocks128(a.N) + min(col0, a.N - 1) / kBlock128) * KB;
      float2 acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      // scales of the next group, in flight while the present one is promoted
      float sa_n[KBS], sw_n[KBS];
#pragma unroll
      for (int j = 0; j < KBS; ++j) {
        sa_n[j] = !idle && j < KB ? sa[j] : 0.f;
        sw_n[j] = !idle && j < KB ? sw[j] : 0.f;
      }
      for (int kb = 0; kb < KB; kb += KBS) {
        float sc[KBS];
#pragma unroll
        for (int j = 0; j < KBS; ++j) {
          sc[j] = sa_n[j] * sw_n[j];
          const bool more = !idle && kb + KBS + j < KB;
          sa_n[j] = more ? sa[kb + KBS + j] : 0.f;
          sw_n[j] = more ? sw[kb + KBS + j] : 0.f;
        }
        pipe_wait(&accf[as], aph, a.ctl, 0x406, gave_up);
        __syncwarp();      // the TMEM loads are the whole warp's
        if (!idle) {
          tc_fence_after();
          const uint32_t base = lane_base + (uint32_t)(as * KBS * BN);
          const int nk = min(KBS, KB - kb);
          // one load ahead of the sums
          uint32_t v[2][LD];
          fg_tmem_ld<LD>(base, v[0]);
#pragma unroll
          for (int i = 0; i < KBS * CH; ++i) {
            const int j = i / CH, c = (i % CH) * LD;
            if (j < nk) {
              fg_tmem_wait<LD>(v[i & 1]);
              if (i + 1 < KBS * CH && (i + 1) / CH < nk)
                fg_tmem_ld<LD>(base + (uint32_t)(((i + 1) / CH) * BN + ((i + 1) % CH) * LD),
                               v[(i + 1) & 1]);
              const float2 sc2 = make_float2(sc[j], sc[j]);
#pragma unroll
              for (int x = 0; x < LD; x += 2)
                fma2(acc[(c + x) / 2],
                     make_float2(__uint_as_float(v[i & 1][x]), __uint_as_float(v[i & 1][x + 1])),
                     sc2);
            }
          }
          tc_fence_before();
        }
        if (elected) fg_arrive(&acce[as]);
        if (++as == C::kGroups) {
          as = 0;
          aph ^= 1u;
        }
      }
      if (idle) continue;
      fg_store<C::kCols, C::kOutCols>(a, acc, stage, row0, min(32, tl.m_end - row0), col0, lane);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// ------------------------------------------------------------ wide tiles
// 128 x 256 tiles for many rows.  A k-block takes about 1,130 cycles (8192 x 4096 x
// 2048: 7 waves of 16 in 77 us at 1.64 GHz under a profiler), of which its MMAs are 540
// and its 48 KB would be 720 at the 68 bytes per cycle and SM that the L2 was measured
// to deliver: neither bounds it.  What is left is the round trip of the two
// accumulators (commit, promotion, hand-back), whose parts were not timed one by one.
// Measured in graphs: 8192 x 4096 x 2048 73 us, 20,480 rows in 512 groups of 1024 x 2048
// 204 us, 81,920 rows 300 us; in a long run, under the power cap, the first takes 87
// and the last 364 us.  Pairs of SMs on 256 x 256 tiles load 32 KB per SM and k-block,
// but the hand-overs between two SMs cost what that saves (65 against 67 us for the
// first, 420 against 305 us for the last, on one box).
//
// One tcgen05.mma takes all 256 columns: at 128 columns a block's MMAs read A
// twice and shared memory at 122 bytes per cycle, which nearly halves their rate.
// TMEM holds two accumulators; two epilogue warps per lane quarter hold 128 sums a
// thread, with the registers that the other warps give up (setmaxnreg).
constexpr int FW_HALF = FG_BM * FG_BK;                 // 16 KB: 128 rows of a k-block
constexpr int FW_STAGE = 3 * FW_HALF;                  // A, two halves of W
constexpr int FW_MAX_STAGES = 4;
constexpr int FW_THREADS = 384;                        // 4 warps of roles, 8 of epilogue
constexpr int FW_SLOTS = 2;                            // TMEM accumulators of 256 columns
constexpr int FW_OUT = 32 * 64 * 2;                    // staging of a warp: 32 rows x 64 columns
constexpr int FW_REGS = 168, FW_REGS_ROLE = 40, FW_REGS_EPI = 232;
static_assert(4 * FW_REGS_ROLE + 8 * FW_REGS_EPI <= 12 * FW_REGS,
              "setmaxnreg hands out what the block was launched with");

__host__ __device__ constexpr size_t fw_smem(int stages, int G) {
  return 1024 + (size_t)stages * FW_STAGE + FG_EPI_WARPS * FW_OUT +
         (2 * FW_MAX_STAGES + 2 * FW_SLOTS + 1) * 8 + 16 + (size_t)(2 * G + 2) * 4;
}

// From 241 groups on their offsets take the place of one stage.
int fw_stages(int G) {
  return fw_smem(FW_MAX_STAGES, G) <= kMaxSmem ? FW_MAX_STAGES : FW_MAX_STAGES - 1;
}

__global__ void __launch_bounds__(FW_THREADS, 1)
    fp8_gemm_wide_kernel(GemmArgs a, int stages, const __grid_constant__ FgMaps mp) {
  constexpr int BN = 256;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* out_s = smem + stages * FW_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_s + FG_EPI_WARPS * FW_OUT);
  uint64_t* empty = full + FW_MAX_STAGES;
  uint64_t* accf = empty + FW_MAX_STAGES;
  uint64_t* acce = accf + FW_SLOTS;
  uint64_t* done = acce + FW_SLOTS;
  uint32_t* holder = reinterpret_cast<uint32_t*>(done + 1);
  uint32_t* gave_up = holder + 1;
  int* rows = reinterpret_cast<int*>(holder + 4);
  int* first = rows + a.G + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int KB = blocks128(a.K);

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < FW_SLOTS; ++s) {
      mbar_init(&accf[s], 1);
      mbar_init(&acce[s], FG_EPI_WARPS);
    }
    mbar_init(done, 1);
    *gave_up = 0u;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(holder, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(
                     reinterpret_cast<uint64_t>(lane == 0 ? &mp.a : lane == 1 ? &mp.a32 : &mp.w))
                 : "memory");
  pdl_wait();
  fg_groups(a, rows, first);
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();   // the TMEM is allocated: no block of the next kernel can take it first
  tc_fence_after();
  const uint32_t tmem = *holder;
  const bool elected = elect_one();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FW_REGS_ROLE));
    if (warp == 0) {
      int s = 0;
      uint32_t ph = 0;
      int fills = 0;
      long long n = 0;
      bool live = !fg_held(a.ctl, kHoldLoads);
      FgTile tl = {};
      for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
        const int nrow = min(FG_BM, tl.m_end - tl.m0), pieces = nrow > 96 ? 0 : (nrow + 31) / 32;
        const uint32_t bytes = ((pieces ? pieces * 32 : FG_BM) + BN) * FG_BK;
        const int wrow = tl.g * a.N + tl.n0;
        for (int kb = 0; kb < KB; ++kb) {
          if (fills == stages) {
            live &= pipe_wait(&empty[s], ph ^ 1u, a.ctl, 0x411, gave_up);
          } else {
            ++fills;
          }
          if (elected && live) {
            ++n;
            unsigned char* st = smem + s * FW_STAGE;
            mbar_arrive_expect_tx(&full[s], bytes);
            if (pieces == 0) {
              fg_tma_2d(st, &mp.a, kb * FG_BK, tl.m0, &full[s]);
            } else {
              for (int p = 0; p < pieces; ++p)
                fg_tma_2d(st + p * 32 * FG_BK, &mp.a32, kb * FG_BK, tl.m0 + 32 * p, &full[s]);
            }
            fg_tma_2d(st + FW_HALF, &mp.w, kb * FG_BK, wrow, &full[s]);
          }
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (elected) pipe_drain(full, stages, n, a.ctl, 0x412);
    } else if (warp == 1) {
      const uint32_t idesc = idesc_f16_f32(FG_BM, BN);
      const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
      int s = 0, as = 0, used = 0;
      uint32_t ph = 0, aph = 0;
      bool live = !fg_held(a.ctl, kHoldMma);
      FgTile tl = {};
      for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
        for (int kb = 0; kb < KB; ++kb) {
          live &= pipe_wait(&full[s], ph, a.ctl, 0x414, gave_up);
          if (used == FW_SLOTS) {
            live &= pipe_wait(&acce[as], aph ^ 1u, a.ctl, 0x413, gave_up);
          } else {
            ++used;
          }
          tc_fence_after();
          if (elected && live) {
            const uint64_t ad = desc0 + (uint64_t)(s * (FW_STAGE >> 4)), bd = ad + (FW_HALF >> 4);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              fg_mma(tmem + (uint32_t)(as * BN), ad + 2 * i, bd + 2 * i, idesc, i > 0 ? 1u : 0u);
            tc_commit(&accf[as]);
            tc_commit(&empty[s]);
          }
          as ^= 1;
          if (as == 0) aph ^= 1u;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every MMA issued has completed before this warp frees the TMEM
      if (elected) tc_commit(done);
      mbar_wait(done, 0, a.ctl, 0x415);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(FW_REGS_EPI));
    constexpr int COLS = 128, LD = 32;
    const int ew = warp - 4, q = warp & 3, part = ew >> 2;     // part: the half of the columns
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(part * COLS);
    unsigned char* stage = out_s + ew * FW_OUT;
    const bool tma_out = (a.N & 7) == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0;
    int as = 0;
    uint32_t aph = 0;
    FgTile tl = {};
    for (long long t = blockIdx.x; fg_tile(t, a, BN, rows, first, &tl); t += gridDim.x) {
      const int row0 = tl.m0 + 32 * q, row = row0 + lane;
      const int col0 = tl.n0 + part * COLS;
      const bool idle = row0 >= tl.m_end || col0 >= a.N;
      const float* sa = a.a_scales + (long long)min(row, a.M - 1) * KB;
      const float* sw = a.w_scales +
                        ((long long)tl.g * blocks128(a.N) + min(col0, a.N - 1) / kBlock128) * KB;
      float2 acc[COLS / 2];
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      float sa_n = idle ? 0.f : sa[0], sw_n = idle ? 0.f : sw[0];
      for (int kb = 0; kb < KB; ++kb) {
        const float sc = sa_n * sw_n;
        if (!idle && kb + 1 < KB) {
          sa_n = sa[kb + 1];
          sw_n = sw[kb + 1];
        }
        pipe_wait(&accf[as], aph, a.ctl, 0x416, gave_up);
        __syncwarp();      // the TMEM loads are the whole warp's
        if (!idle) {
          tc_fence_after();
          const uint32_t base = lane_base + (uint32_t)(as * BN);
          const float2 sc2 = make_float2(sc, sc);
          uint32_t v[2][LD];
          fg_tmem_ld<LD>(base, v[0]);
#pragma unroll
          for (int i = 0; i < COLS / LD; ++i) {
            fg_tmem_wait<LD>(v[i & 1]);
            if (i + 1 < COLS / LD) {
              fg_tmem_ld<LD>(base + (uint32_t)((i + 1) * LD), v[(i + 1) & 1]);
            } else {
              // everything is in registers: hand the accumulator back before the last sums
              tc_fence_before();
              if (elected) fg_arrive(&acce[as]);
            }
#pragma unroll
            for (int x = 0; x < LD; x += 2)
              fma2(acc[(i * LD + x) / 2],
                   make_float2(__uint_as_float(v[i & 1][x]), __uint_as_float(v[i & 1][x + 1])), sc2);
          }
        } else if (elected) {
          fg_arrive(&acce[as]);
        }
        as ^= 1;
        if (as == 0) aph ^= 1u;
      }
      if (idle) continue;
      if (tma_out && (!a.offsets || row0 + 32 <= tl.m_end)) {
        // TMA stores of 32 rows x 64 columns (128-byte swizzle: piece p of row r at
        // p ^ (r & 7)); the copy clips rows and columns of no product, and the
        // second runs while the next tile is summed
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = acc[32 * h + 4 * p + j];
              const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
              w[j] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((p ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && col0 + 64 * h < a.N) {
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                    reinterpret_cast<uint64_t>(&mp.c)),
                "r"(col0 + 64 * h), "r"(row0), "r"(smem_u32(stage))
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      } else {
        // the staging buffer is free once the previous tile's store has read it
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        fg_store<COLS, 64>(a, acc, reinterpret_cast<uint32_t*>(stage), row0,
                           min(32, tl.m_end - row0), col0, lane);
        __syncwarp();
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Looked up once; calls of several threads that come first together each look it up
// and find the same.
PFN_cuTensorMapEncodeTiled_v12000 fg_encode() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = cached.load(std::memory_order_acquire);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
      cached.store(fn, std::memory_order_release);
    }
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

template <int BN, int AR>
cudaError_t fg_launch(const GemmArgs& a, long long tiles, cudaStream_t st) {
  // before the maps: this call makes the device's context current to a thread that
  // has made none yet, and the driver encodes no map without one
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fp8_gemm_kernel<BN, AR>),
                                   kMaxSmem);
  if (e != cudaSuccess) return e;
  FgMaps mp = {};
  if ((AR == FG_BM && !fg_map(&mp.a, a.a, (uint64_t)a.K, (uint64_t)a.M, FG_BM)) ||
      !fg_map(&mp.a32, a.a, (uint64_t)a.K, (uint64_t)a.M, 32) ||
      !fg_map(&mp.w, a.w, (uint64_t)a.K, (uint64_t)a.N * a.G, BN))
    return cudaErrorInvalidValue;
  const long long grid = tiles < sm_count() ? tiles : sm_count();
  return launch_pdl(fp8_gemm_kernel<BN, AR>, dim3((unsigned)grid), dim3(FG_THREADS),
                    FgCfg<BN, AR>::smem(a.G), st, a, mp);
}

cudaError_t fg_launch_wide(const GemmArgs& a, const GemmPlan& p, cudaStream_t st) {
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fp8_gemm_wide_kernel), kMaxSmem);
  if (e != cudaSuccess) return e;
  FgMaps mp = {};
  if (!fg_map(&mp.a, a.a, (uint64_t)a.K, (uint64_t)a.M, FG_BM) ||
      !fg_map(&mp.a32, a.a, (uint64_t)a.K, (uint64_t)a.M, 32) ||
      !fg_map(&mp.w, a.w, (uint64_t)a.K, (uint64_t)a.N * a.G, 256))
    return cudaErrorInvalidValue;
  if ((a.N & 7) == 0 && (reinterpret_cast<uintptr_t>(a.c) & 15) == 0) {
    cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)a.N * 2};
    cuuint32_t box[2] = {64, 32}, estr[2] = {1, 1};
    if (fg_encode()(&mp.c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.c, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // a block launched with fewer registers than the split hands out would wait for ever
  cudaFuncAttributes at;
  e = cudaFuncGetAttributes(&at, reinterpret_cast<const void*>(fp8_gemm_wide_kernel));
  if (e != cudaSuccess) return e;
  if (at.numRegs != FW_REGS) return cudaErrorInvalidConfiguration;
  const long long grid = p.tiles < sm_count() ? p.tiles : sm_count();
  return launch_pdl(fp8_gemm_wide_kernel, dim3((unsigned)grid), dim3(FW_THREADS),
                    fw_smem(p.stages, a.G), st, a, p.stages, mp);
}

}  // namespace

// The tile width with the least estimated time.  The estimate of a wave of tiles is
// the rows of A and of W that a block loads per k-block and a fixed part: no account of
// what bounds a kernel, but an order of the widths that measurement bears out.  Times
// in us by width, * the choice (G: groups):
//         M      N     K    G     16      32      64     128     256
//         4   2048  2048          5.0*    4.8     5.2     6.6
//         4   4096  2048          7.8     5.4*    5.5     6.7
//         4   8192  2048         12.3     8.3     6.4*    6.9
//         4  16384  2048         21.5    14.4    10.6     9.0*
//       100   2048  2048          5.6*    5.7     6.0     7.3    11.2
//       333   1000  1936          9.8     6.6*    7.6     9.8    13.6
//       512   4096  2048         25.6    16.4    10.6     8.2*   12.0
//      1024   4096  2048         47.9    26.4    18.1    14.2    12.5*
//      8192   4096  2048        359     186     105      84.8    73.9*
//        20   2048  2048  512    57.3    36.9    28.9    27.7*
//       640   2048   512  512   349     185     115      85.2    80.1*
//     5,000   1024  2048  512   766     398     220     191     201*
//    81,920   1024  2048  512  1362     724     459     361     353*
GemmPlan plan_fp8_gemm(int M, int N, int G, bool grouped, int sms) {
  // row tiles: the groups hold M rows in all, each at most one partial tile
  const int groups = grouped ? (G < M ? G : M) : 1;
  const long long mt = grouped ? M / FG_BM + groups : (M + FG_BM - 1) / FG_BM;
  const long long avg = groups ? ((long long)M + groups - 1) / groups : 0;
  const long long rows = avg >= FG_BM ? FG_BM : (avg + 31) / 32 * 32;
  const bool few = M <= 32;        // no tile has more than 32 rows
  GemmPlan p = {};
  long long best = 0;
  for (int b = few ? 128 : 256; b >= 16; b >>= 1) {
    const long long t = mt * ((N + b - 1) / b);
    const long long cost = (t + sms - 1) / sms * (rows + b + 32);
    // (equal cost: the wider, except that 256 has to be better)
    if (p.bn == 0 || cost < best || (p.bn == 256 && cost == best)) {
      best = cost;
      p.bn = b;
      p.tiles = t;
    }
  }
  p.a_rows = few ? 32 : FG_BM;
  p.stages = p.bn == 256   ? fw_stages(G)
             : p.bn == 128 ? (few ? FgCfg<128, 32>::kStages : FgCfg<128, 128>::kStages)
             : p.bn == 64  ? (few ? FgCfg<64, 32>::kStages : FgCfg<64, 128>::kStages)
             : p.bn == 32  ? (few ? FgCfg<32, 32>::kStages : FgCfg<32, 128>::kStages)
                           : (few ? FgCfg<16, 32>::kStages : FgCfg<16, 128>::kStages);
  return p;
}

cudaError_t launch_fp8_gemm(const GemmArgs& a, cudaStream_t st) {
  const GemmPlan p = plan_fp8_gemm(a.M, a.N, a.G, a.offsets != nullptr, sm_count());
  if (p.a_rows == 32) {
    switch (p.bn) {
      case 128: return fg_launch<128, 32>(a, p.tiles, st);
      case 64: return fg_launch<64, 32>(a, p.tiles, st);
      case 32: return fg_launch<32, 32>(a, p.tiles, st);
      default: return fg_launch<16, 32>(a, p.tiles, st);
    }
  }
  switch (p.bn) {
    case 256: return fg_launch_wide(a, p, st);
    case 128: return fg_launch<128, 128>(a, p.tiles, st);
    case 64: return fg_launch<64, 128>(a, p.tiles, st);
    case 32: return fg_launch<32, 128>(a, p.tiles, st);
    default: return fg_launch<16, 128>(a, p.tiles, st);
  }
}

}  // namespace moe
