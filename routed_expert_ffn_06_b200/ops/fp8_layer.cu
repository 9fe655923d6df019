// fp8_layer.cu -- a whole MoE layer with e4m3 experts for a window of up to 8
// tokens, in one kernel: router, top-k selection, gate/up products with SwiGLU,
// down product, weighted sum.
//
//   logits[t][e] = sum_i x[t][i] Wr[e][i] + b[e]                    phase 1
//   (every block)  ids, w = top-k and softmax over the selected      phase 2
//   h[u][t] = w[t][u] silu(Wg_u x_t) (Wu_u x_t)                     phase 3
//   y[t] = sum_u Wd_u h[u][t]   (u: the window's experts, shared)   phase 4
//
// The layer is bound by the bytes of the window's experts, each read once. One
// block of 16 warps per SM; blocks meet at two grid barriers (after phases 1
// and 3). The shared expert, which needs no routing, goes to the L2 at the start
// and through phase 3 behind the routed ones (its units first, before the first
// barrier, kept the blocks that had one from the selection for 4 us); before the
// second barrier each warp has its first down weights on their way.
//
// Every warp streams its own weights through a ring of its own in shared memory
// (cp.async; a lane reads back what it asked for, so a warp waits for nobody), and
// no block barrier divides the stream: a unit of phase 3 (8 hidden channels of an
// expert: their gate rows and their up rows) is one warp's, which walks the
// whole of d; where a block has fewer units than warps, groups of S warps share
// one, each taking every S-th block of 128 columns.  What a
// call costs beside the bytes is mostly instruction fetches, since a small window
// runs most of the code once: the loops are short and not unrolled.  Measured on
// the way, 8 tokens of 512 experts (d 2048, ffn 512): all 16 warps on each unit
// by columns, added up between block barriers, 100 us; the same from rings of
// bulk copies 85 us; one warp per unit with rotating registers (loops unrolled
// four times) 79 us; this form 67 us (gate/up 27 us at 5 TB/s, down
// 23 us at 3.2 TB/s), and 25 us for one token.
//
// Rows 0-7 of the 16 of mma.sync m16n8k32 are gate rows and rows 8-15 the up
// rows of the same channels, which leaves gate and up of one channel and token in
// one thread. A lane's 16 consecutive codes are two k-steps (the order in which k
// is summed is free, so lane t of a row takes codes 16t..16t+15 and the token
// operand is permuted to match).
//
// Phase 3 multiplies e4m3 by e4m3, the weights as they are (121 cycles per SM for
// 32 KB of them, where converting them to fp16 and multiplying takes 356). The
// tokens are split into two e4m3 terms with separate sums: each 128 columns of a
// token are scaled by a power of two that brings their largest to 2^7..2^8, the
// first term holds the upper 4 bits of a value's 8, the second, times 16, the
// rest: exact down to 2^-13 of the block's largest, and off by at most 2^-21 of
// it below. Phase 4 multiplies fp16: the codes convert exactly, and the hidden
// values (fp32 in memory), scaled by a power of two per expert and token that
// brings the largest to 2^14..2^15, are the sum of two fp16 terms, so that each
// keeps 22 bits or an error below 2^-39 of the largest.  (The first term alone, 11
// bits, takes 64 us in place of 67 and is off by more than everything else in the
// layer together.)
#include "ops.h"
#include "select.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int FL_WARPS = 16;
constexpr int FL_THREADS = 32 * FL_WARPS;
constexpr int FL_T = kFp8Window;
constexpr int FL_MAX_U = FL_T * 16;     // unique routed experts of a window (top_k <= 16)

// The grid's counters, in the unused words of the workspace's control block.
struct FlSync {
  uint32_t logits;   // blocks whose logits are written
  uint32_t hidden;   // blocks whose hidden values are written
  uint32_t done;     // blocks that are through; the last one clears everything here
  uint32_t pad;
  uint32_t shared_top[kFp8Window];   // as FlArgs::top, of the shared expert
};
__device__ __forceinline__ FlSync* fl_sync(Control* c) { return reinterpret_cast<FlSync*>(c->pad); }

struct FlArgs {
  Fp8LayerDev L;
  const uint16_t* x;
  int T;
  uint16_t* y;
  int32_t* ids;       // or nullptr
  float* w;           // or nullptr
  Control* ctl;
  float* logits;      // [8][E]
  uint32_t* top;      // [U][8] bits of the largest |hidden value| of (expert, token)
  float* hidden;      // [U][8][Fmax], routing weights folded in; the shared expert last
  int hstride;        // elements of one expert's hidden block: 8 * Fmax
  int shared_u;       // the shared expert's index in hidden
};

__device__ __forceinline__ void grid_arrive(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Wait until *p reaches n (by signed distance: a counter that starts below zero has
// not reached it); bounded like every wait of the library.
__device__ __forceinline__ bool grid_wait(const uint32_t* p, uint32_t n, Control* ctl,
                                          uint32_t where) {
  if ((int32_t)(load_acquire(p) - n) >= 0) return true;
  const unsigned long long t0 = globaltimer_ns();
  unsigned long long limit = 0;
  for (;;) {
    if ((int32_t)(load_acquire(p) - n) >= 0) return true;
    const unsigned long long el = globaltimer_ns() - t0;
    if (el > kWaitFloorNs) {
      if (limit == 0) {
        const uint32_t us = *reinterpret_cast<volatile uint32_t*>(&ctl->wait_limit_us);
        limit = us ? 1000ull * us : kWaitLimitNs;
      }
      if (el > limit) {
        record_error(ctl, kErrTimeout, where);
        return false;
      }
    }
  }
}

// Four codes k0..k3 of a word to fp16 pairs (k0, k1) and (k2, k3).
__device__ __forceinline__ void dequant4h(uint32_t w, uint32_t& p01, uint32_t& p23) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(p01), "=r"(p23)
      : "r"(w));
}

// D(16x8 f32) += A(16x32 e4m3, row) * B(32x8 e4m3, col)
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats to two e4m3 codes (nearest, clamped), and what is left of them.
__device__ __forceinline__ uint32_t split_e4m3(float& a, float& b) {
  uint16_t c;
  uint32_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  const float2 f = __half22float2(u32_as_h2(h));
  a -= f.x;
  b -= f.y;
  return c;
}

// D(16x8 f32) += A(16x16 bf16, row) * B(16x8 bf16, col)
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with fp16 operands.
__device__ __forceinline__ void mma_half(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One warp selects the top k of E logits of one token, given as orderable keys in
// shared memory: ids largest first (equal values to the lower index, NaN below
// every number) and the softmax weights over the selected.  The k-th largest of
// the lanes' own maxima bounds the k-th largest logit from below, so the keys at
// or above it hold the whole selection; usually a dozen are left, which are
// ranked against each other at once.  More than 32 (many ties) take the
// round-by-round selection over the logits in memory.  The code runs once a call,
// so it is kept short: its time is instruction fetches more than work (unrolled
// over registers it took 7,000 cycles, this takes 3,000).
__device__ __noinline__ void fl_topk(const uint32_t* keys, const float* row, int E, int k,
                                     int32_t* ids, float* w, uint2* cand) {
  const int lane = threadIdx.x & 31;
  uint32_t best = 0u;
#pragma unroll 4
  for (int e = lane; e < E; e += 32) best = max(best, keys[e]);
  // the lane whose maximum ranks k-th (equal ones by lane; lanes past E last)
  int place = 0;
#pragma unroll 4
  for (int j = 0; j < 32; ++j) {
    const uint32_t o = __shfl_sync(0xffffffffu, best, j);
    place += (o > best || (o == best && j < lane)) ? 1 : 0;
  }
  const uint32_t kth = __ballot_sync(0xffffffffu, place == k - 1);
  const uint32_t thr = __shfl_sync(0xffffffffu, best, __ffs(kth) - 1);
  int n = 0;
#pragma unroll 4
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    const uint32_t key = e < E ? keys[e] : 0u;
    const bool c = e < E && key >= thr;
    const uint32_t m = __ballot_sync(0xffffffffu, c);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (c && at < 32) cand[at] = make_uint2(key, (uint32_t)e);
    n += __popc(m);
  }
  __syncwarp();
  if (n > 32) {
    warp_topk<true>(row, nullptr, nullptr, E, k, ids, w, nullptr, false);
    return;
  }
  const uint2 mine = lane < n ? cand[lane] : make_uint2(0u, 0xFFFFFFFFu);
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint2 o = cand[j];
    rank += (o.x > mine.x || (o.x == mine.x && o.y < mine.y)) ? 1 : 0;
  }
  const bool sel = lane < n && rank < k;
  const uint32_t top = __reduce_max_sync(0xffffffffu, mine.x);
  const float v0 = __uint_as_float((top & 0x80000000u) ? (top & 0x7FFFFFFFu) : ~top);
  const float mv = __uint_as_float((mine.x & 0x80000000u) ? (mine.x & 0x7FFFFFFFu) : ~mine.x);
  const float ex = sel ? expf(mv - v0) : 0.f;
  const float den = warp_sum(ex);
  if (sel) {
    ids[rank] = (int32_t)mine.y;
    w[rank] = ex / den;
  }
}

// 16 bytes (or, with on = false, zeros) to this lane's place of a ring slot.
// The L2 is asked for 256 bytes of a row at a time, the next column block with this
// one: the streams of all warps lie in tens of thousands of rows, and half as many
// visits to each took 8 tokens from 67.2 to 64.4 us (before the second term of the
// hidden values).
__device__ __forceinline__ void fl_copy16(unsigned char* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16u : 0u)
               : "memory");
}
__device__ __forceinline__ void fl_copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A warp's ring.  Phase 3: slots of a column block of a unit, gate and up rows in
// two 64-column halves, 2 KB.  Phase 4: slots of a column block of 16 rows of
// an expert, 2 KB, and its scale (a copy per lane).
constexpr int FL_DEPTH = 4, FL_SLOT = 2048;
constexpr int FL_DEPTH4 = 3, FL_SLOT4 = 2048 + 128;
constexpr int FL_MAX_KB = 32;    // column blocks of d
constexpr int FL_RING = FL_DEPTH * FL_SLOT;
static_assert(FL_RING >= FL_DEPTH4 * FL_SLOT4, "one ring serves both phases");

__global__ void __launch_bounds__(FL_THREADS, 1) fp8_layer_kernel(FlArgs a) {
  const Fp8LayerDev& L = a.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int nblk = gridDim.x, T = a.T, d = L.d;
  const int KBd = blocks128(d), KBf = blocks128(L.F), KBs = blocks128(L.Fs);
  const int n_sh = L.Fs >> 3, n_f = L.F >> 3;  // units of the shared and of one routed expert
  const int tiles = d >> 4;                    // row tiles of phase 4

  // the tokens as MMA operands: [column block][k-step of 32][lane] of
  // (first term b0, b1, second term b0, b1)
  extern __shared__ uint4 s_x[];               // then the warps' rings
  unsigned char* ring = reinterpret_cast<unsigned char*>(s_x + blocks128(d) * 128) +
                        (threadIdx.x >> 5) * FL_RING + (threadIdx.x & 31) * 16;
  // scales of a warp's present and next unit: gate, up, by column block.  With a
  // single column block the loads run four units ahead: four half-filled buffers
  __shared__ float s_scale[FL_WARPS][2][2][FL_MAX_KB];
  const int sbufs = KBd == 1 ? 4 : 2;
  __shared__ float2 s_xs[FL_MAX_KB][4];        // what undoes their scales, by pairs of tokens
  __shared__ float4 s_red[2][FL_WARPS][32];
  float(*s_part)[FL_T][8] = reinterpret_cast<float(*)[FL_T][8]>(s_red);   // phase 1: [warp][token][expert]
  __shared__ int32_t s_ids[FL_T][16];
  __shared__ float s_w[FL_T][16];
  __shared__ uint2 s_cand[FL_T][32];
  __shared__ uint32_t s_bits[32];
  __shared__ int s_list[FL_MAX_U];             // the window's experts, each once
  // routing weight of (expert, token) in phase 3; scale of its hidden values in
  // phase 4, the shared expert's at U
  __shared__ float s_mix[FL_MAX_U + 1][FL_T];
  __shared__ uint32_t s_sel[FL_MAX_U];         // bit t: token t selected the expert
  __shared__ int s_ok, s_u;

  pdl_wait();
  FlSync* sy = fl_sync(a.ctl);
  // read by nobody before the first grid barrier, raised by units after it
  for (int i = blockIdx.x * FL_THREADS + tid; i < FL_MAX_U * FL_T; i += nblk * FL_THREADS)
    a.top[i] = 0u;
  // the shared expert is known: its rows go to the L2 while the routing is found
  for (int i = blockIdx.x + nblk * tid; i < 2 * n_sh + (L.Fs ? tiles : 0); i += nblk * FL_THREADS) {
    if (i < 2 * n_sh)
      prefetch_l2(L.sgu + (size_t)i * 8 * d, 8u * d);
    else
      prefetch_l2(L.sdn + (size_t)(i - 2 * n_sh) * 16 * L.Fs, 16u * L.Fs);
  }

  // ---- phase 1: logits of rows e = block, block + nblk, ..., eight at a time as
  // the columns of mma.sync m16n8k16 (the tokens are its rows); warp w takes column
  // blocks w and w + 16.  The tokens are bf16 as they are; a weight is the exact
  // sum of three bf16 terms.
  for (int e0 = blockIdx.x; e0 < L.E; e0 += 8 * nblk) {
    const int e = e0 + g * nblk;
    float acc[3][4] = {};
#pragma unroll 1
    for (int kb = warp; kb < KBd; kb += FL_WARPS) {
      float4 wv[8];
      uint2 xv[8];
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const int k0 = kb * kBlock128 + 16 * m + 4 * tq;
        wv[m] = e < L.E && k0 < d ? __ldg(reinterpret_cast<const float4*>(L.Wr + (size_t)e * d + k0))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
        xv[m] = g < T && k0 < d ? *reinterpret_cast<const uint2*>(a.x + (size_t)g * d + k0)
                                : make_uint2(0u, 0u);
      }
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        float4 v = wv[m];
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y), q = __floats2bfloat162_rn(v.z, v.w);
          mma_bf16(acc[t], xv[m].x, 0u, xv[m].y, 0u, *reinterpret_cast<const uint32_t*>(&p),
                   *reinterpret_cast<const uint32_t*>(&q));
          const float2 pf = __bfloat1622float2(p), qf = __bfloat1622float2(q);
          v = make_float4(v.x - pf.x, v.y - pf.y, v.z - qf.x, v.w - qf.y);
        }
      }
    }
    // row g = token, columns 2 tq and 2 tq + 1 = experts
    *reinterpret_cast<float2*>(&s_part[warp][g][2 * tq]) =
        make_float2((acc[2][0] + acc[1][0]) + acc[0][0], (acc[2][1] + acc[1][1]) + acc[0][1]);
    __syncthreads();
    if (tid < 64) {
      const int t = tid >> 3, er = e0 + (tid & 7) * nblk;
      if (t < T && er < L.E) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < FL_WARPS; ++w) v += s_part[w][t][tid & 7];
        a.logits[(size_t)t * L.E + er] = v + (L.bias ? L.bias[er] : 0.f);
      }
    }
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) grid_arrive(&sy->logits);   // after a block barrier: the block's stores are ordered before it

  // ---- the tokens as MMA operands: warp w splits column blocks w and w + 16
  for (int kb = warp; kb < KBd; kb += FL_WARPS) {
    uint32_t w[2][8];
    uint32_t top = 0;                            // exponent field of the largest magnitude
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k0 = kb * kBlock128 + 64 * j + 16 * tq;
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (g < T && k0 < d) {
        v0 = *reinterpret_cast<const uint4*>(a.x + (size_t)g * d + k0);
        v1 = *reinterpret_cast<const uint4*>(a.x + (size_t)g * d + k0 + 8);
      }
      w[j][0] = v0.x, w[j][1] = v0.y, w[j][2] = v0.z, w[j][3] = v0.w;
      w[j][4] = v1.x, w[j][5] = v1.y, w[j][6] = v1.z, w[j][7] = v1.w;
#pragma unroll
      for (int s = 0; s < 8; ++s)
        top = max(top, max((w[j][s] >> 7) & 0xFFu, (w[j][s] >> 23) & 0xFFu));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^e with e = 7 - (top - 127), held to what fp32 can undo; a block with an
    // infinity or NaN (field 255) makes its token's sums NaN
    const int e = min(134 - (int)top, 120);
    const float f = __uint_as_float((uint32_t)(e + 127) << 23);
    const float undo = top == 255u ? __uint_as_float(0x7FC00000u)
                                   : __uint_as_float((uint32_t)(127 - e) << 23);
    if (tq == 0) reinterpret_cast<float*>(&s_xs[kb][0])[g] = undo;
#pragma unroll
    for (int m = 0; m < 4; ++m) {                // k-steps: 8 columns a lane, two words of codes
      uint32_t b[4];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        float c[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = w[m >> 1][4 * (m & 1) + 2 * s + x];
          c[2 * x] = __uint_as_float(v << 16) * f;
          c[2 * x + 1] = __uint_as_float(v & 0xFFFF0000u) * f;
        }
        b[s] = split_e4m3(c[0], c[1]) | (split_e4m3(c[2], c[3]) << 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) c[x] *= 16.f;
        b[2 + s] = split_e4m3(c[0], c[1]) | (split_e4m3(c[2], c[3]) << 16);
      }
      s_x[(kb * 4 + m) * 32 + lane] = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
  __syncthreads();

  int U = 0;                                   // unique routed experts
  // ---- phase 3 over the block's units, block, block + nblk, ... of one
  // numbering: the routed experts' units, then the shared expert's
  auto run_units = [&]() {
    const int n_r = U * n_f, all = n_r + n_sh, q0 = blockIdx.x;
    const int n = q0 < all ? (all - q0 + nblk - 1) / nblk : 0;    // the block's units
    if (n == 0) return;
    // warps that share a unit; with more than one, every group has one unit at most
    const int S = max(1, min(FL_WARPS / n, KBd));
    const int groups = FL_WARPS / S, grp = warp / S, rank = warp - grp * S;
    int parity = 0;
    // the next column block to ask for
    const uint8_t* base;
    size_t up;
    int ai = grp, ak = rank, aslot = 0, abuf = 0;
    auto ask = [&]() {
      if (ai < n) {
        if (ak == rank) {                      // a new unit: its addresses, and its scales
          const int q = q0 + ai * nblk;
          const bool sh = q >= n_r;
          const int u = sh ? 0 : q / n_f, f0 = 8 * (sh ? q - n_r : q - u * n_f);
          const int F = sh ? L.Fs : L.F, RB = sh ? KBs : KBf;
          const size_t e = sh ? 0 : s_list[u];
          base = (sh ? L.sgu : L.gu + e * 2 * F * d) + (size_t)(f0 + g) * d + 16 * tq;
          up = (size_t)F * d;
          const float* sc = (sh ? L.sgus : L.gus + e * 2 * RB * KBd) + (f0 / kBlock128) * KBd;
          if (lane < KBd) {
            float* o = &s_scale[warp][abuf & 1][0][16 * (abuf >> 1) + lane];
            fl_copy4(o, sc + lane);
            fl_copy4(o + FL_MAX_KB, sc + RB * KBd + lane);
          }
          abuf = (abuf + 1) & (sbufs - 1);
        }
        const uint8_t* p = base + ak * kBlock128;
        const int k0 = ak * kBlock128 + 16 * tq;
        unsigned char* o = ring + aslot * FL_SLOT;
        fl_copy16(o, p, k0 < d);
        fl_copy16(o + 512, p + up, k0 < d);
        fl_copy16(o + 1024, p + 64, k0 + 64 < d);
        fl_copy16(o + 1536, p + up + 64, k0 + 64 < d);
        ak += S;
        if (ak >= KBd) {
          ak = rank;
          ai += groups;
        }
      }
      aslot = (aslot + 1) & (FL_DEPTH - 1);
      cp_async_commit();
    };
    for (int i = 0; i < FL_DEPTH; ++i) ask();
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    int ci = grp, ck = rank, cslot = 0, cbuf = 0;   // the column block to compute
    float sg = 0.f, su = 0.f;                  // the unit's scales: lane = column block
#pragma unroll 1
    while (ci < n) {
          cp_async_wait<FL_DEPTH - 1>();
          const uint4* b = reinterpret_cast<const uint4*>(ring + cslot * FL_SLOT);
          const uint4 g0 = b[0], u0 = b[32], g1 = b[64], u1 = b[96];
          if (ck == rank) {
            const float* o = &s_scale[warp][cbuf & 1][0][16 * (cbuf >> 1) + (KBd == 1 ? 0 : lane)];
            sg = o[0];
            su = o[FL_MAX_KB];
            cbuf = (cbuf + 1) & (sbufs - 1);
          }
          float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
          const uint4* xo = s_x + ck * 128 + lane;
          const uint4 x0 = xo[0], x1 = xo[32], x2 = xo[64], x3 = xo[96];
          mma_e4m3(hi, g0.x, u0.x, g0.y, u0.y, x0.x, x0.y);
          mma_e4m3(lo, g0.x, u0.x, g0.y, u0.y, x0.z, x0.w);
          mma_e4m3(hi, g0.z, u0.z, g0.w, u0.w, x1.x, x1.y);
          mma_e4m3(lo, g0.z, u0.z, g0.w, u0.w, x1.z, x1.w);
          mma_e4m3(hi, g1.x, u1.x, g1.y, u1.y, x2.x, x2.y);
          mma_e4m3(lo, g1.x, u1.x, g1.y, u1.y, x2.z, x2.w);
          mma_e4m3(hi, g1.z, u1.z, g1.w, u1.w, x3.x, x3.y);
          mma_e4m3(lo, g1.z, u1.z, g1.w, u1.w, x3.z, x3.w);
          const float fg = __shfl_sync(0xffffffffu, sg, ck), fu = __shfl_sync(0xffffffffu, su, ck);
          const float2 xs = s_xs[ck][tq];
          sum.x = fmaf(fmaf(lo[0], 0.0625f, hi[0]) * xs.x, fg, sum.x);
          sum.y = fmaf(fmaf(lo[1], 0.0625f, hi[1]) * xs.y, fg, sum.y);
          sum.z = fmaf(fmaf(lo[2], 0.0625f, hi[2]) * xs.x, fu, sum.z);
          sum.w = fmaf(fmaf(lo[3], 0.0625f, hi[3]) * xs.y, fu, sum.w);
          ask();                               // the slot's values are in registers
          cslot = (cslot + 1) & (FL_DEPTH - 1);
          ck += S;
          if (ck >= KBd) {
            // the unit's end: its warps' sums meet in the first of them
            if (S > 1) {
              s_red[parity][warp][lane] = sum;
              named_bar_sync(1 + grp, 32 * S);
              if (rank == 0)
                for (int r = 1; r < S; ++r) {
                  const float4 o = s_red[parity][warp + r][lane];
                  sum.x += o.x, sum.y += o.y, sum.z += o.z, sum.w += o.w;
                }
              parity ^= 1;
            }
            if (rank == 0) {
              const int q = q0 + ci * nblk;
              const bool sh = q >= n_r;
              const int u = sh ? 0 : q / n_f, f0 = 8 * (sh ? q - n_r : q - u * n_f);
              const uint32_t sel = sh ? (1u << T) - 1u : s_sel[u];
              float* out = a.hidden + (size_t)(sh ? a.shared_u : u) * a.hstride + f0 + g;
              uint32_t* top = sh ? sy->shared_top : a.top + u * FL_T;
#pragma unroll 1
              for (int c = 0; c < 2; ++c) {
                const int t = 2 * tq + c;
                const bool on = (sel >> t) & 1u;
                const float gate = c ? sum.y : sum.x, upv = c ? sum.w : sum.z;
                float h = gate / (1.f + expf(-gate)) * upv;
                if (!sh) h *= s_mix[u][t];
                if (on) out[t * (a.hstride >> 3)] = h;
                // the largest of the unit's channels of a token, then of all units'
                uint32_t big = on ? __float_as_uint(h) & 0x7FFFFFFFu : 0u;
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 4));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 8));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 16));
                if (on && g == 0) atomicMax(top + t, big);
              }
            }
            sum = make_float4(0.f, 0.f, 0.f, 0.f);
            ck = rank;
            ci += groups;
          }
    }
    cp_async_wait<0>();                        // the empty groups at the end
  };
  // ---- phase 2: selection, by every block for itself
  if (tid == 0) s_ok = grid_wait(&sy->logits, nblk, a.ctl, 0x500) ? 1 : 0;
  if (tid < 32) s_bits[tid] = 0u;
  for (int i = tid; i < FL_MAX_U * FL_T; i += FL_THREADS) (&s_mix[0][0])[i] = 0.f;
  if (tid < FL_MAX_U) s_sel[tid] = 0u;
  __syncthreads();
  const bool ok = s_ok != 0;
  int down_end = 0;                            // experts of phase 4, the shared one included
  if (ok) {
    // keys of as many tokens at a time as the sums' buffer holds (four at least)
    uint32_t* keys = reinterpret_cast<uint32_t*>(s_red);
    const int group = min(T, (int)(sizeof(s_red) / 4) / L.E);
    for (int t0 = 0; t0 < T; t0 += group) {
      const int n = min(group, T - t0);
#pragma unroll 4
      for (int i = tid; i < n * L.E; i += FL_THREADS)
        keys[i] = order_key(__ldcg(a.logits + (size_t)t0 * L.E + i));
      __syncthreads();
      if (warp < n) {
        const int t = t0 + warp;
        fl_topk(keys + warp * L.E, a.logits + (size_t)t * L.E, L.E, L.k, s_ids[t], s_w[t],
                s_cand[warp]);
        __syncwarp();
        if (lane < L.k) atomicOr(&s_bits[s_ids[t][lane] >> 5], 1u << (s_ids[t][lane] & 31));
      }
      __syncthreads();
    }
    if (T == 1) {
      // a single token's experts are its list, in its order
      if (tid < L.k) {
        s_list[tid] = s_ids[0][tid];
        s_mix[tid][0] = s_w[0][tid];
        s_sel[tid] = 1u;
        if (tid == 0) s_u = L.k;
      }
    } else if (warp < T) {
      // the unique experts in ascending order: a bitmap and its prefix counts, by
      // the warp of each token
      const uint32_t bits = s_bits[lane];
      const int n = __popc(bits);
      int v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      if (warp == 0 && lane == 31) s_u = v;
      const int e = lane < L.k ? s_ids[warp][lane] : 0;
      const int before = __shfl_sync(0xffffffffu, v - n, e >> 5);
      const uint32_t same = __shfl_sync(0xffffffffu, bits, e >> 5);
      if (lane < L.k) {
        const int u = before + __popc(same & ((1u << (e & 31)) - 1u));
        s_list[u] = e;                        // equal values from every token that chose e
        s_mix[u][warp] = s_w[warp][lane];
        atomicOr(&s_sel[u], 1u << warp);
      }
    }
    if (warp == 1 && blockIdx.x == 0) {
      for (int i = lane; i < T * L.k; i += 32) {
        if (a.ids) a.ids[i] = s_ids[i / L.k][i % L.k];
        if (a.w) a.w[i] = s_w[i / L.k][i % L.k];
      }
    }
    __syncthreads();
    U = s_u;
    down_end = U + (L.Fs ? 1 : 0);
    run_units();
  }

  // ---- phase 4: 16 output rows per tile; items (expert, column block of F), the
  // shared expert's last, spread over the warps, each summed in registers, the
  // warps joined in order
  const int n_items = U * KBf + (down_end > U ? KBs : 0);
  struct Item {
    int it, u, kb;                             // u == U: the shared expert
  };
  auto start = [&]() {
    Item m;
    m.it = warp;
    m.u = min(warp / KBf, U);
    m.kb = warp - m.u * KBf;
    return m;
  };
  const int du = FL_WARPS / KBf, dk = FL_WARPS - du * KBf;
  auto step = [&](Item& m) {
    m.it += FL_WARPS;
    m.u += du;
    m.kb += dk;
    if (m.kb >= KBf) {
      m.kb -= KBf;
      ++m.u;
    }
    if (m.it >= U * KBf) {
      m.u = U;
      m.kb = m.it - U * KBf;
    }
  };
  auto ask_w = [&](int slot, const Item& m, int row0) {
    if (m.it < n_items) {
      const bool sh = m.u == U;
      const int F = sh ? L.Fs : L.F;
      const size_t e = sh ? 0 : s_list[m.u];
      const int k0 = m.kb * kBlock128 + 16 * tq;
      const uint8_t* p = (sh ? L.sdn : L.dn + e * d * F) + (size_t)(row0 + g) * F + k0;
      const uint8_t* p8 = p + 8 * (size_t)F;
      unsigned char* o = ring + slot * FL_SLOT4;
      fl_copy16(o, p, k0 < F);
      fl_copy16(o + 512, p8, k0 < F);
      fl_copy16(o + 1024, p + 64, k0 + 64 < F);
      fl_copy16(o + 1536, p8 + 64, k0 + 64 < F);
      fl_copy4(o + 2048 - 12 * lane, (sh ? L.sdns + (row0 / kBlock128) * KBs
                                         : L.dns + (e * KBd + row0 / kBlock128) * KBf) + m.kb);
    }
    cp_async_commit();
  };
  auto load_h = [&](float4 (&h)[8], const Item& m) {
    const bool sh = m.u == U;
    const int k0 = m.kb * kBlock128 + 16 * tq, F = sh ? L.Fs : L.F;
    const bool sel = m.it < n_items && (sh ? g < T : (s_sel[m.u] >> g) & 1u);
    const float4* hp = reinterpret_cast<const float4*>(
        a.hidden + (size_t)(sh ? a.shared_u : m.u) * a.hstride + (size_t)g * (a.hstride >> 3) + k0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool on = sel && k0 + 64 * j < F;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        h[4 * j + s] = on ? __ldcg(hp + 16 * j + s) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  if (blockIdx.x < tiles) {
    Item m = start();
    for (int i = 0; i < FL_DEPTH4; ++i) {
      ask_w(i, m, 16 * blockIdx.x);
      step(m);
    }
  }
  __syncthreads();
  if (tid == 0) {
    grid_arrive(&sy->hidden);
    grid_wait(&sy->hidden, nblk, a.ctl, 0x501);
  }
  __syncthreads();
  float4 h[2][8];                              // hidden values, one item ahead
  if (blockIdx.x < tiles) load_h(h[0], start());
  for (int i = tid; i < down_end * FL_T; i += FL_THREADS) {
    const int u = i >> 3, t = i & 7;
    const int top = (int)(__ldcg(u < U ? &a.top[i] : &sy->shared_top[t]) >> 23);
    const int e = top == 255 ? 0 : min(141 - top, 120);      // as the tokens', to 2^14..2^15
    // 0 marks a token that did not select the expert: whatever the expert's weights
    // are, NaN included, the token's sums leave its products out
    const bool on = u < U ? (s_sel[u] >> t) & 1u : t < T;
    s_mix[u][t] = on ? __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
  }
  __syncthreads();

  for (int r = blockIdx.x; r < tiles; r += nblk) {
    const int row0 = 16 * r;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    Item m = start(), ahead = m, hm = m;
    if (r != blockIdx.x) load_h(h[0], hm);
    for (int i = 0; i < FL_DEPTH4; ++i) {
      if (r != blockIdx.x) ask_w(i, ahead, row0);
      step(ahead);
    }
    int slot = 0;
#pragma unroll 1
    while (m.it < n_items) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x == 1 && m.it >= n_items) break;
        step(hm);
        load_h(h[x ^ 1], hm);
        cp_async_wait<FL_DEPTH4 - 1>();
        const unsigned char* o = ring + slot * FL_SLOT4;
        const float sc = *reinterpret_cast<const float*>(o + 2048 - 12 * lane);
        const float f = s_mix[m.u][g];
        // the scales of the two tokens whose sums this thread receives are powers
        // of two: 2^-e from 2^e by the exponent field
        const float2 mx = *reinterpret_cast<const float2*>(&s_mix[m.u][2 * tq]);
        const float i0 = __uint_as_float((254u << 23) - __float_as_uint(mx.x)) * sc;
        const float i1 = __uint_as_float((254u << 23) - __float_as_uint(mx.y)) * sc;
        float acc[2][4] = {};                  // two chains of MMAs
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4 v0 = *reinterpret_cast<const uint4*>(o + 1024 * j);
          const uint4 v1 = *reinterpret_cast<const uint4*>(o + 1024 * j + 512);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t a01, a23, c01, c23;
            dequant4h(word(v0, s), a01, a23);
            dequant4h(word(v1, s), c01, c23);
            const float4 hv = h[x][4 * j + s];   // times f, as two fp16 terms
            const float2 v01 = make_float2(hv.x * f, hv.y * f), v23 = make_float2(hv.z * f, hv.w * f);
            const __half2 p01 = __float22half2_rn(v01), p23 = __float22half2_rn(v23);
            mma_half(acc[j], a01, c01, a23, c23, h2_as_u32(p01), h2_as_u32(p23));
            const float2 q01 = __half22float2(p01), q23 = __half22float2(p23);
            mma_half(acc[j], a01, c01, a23, c23,
                     h2_as_u32(__floats2half2_rn(v01.x - q01.x, v01.y - q01.y)),
                     h2_as_u32(__floats2half2_rn(v23.x - q23.x, v23.y - q23.y)));
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((c & 1 ? mx.y : mx.x) != 0.f)
            sum[c] = fmaf(acc[0][c] + acc[1][c], c & 1 ? i1 : i0, sum[c]);
        ask_w(slot, ahead, row0);              // the slot's values are in registers
        step(ahead);
        m = hm;
        if (++slot == FL_DEPTH4) slot = 0;
      }
    }
    cp_async_wait<0>();
    s_red[0][warp][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    __syncthreads();
    if (tid < 128) {
      const int l = tid >> 2, c = tid & 3;
      const float* p = reinterpret_cast<const float*>(&s_red[0][0][0]) + tid;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < FL_WARPS; ++w) v += p[w * 128];
      const int t = 2 * (l & 3) + (c & 1), row = row0 + (l >> 2) + 8 * (c >> 1);
      if (t < T) a.y[(size_t)t * d + row] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    __syncthreads();
  }
  // the last block clears what the next call finds
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&sy->done, 1u) == (uint32_t)nblk - 1) {
      sy->logits = 0u;
      sy->hidden = 0u;
      sy->done = 0u;
      for (int t = 0; t < FL_T; ++t) sy->shared_top[t] = 0u;
    }
  }
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t fp8_layer_ws_bytes(const Fp8LayerDev& L) {
  const int Fmax = L.F > L.Fs ? L.F : L.Fs;
  return align256(sizeof(Control)) + align256((size_t)FL_T * L.E * 4) +
         align256((size_t)FL_MAX_U * FL_T * 4) + align256((size_t)(FL_T * L.k + 1) * FL_T * Fmax * 4);
}

cudaError_t launch_fp8_layer(const Fp8LayerDev& L, const uint16_t* x, int T, uint16_t* y,
                             int32_t* ids, float* w, char* ws, cudaStream_t st) {
  const int Fmax = L.F > L.Fs ? L.F : L.Fs;
  FlArgs a;
  a.L = L;
  a.x = x;
  a.T = T;
  a.y = y;
  a.ids = ids;
  a.w = w;
  a.ctl = reinterpret_cast<Control*>(ws);
  a.logits = reinterpret_cast<float*>(ws + align256(sizeof(Control)));
  a.top = reinterpret_cast<uint32_t*>(ws + align256(sizeof(Control)) +
                                      align256((size_t)FL_T * L.E * 4));
  a.hidden = reinterpret_cast<float*>(reinterpret_cast<char*>(a.top) +
                                      align256((size_t)FL_MAX_U * FL_T * 4));
  a.hstride = FL_T * Fmax;
  a.shared_u = FL_T * L.k;
  // cooperative: the blocks wait for one another, so all of them are resident
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sm_count());
  cfg.blockDim = dim3(FL_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = (size_t)blocks128(L.d) * 4 * 32 * sizeof(uint4) + FL_WARPS * FL_RING;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fp8_layer_kernel),
                                   FL_MAX_KB * 128 * sizeof(uint4) + FL_WARPS * FL_RING);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, fp8_layer_kernel, a);
}

}  // namespace moe
