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
// and 3). What hides their latency: the shared expert's gate/up units, which
// need no routing, run before the first; before the second, each block has
// asked for its down weights (an L2 prefetch per expert as soon as the experts
// are known, and its first tiles into registers).
//
// Weights go from global memory straight to registers: a lane's 16 consecutive
// codes are four k-steps of mma.sync m16n8k16 (the order in which k is summed
// is free, so lane t of a row takes codes 16t..16t+15 and the token operand is
// permuted to match). A unit of phase 3 is 8 hidden channels: rows 0-7 of the
// MMA's 16 are their gate rows and rows 8-15 their up rows, which leaves gate
// and up of one channel and token in one thread. Warp w holds the tokens'
// columns of scale block w (128 columns) in registers for the whole phase, so
// one scale per half of the tile and unit suffices. An e4m3 code becomes bf16
// exactly: its 7 magnitude bits in the bf16's field from bit 4 on are the value
// times 2^-120, subnormals included, and one packed multiply by 2^120
// restores it.
#include "ops.h"
#include "select.cuh"

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
  uint32_t done;     // blocks that are past every wait; the last one clears all three
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
  uint32_t* hidden;   // [U][8][Fmax] (bf16 hi, bf16 lo) pairs; the shared expert last
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

// Wait until *p reaches n; bounded like every wait of the library.
__device__ __forceinline__ bool grid_wait(const uint32_t* p, uint32_t n, Control* ctl,
                                          uint32_t where) {
  if (load_acquire(p) >= n) return true;
  const unsigned long long t0 = globaltimer_ns();
  unsigned long long limit = 0;
  for (;;) {
    if (load_acquire(p) >= n) return true;
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

// Streamed weights: read once, kept out of L1.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Four codes k0..k3 of a word to bf16 pairs (k0, k2) and (k1, k3).
__device__ __forceinline__ void dequant4(uint32_t w, uint32_t& p02, uint32_t& p13) {
  const uint32_t lo = and_or(w << 8, 0x80008000u, (w << 4) & 0x07F007F0u);
  const uint32_t hi = and_or(w, 0x80008000u, (w >> 4) & 0x07F007F0u);
  const __nv_bfloat162 up = __halves2bfloat162(__ushort_as_bfloat16(0x7B80), __ushort_as_bfloat16(0x7B80));
  const __nv_bfloat162 a = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&lo), up);
  const __nv_bfloat162 b = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&hi), up);
  p02 = *reinterpret_cast<const uint32_t*>(&a);
  p13 = *reinterpret_cast<const uint32_t*>(&b);
}

// D(16x8 f32) += A(16x16 bf16, row) * B(16x8 bf16, col)
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A unit's codes in flight: gate and up rows, two 64-column halves, and the
// scales of the two row blocks; NKB scale blocks of columns per warp.
template <int NKB>
struct FlUnit {
  uint4 v[NKB][4];     // gate j=0, gate j=1, up j=0, up j=1
  float sg[NKB], su[NKB];
};

template <int NKB>
__global__ void __launch_bounds__(FL_THREADS, 1) fp8_layer_kernel(FlArgs a) {
  const Fp8LayerDev& L = a.L;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const int nblk = gridDim.x, T = a.T, d = L.d;
  const int KBd = blocks128(d), KBf = blocks128(L.F), KBs = blocks128(L.Fs);

  __shared__ float4 s_red[2][FL_WARPS][32];
  __shared__ float s_part[4][4][FL_T];
  __shared__ int32_t s_ids[FL_T][16];
  __shared__ float s_w[FL_T][16];
  __shared__ uint32_t s_bits[32];
  __shared__ int s_pre[33];
  __shared__ int s_list[FL_MAX_U];             // unique experts, ascending
  __shared__ float s_mix[FL_MAX_U][FL_T];      // routing weight of (expert, token)
  __shared__ uint32_t s_sel[FL_MAX_U];         // bit t: token t selected the expert
  __shared__ int s_ok;

  pdl_wait();
  FlSync* sy = fl_sync(a.ctl);

  // ---- phase 1: logits of rows e = block, block + nblk, ...; four warps per
  // row, a quarter of the columns each
  {
    const int slot = warp >> 2, quarter = warp & 3;
    const int nc = d >> 2, c0 = quarter * nc / 4, c1 = (quarter + 1) * nc / 4;
    for (int e0 = blockIdx.x; e0 < L.E; e0 += 4 * nblk) {
      const int e = e0 + slot * nblk;
      float acc[FL_T];
#pragma unroll
      for (int t = 0; t < FL_T; ++t) acc[t] = 0.f;
      if (e < L.E) {
        const float4* wr = reinterpret_cast<const float4*>(L.Wr + (size_t)e * d);
#pragma unroll 4
        for (int c = c0 + lane; c < c1; c += 32) {
          const float4 wv = __ldg(wr + c);
#pragma unroll
          for (int t = 0; t < FL_T; ++t) {
            if (t < T) {
              const uint2 xv = *reinterpret_cast<const uint2*>(a.x + (size_t)t * d + 4 * c);
              acc[t] = fmaf(__uint_as_float(xv.x << 16), wv.x, acc[t]);
              acc[t] = fmaf(__uint_as_float(xv.x & 0xFFFF0000u), wv.y, acc[t]);
              acc[t] = fmaf(__uint_as_float(xv.y << 16), wv.z, acc[t]);
              acc[t] = fmaf(__uint_as_float(xv.y & 0xFFFF0000u), wv.w, acc[t]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < FL_T; ++t) {
          if (t < T) {
            const float s = warp_sum(acc[t]);
            if (lane == 0) s_part[slot][quarter][t] = s;
          }
        }
      }
      __syncthreads();
      if (tid < 4 * FL_T) {
        const int r = tid >> 3, t = tid & 7, er = e0 + r * nblk;
        if (er < L.E && t < T)
          a.logits[(size_t)t * L.E + er] = ((s_part[r][0][t] + s_part[r][1][t]) +
                                            (s_part[r][2][t] + s_part[r][3][t])) +
                                           (L.bias ? L.bias[er] : 0.f);
      }
      __syncthreads();
    }
  }
  if (tid == 0) grid_arrive(&sy->logits);   // after the barrier above: the block's stores are ordered before it

  // ---- the tokens as MMA operands: this warp's scale blocks
  uint32_t xb[NKB][8][2];
#pragma unroll
  for (int i = 0; i < NKB; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k0 = (warp + FL_WARPS * i) * kBlock128 + 64 * j + 16 * tq;
      uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
      if (g < T && k0 < d) {
        v0 = *reinterpret_cast<const uint4*>(a.x + (size_t)g * d + k0);
        v1 = *reinterpret_cast<const uint4*>(a.x + (size_t)g * d + k0 + 8);
      }
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        xb[i][4 * j + s][0] = __byte_perm(w[2 * s], w[2 * s + 1], 0x5410);
        xb[i][4 * j + s][1] = __byte_perm(w[2 * s], w[2 * s + 1], 0x7632);
      }
    }
  }

  int U = 0;                                     // unique routed experts
  const int n_sh = L.Fs >> 3, n_f = L.F >> 3;    // units of the shared and of one routed expert
  int parity = 0;                                // which s_red buffer

  // ---- phase 3 over units [q0, q1): shared units first, then routed ones
  auto run_units = [&](int q0, int q1) {
    auto issue = [&](FlUnit<NKB>& b, int q) {
      if (q >= q1) return;
      const bool sh = q < n_sh;
      const int u = sh ? 0 : (q - n_sh) / n_f, f0 = 8 * (sh ? q : (q - n_sh) - u * n_f);
      const int e = sh ? 0 : s_list[u];
      const int F = sh ? L.Fs : L.F;
      const int RB = sh ? KBs : KBf;
      const uint8_t* base = sh ? L.sgu : L.gu + (size_t)e * 2 * F * d;
      const float* sc = (sh ? L.sgus : L.gus + (size_t)e * 2 * RB * KBd) + (f0 / kBlock128) * KBd;
#pragma unroll
      for (int i = 0; i < NKB; ++i) {
        const int kb = warp + FL_WARPS * i;
        b.sg[i] = b.su[i] = 0.f;
        if (kb < KBd) {
          b.sg[i] = __ldg(sc + kb);
          b.su[i] = __ldg(sc + RB * KBd + kb);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int k0 = kb * kBlock128 + 64 * j + 16 * tq;
          const uint8_t* p = base + (size_t)(f0 + g) * d + k0;
          if (k0 < d) {
            b.v[i][j] = ld_stream(p);
            b.v[i][2 + j] = ld_stream(p + (size_t)F * d);
          } else {
            b.v[i][j] = b.v[i][2 + j] = make_uint4(0, 0, 0, 0);
          }
        }
      }
    };
    auto process = [&](const FlUnit<NKB>& b, int q, int turn) {
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NKB; ++i) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t g02, g13, u02, u13;
            dequant4(word(b.v[i][j], s), g02, g13);
            dequant4(word(b.v[i][2 + j], s), u02, u13);
            mma_bf16(acc, g02, u02, g13, u13, xb[i][4 * j + s][0], xb[i][4 * j + s][1]);
          }
        }
        sum.x = fmaf(acc[0], b.sg[i], sum.x);
        sum.y = fmaf(acc[1], b.sg[i], sum.y);
        sum.z = fmaf(acc[2], b.su[i], sum.z);
        sum.w = fmaf(acc[3], b.su[i], sum.w);
      }
      s_red[parity][warp][lane] = sum;
      __syncthreads();
      // two warps, taking turns, add the 16 column blocks: thread = (lane of
      // the tile, one of its two tokens)
      const int mine = (turn & 7) * 2;
      if (warp == mine || warp == mine + 1) {
        const int i = ((warp & 1) << 5) | lane, l = i >> 1, c = i & 1;
        const float* r = reinterpret_cast<const float*>(&s_red[parity][0][0]) + 4 * l + c;
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < FL_WARPS; ++w) {
          gate += r[w * 128];
          up += r[w * 128 + 2];
        }
        const bool sh = q < n_sh;
        const int u = sh ? 0 : (q - n_sh) / n_f, f0 = 8 * (sh ? q : (q - n_sh) - u * n_f);
        const int f = f0 + (l >> 2), t = 2 * (l & 3) + c;
        if (sh ? t < T : (s_sel[u] >> t) & 1u) {
          float h = gate / (1.f + expf(-gate)) * up;
          if (!sh) h *= s_mix[u][t];
          const __nv_bfloat16 hi = __float2bfloat16_rn(h);
          // two bf16 terms keep 16 mantissa bits (a residual below 2^-17 |h|);
          // an infinity or NaN stays in the first
          const float rest = h - __bfloat162float(hi);
          const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
          a.hidden[(size_t)(sh ? a.shared_u : u) * a.hstride + (size_t)t * (a.hstride >> 3) + f] =
              (uint32_t)__bfloat16_as_ushort(hi) | ((uint32_t)__bfloat16_as_ushort(lo) << 16);
        }
      }
      parity ^= 1;
    };
    constexpr int DEPTH = NKB == 1 ? 3 : 2;
    FlUnit<NKB> buf[DEPTH];
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) issue(buf[p], q0 + p * nblk);
    int turn = 0;
    for (int q = q0; q < q1; q += DEPTH * nblk) {
#pragma unroll
      for (int p = 0; p < DEPTH; ++p) {
        const int qq = q + p * nblk;
        if (qq < q1) {
          process(buf[p], qq, turn++);
          issue(buf[p], qq + DEPTH * nblk);
        }
      }
    }
  };

  run_units(blockIdx.x, n_sh);

  // ---- phase 2: selection, by every block for itself
  if (tid == 0) s_ok = grid_wait(&sy->logits, nblk, a.ctl, 0x500) ? 1 : 0;
  if (tid < 32) s_bits[tid] = 0u;
  for (int i = tid; i < FL_MAX_U * FL_T; i += FL_THREADS) (&s_mix[0][0])[i] = 0.f;
  if (tid < FL_MAX_U) s_sel[tid] = 0u;
  __syncthreads();
  const bool routed = s_ok != 0;
  if (routed) {
    if (warp < T)
      warp_topk(a.logits + (size_t)warp * L.E, nullptr, nullptr, L.E, L.k, s_ids[warp], s_w[warp],
                a.ctl, false);
    __syncthreads();
    const int pt = tid / L.k, pj = tid - pt * L.k;
    const bool pair = tid < T * L.k;
    const int e = pair ? s_ids[pt][pj] : 0;
    if (pair) {
      atomicOr(&s_bits[e >> 5], 1u << (e & 31));
      if (blockIdx.x == 0) {
        if (a.ids) a.ids[tid] = e;
        if (a.w) a.w[tid] = s_w[pt][pj];
      }
    }
    __syncthreads();
    if (warp == 0) {
      const int n = __popc(s_bits[lane]);
      int v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += up;
      }
      s_pre[lane] = v - n;
      if (lane == 31) s_pre[32] = v;
    }
    __syncthreads();
    if (pair) {
      const int u = s_pre[e >> 5] + __popc(s_bits[e >> 5] & ((1u << (e & 31)) - 1u));
      s_list[u] = e;                      // equal values from every token that chose e
      s_mix[u][pt] = s_w[pt][pj];
      atomicOr(&s_sel[u], 1u << pt);
    }
    __syncthreads();
    U = s_pre[32];

    // ask for this block's down rows: 16 rows of an expert are contiguous
    for (int r = blockIdx.x; r < (d >> 4); r += nblk) {
      for (int u = tid; u <= U; u += FL_THREADS) {
        if (u < U)
          prefetch_l2(L.dn + ((size_t)s_list[u] * d + 16 * r) * L.F, 16u * L.F);
        else if (L.Fs)
          prefetch_l2(L.sdn + (size_t)16 * r * L.Fs, 16u * L.Fs);
      }
    }
    // routed units follow the shared ones in one numbering over the blocks
    const int total = n_sh + U * n_f;
    int q = blockIdx.x;
    if (q < n_sh) q += (n_sh - q + nblk - 1) / nblk * nblk;
    run_units(q, total);
  }
  __syncthreads();
  if (tid == 0) {
    grid_arrive(&sy->hidden);
    s_ok = routed && grid_wait(&sy->hidden, nblk, a.ctl, 0x501) ? 1 : 0;
    // past every wait: the last block to get here clears the counters
    const uint32_t n = atomicAdd(&sy->done, 1u);
    if (n == (uint32_t)nblk - 1) {
      sy->logits = 0u;
      sy->hidden = 0u;
      sy->done = 0u;
    }
  }
  __syncthreads();
  if (s_ok == 0) return;

  // ---- phase 4: 16 output rows per tile; items (expert, scale block of F)
  // spread over the warps, each summed in registers, the warps joined in order
  const int n_items = U * KBf + (L.Fs ? KBs : 0);
  for (int r = blockIdx.x; r < (d >> 4); r += nblk) {
    const int row0 = 16 * r;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int it = warp; it < n_items; it += FL_WARPS) {
      const bool sh = it >= U * KBf;
      const int u = sh ? a.shared_u : it / KBf, kb = sh ? it - U * KBf : it - u * KBf;
      const int F = sh ? L.Fs : L.F;
      const size_t e = sh ? 0 : s_list[u];
      const uint8_t* base = sh ? L.sdn : L.dn + e * d * F;
      const float sc = sh ? __ldg(L.sdns + (row0 / kBlock128) * KBs + kb)
                          : __ldg(L.dns + (e * KBd + row0 / kBlock128) * KBf + kb);
      const bool sel = sh ? g < T : (s_sel[u] >> g) & 1u;
      const uint32_t* hp = a.hidden + (size_t)u * a.hstride + (size_t)g * (a.hstride >> 3);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k0 = kb * kBlock128 + 64 * j + 16 * tq;
        uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0, h[4] = {v0, v0, v0, v0};
        if (k0 < F) {
          v0 = ld_stream(base + (size_t)(row0 + g) * F + k0);
          v1 = ld_stream(base + (size_t)(row0 + g + 8) * F + k0);
          if (sel) {
#pragma unroll
            for (int s = 0; s < 4; ++s) h[s] = __ldcg(reinterpret_cast<const uint4*>(hp + k0) + s);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t a02, a13, c02, c13;
          dequant4(word(v0, s), a02, a13);
          dequant4(word(v1, s), c02, c13);
          mma_bf16(acc, a02, c02, a13, c13, __byte_perm(h[s].x, h[s].z, 0x5410),
                   __byte_perm(h[s].y, h[s].w, 0x5410));
          mma_bf16(acc, a02, c02, a13, c13, __byte_perm(h[s].x, h[s].z, 0x7632),
                   __byte_perm(h[s].y, h[s].w, 0x7632));
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) sum[c] = fmaf(acc[c], sc, sum[c]);
    }
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
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t fp8_layer_ws_bytes(const Fp8LayerDev& L) {
  const int Fmax = L.F > L.Fs ? L.F : L.Fs;
  return align256(sizeof(Control)) + align256((size_t)FL_T * L.E * 4) +
         align256((size_t)(FL_T * L.k + 1) * FL_T * Fmax * 4);
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
  a.hidden = reinterpret_cast<uint32_t*>(ws + align256(sizeof(Control)) +
                                         align256((size_t)FL_T * L.E * 4));
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
  return blocks128(L.d) <= FL_WARPS ? cudaLaunchKernelEx(&cfg, fp8_layer_kernel<1>, a)
                                    : cudaLaunchKernelEx(&cfg, fp8_layer_kernel<2>, a);
}

}  // namespace moe
