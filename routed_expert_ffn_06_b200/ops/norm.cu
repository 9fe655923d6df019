// norm.cu -- the norms before and after a block, fused with the block's gate
// and the residual scales, and the quantiser of bf16 rows to e4m3.
//
//   u = y [* rsqrt(mean(y^2) + eps) * W(post_w)]
//   r = a x + b act(gate) u              -> x_out
//   h = r * rsqrt(mean(r^2) + eps) * W(pre_w)   -> bf16 and/or e4m3 with a
//                                           scale per 128 columns
//
// One pass over memory: a row stays in registers between the loads and the
// stores, so every byte is read once and written once.  Many rows are bound by
// HBM with the second norm alone (8192 x 2048: 22.5 us, 6.0 TB/s), by the instructions
// issued with a post norm (27.0 us, 5.0 TB/s) and with a gate and the quantiser as
// well (35.4 us, 5.2 TB/s); one row by its launch and two dependent reductions.
// A thread owns chunks of 8 consecutive channels (16-byte accesses in bf16).
// Rows of up to 512 channels take one warp each (no block barrier); wider rows
// take a block each, of as many threads as chunks (measured: 777 x 1000 channels
// 3.9 us against 6.6 us with a warp per row, 8192 x 1024 17.5 against 22.6; at
// 30,000 x 512 the warps win, 22.0 against 32.4).  Blocks that walk the rows,
// with the weights in registers and the next row on its way, gained 2% at
// 8192 x 2048 and lost 20% at 8192 x 1024.  128 channels are 16 chunks = 16
// consecutive lanes, so the largest |h| of a scale block is a half-warp maximum.
#include "ops.h"

namespace moe {

namespace {

// Channels are held in pairs: fp32 arithmetic on a pair is one instruction
// (fma.rn.f32x2), each half rounded as alone.
__device__ __forceinline__ unsigned long long bits64(float2 v) {
  return *reinterpret_cast<const unsigned long long*>(&v);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits64(a)), "l"(bits64(b)), "l"(bits64(c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits64(a)), "l"(bits64(b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits64(a)), "l"(bits64(b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&o)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load8f(const float* p, float2 (&o)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  o[0] = make_float2(a.x, a.y), o[1] = make_float2(a.z, a.w);
  o[2] = make_float2(b.x, b.y), o[3] = make_float2(b.z, b.w);
}

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Four floats to four e4m3 codes, nearest with ties to even, clamped to +-448.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Quantise one chunk of 8 channels of a block of 16 lanes.  A NaN or infinity
// survives the maximum.  `live`: the chunk lies inside the row (all lanes of the
// warp call this).
__device__ __forceinline__ void quant8(const float2 (&v)[4], bool live, uint8_t* codes,
                                       float* scale) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max3_abs(top, v[j].x, v[j].y);
  if (!live) top = 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max3_abs(top, __shfl_xor_sync(0xffffffffu, top, o), 0.f);
  if (!live) return;
  // Both quotients are rounded as by a division: a product with the reciprocal, and
  // what it leaves of the dividend (exact, by fma) divided again.
  float s = top * (1.f / kE4m3Max);
  s = fmaf(fmaf(-s, kE4m3Max, top), 1.f / kE4m3Max, s);
  float2 q[4];
  if (top > 1e-24f && top < 1e38f) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[j] = mul2(v[j], both(inv));
      q[j] = fma2(fma2(q[j], both(-s), v[j]), both(inv), q[j]);
    }
  } else {   // zeros, values whose remainders underflow, infinities, NaN
    s = top / kE4m3Max;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = s != 0.f ? make_float2(v[j].x / s, v[j].y / s) : v[j];
  }
  *reinterpret_cast<uint2*>(codes) =
      make_uint2(e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y), e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
  if ((threadIdx.x & 15) == 0) *scale = s;
}

// Sum over the row's threads: a warp, or the whole block (red: a float per
// warp; one barrier, so two sums of one row use two arrays).
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (WARP_ROW) return v;
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < nw ? red[lane] : 0.f);
}

// 1 / (1 + e^-x): the fast exponential is off by 2 + 1.2 |x| last bits and the fast
// division by 2, which is 2^-21 of 1 at most; exact division and exp took a third
// of the kernel's time.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

constexpr int kWarpRows = 4;   // rows (warps) of a block when a row takes one warp

// 32 registers keep two blocks of 1024 threads, or eight of 256, on an SM, and spill
// 16 bytes a thread; without the bound one token of 2048 channels takes 2.29 us in
// place of 2.13, 8192 x 1024 17.7 in place of 17.4, and the rows bound by issue gain:
// 8192 x 2048 34.6 in place of 35.4, 2048 x 8192 36.3 in place of 37.6.  Pairs in
// place of single floats took 8192 x 2048 from 37.1 to 35.5 us and 30,000 x 512 from
// 22.7 to 22.0.
template <bool F32, bool WARP_ROW, int CH>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kWarpRows : 1024, WARP_ROW ? 1 : 2) norm_block_kernel(NormArgs a) {
  __shared__ float red[2][32];
  const int lane = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int nt = WARP_ROW ? 32 : blockDim.x;
  const int row = WARP_ROW ? blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (WARP_ROW && row >= a.T) return;
  const int nc = a.d >> 3;
  float2 r[CH][4];         // the stream, then r
  uint4 yv[CH], gv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * nt;
    const bool live = c < nc;
    if (F32) {
      if (live) {
        load8f(static_cast<const float*>(a.x) + row * a.x_ld + 8 * c, r[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = both(0.f);
      }
    } else {
      const uint4 xv = live ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) +
                                                              row * a.x_ld + 8 * c)
                            : make_uint4(0, 0, 0, 0);
      unpack8(xv, r[i]);
    }
    yv[i] = gv[i] = make_uint4(0, 0, 0, 0);
    if (a.y && live) yv[i] = *reinterpret_cast<const uint4*>(a.y + row * a.y_ld + 8 * c);
    if (a.gate_kind >= MOE_GATE_CHANNEL && live)
      gv[i] = *reinterpret_cast<const uint4*>(
          a.gate + (a.gate_kind == MOE_GATE_FULL ? row * a.gate_ld : 0ll) + 8 * c);
  }
  float gt = 1.f;
  if (a.gate_kind == MOE_GATE_TOKEN) {
    gt = bf16_bits_to_float(a.gate[row]);
    if (a.sigmoid) gt = sigmoid(gt);
  }
  float inv_y = 1.f;
  if (a.post) {
    float2 ss = both(0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float2 v[4];
      unpack8(yv[i], v);
#pragma unroll
      for (int j = 0; j < 4; ++j) ss = fma2(v[j], v[j], ss);
    }
    inv_y = rsqrtf(row_sum<WARP_ROW>(ss.x + ss.y, red[0]) * a.inv_d + a.eps);
  }
  float2 ss = both(0.f);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * nt;
    float2 u[4], g[4];
    unpack8(yv[i], u);
    if (a.post) {
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], both(inv_y));
      if (a.post_w && c < nc) {
        float2 w[4];
        load8f(a.post_w + 8 * c, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], add2(w[j], both(a.w_off)));
      }
    }
    if (a.gate_kind >= MOE_GATE_CHANNEL) {
      unpack8(gv[i], g);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = mul2(u[j], a.sigmoid ? make_float2(sigmoid(g[j].x), sigmoid(g[j].y)) : g[j]);
    } else if (a.gate_kind == MOE_GATE_TOKEN) {
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], both(gt));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = mul2(both(a.a), r[i][j]);
      r[i][j] = a.y ? fma2(both(a.b), u[j], x) : x;
      ss = fma2(r[i][j], r[i][j], ss);
    }
    if (a.x_out && c < nc) {
      if (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.x_out) + row * a.x_out_ld + 8 * c);
        o[0] = make_float4(r[i][0].x, r[i][0].y, r[i][1].x, r[i][1].y);
        o[1] = make_float4(r[i][2].x, r[i][2].y, r[i][3].x, r[i][3].y);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x_out) + row * a.x_out_ld + 8 * c) =
            pack8(r[i]);
      }
    }
  }
  if (!a.h && !a.codes) return;
  const float inv = rsqrtf(row_sum<WARP_ROW>(ss.x + ss.y, red[1]) * a.inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = lane + i * nt;
    const bool live = c < nc;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[i][j] = mul2(r[i][j], both(inv));
    if (a.pre_w && live) {
      float2 w[4];
      load8f(a.pre_w + 8 * c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = mul2(r[i][j], add2(w[j], both(a.w_off)));
    }
    if (a.h && live) *reinterpret_cast<uint4*>(a.h + row * a.h_ld + 8 * c) = pack8(r[i]);
    if (a.codes)
      quant8(r[i], live, a.codes + (long long)row * a.d + 8 * c,
             a.scales + (long long)row * blocks128(a.d) + (c >> 4));
  }
}

// bf16 rows to e4m3: one half-warp per 128 columns.
__global__ void __launch_bounds__(256) fp8_quant_kernel(const uint16_t* __restrict__ x, long long ld,
                                                        int T, int d, uint8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int kb = blocks128(d);
  const long long n = (long long)T * kb;
  const long long step = (long long)gridDim.x * (blockDim.x >> 4);
  const int l = threadIdx.x & 15;
  // whole warps walk the loop: the two halves of a warp differ by one block
  for (long long b0 = (long long)blockIdx.x * (blockDim.x >> 4) + ((threadIdx.x >> 5) << 1); b0 < n;
       b0 += step) {
    const long long b = b0 + ((threadIdx.x >> 4) & 1);
    const long long row = b / kb;
    const int cb = (int)(b - row * kb), c = cb * kBlock128 + 8 * l;
    const bool live = b < n && c < d;
    float2 v[4];
    unpack8(live ? *reinterpret_cast<const uint4*>(x + row * ld + c) : make_uint4(0, 0, 0, 0), v);
    quant8(v, live, codes + row * d + c, scales + b);
  }
}

template <bool F32, bool WARP_ROW, int CH>
cudaError_t launch_norm(const NormArgs& a, int threads, cudaStream_t st) {
  const int grid = WARP_ROW ? (a.T + kWarpRows - 1) / kWarpRows : a.T;
  return launch_pdl(norm_block_kernel<F32, WARP_ROW, CH>, dim3(grid), dim3(threads), 0, st, a);
}

template <bool F32>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t st) {
  const int nc = a.d >> 3;
  if (nc <= 32) return launch_norm<F32, true, 1>(a, 32 * kWarpRows, st);
  if (nc <= 64) return launch_norm<F32, true, 2>(a, 32 * kWarpRows, st);
  return launch_norm<F32, false, 1>(a, (nc + 31) / 32 * 32, st);
}

}  // namespace

cudaError_t launch_norm_block(const NormArgs& a, bool stream_f32, cudaStream_t st) {
  return stream_f32 ? launch_norm_t<true>(a, st) : launch_norm_t<false>(a, st);
}

cudaError_t launch_fp8_quant(const uint16_t* x, long long ld, int T, int d, uint8_t* codes,
                             float* scales, cudaStream_t st) {
  const long long n = (long long)T * blocks128(d);
  long long grid = (n + 15) / 16;
  if (grid > 8ll * sm_count()) grid = 8ll * sm_count();
  return launch_pdl(fp8_quant_kernel, dim3((unsigned)grid), dim3(256), 0, st, x, ld, T, d, codes,
                    scales);
}

}  // namespace moe
