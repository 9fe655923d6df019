// ops.h -- internal declarations of the operators of include/moe_ops.h.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"
#include "moe_ops.h"

namespace moe {

constexpr int kBlock128 = 128;           // columns (and weight rows) that share one scale
constexpr float kE4m3Max = 448.f;

__host__ __device__ inline int blocks128(int n) { return (n + kBlock128 - 1) / kBlock128; }

// Let a kernel use up to that much dynamic shared memory: the same number in every
// call, so that calls of several threads do not take it from one another.
cudaError_t allow_smem(const void* kernel, size_t most);
constexpr size_t kMaxSmem = 227 * 1024;  // of a block, static included
// Rows of one call: below 2^31 with room for a rounding up to tiles.
constexpr int kMaxRows = 0x7FFFFF00;

struct NormArgs {
  int d, T;
  int gate_kind;
  bool post, sigmoid;
  float eps, a, b;
  float inv_d;                 // 1 / d
  float w_off;                 // added to the weights (1 when they are zero-centred)
  const float *pre_w, *post_w; // or nullptr
  long long x_ld, y_ld, gate_ld, x_out_ld, h_ld;
  const void* x;
  const uint16_t* y;           // or nullptr
  const uint16_t* gate;
  void* x_out;                 // or nullptr
  uint16_t* h;                 // or nullptr
  uint8_t* codes;              // or nullptr
  float* scales;
};
cudaError_t launch_norm_block(const NormArgs& a, bool stream_f32, cudaStream_t st);
cudaError_t launch_fp8_quant(const uint16_t* x, long long ld, int T, int d, uint8_t* codes,
                             float* scales, cudaStream_t st);

struct GemmArgs {
  int M, N, K, G;
  const uint8_t* a;
  const float* a_scales;
  const uint8_t* w;
  const float* w_scales;
  const int32_t* offsets;      // nullptr: dense
  uint16_t* c;
  Control* ctl;                // or nullptr
};
// The kernel a product takes on a device of `sms` SMs.
struct GemmPlan {
  int bn;            // columns of a tile
  int a_rows;        // rows of A staged for a tile
  int stages;        // of the operand ring
  long long tiles;   // at most
};
GemmPlan plan_fp8_gemm(int M, int N, int G, bool grouped, int sms);
cudaError_t launch_fp8_gemm(const GemmArgs& a, cudaStream_t st);

struct Fp8LayerDev {
  int d, E, F, k, Fs;
  const float *Wr, *bias;
  const uint8_t *gu, *dn, *sgu, *sdn;
  const float *gus, *dns, *sgus, *sdns;
};
constexpr int kFp8Window = 8;            // tokens of one launch (mma n = 8)
size_t fp8_layer_ws_bytes(const Fp8LayerDev& L);
cudaError_t launch_fp8_layer(const Fp8LayerDev& L, const uint16_t* x, int T, uint16_t* y,
                             int32_t* ids, float* w, char* ws, cudaStream_t st);

}  // namespace moe
