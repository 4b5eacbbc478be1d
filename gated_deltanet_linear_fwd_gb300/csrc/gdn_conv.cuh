// Arguments of the short causal convolution before the gated delta rule.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "gdn_internal.cuh"
#include "sm103_ptx.cuh"

namespace gdn {

constexpr int kConvD = 128;      // channels of a head
constexpr int kConvMaxTaps = 4;

struct ConvArgs {
  const void* x;           // [T, C], row stride x_stride
  const float* weight;     // [C, W]
  const float* bias;       // [C] or null
  const void* state;       // [n_seqs, W - 1, C] inputs before each sequence, or null (zeros)
  const int32_t* cu;       // [n_seqs + 1] or null
  void* q;                 // [T, h_qk, 128]; backward: the gradient, read
  void* k;                 // [T, h_qk, 128]
  void* v;                 // [T, h_v, 128]
  void* final_state;       // [n_seqs, W - 1, C] or null
  int64_t x_stride, dx_stride;
  int n_seqs, T, n_each, h_qk, h_v;
  int width, silu, norm;
  float eps;
  // Heads whose norm is taken, the first n_unit, and the others: they cost more, so
  // a warp takes fewer of their tokens in a row.
  int n_unit;
  int run[2];              // tokens a warp takes, of the former, of the others
  int runs[2];             // runs of all tokens (backward: groups of 8 of them)
  int blocks;              // CTAs before those for the final states
  // backward
  const void* d_final;     // [n_seqs, W - 1, C] or null (zero)
  void* dx;                // [T, C], row stride dx_stride
  void* d_state;           // [n_seqs, W - 1, C] or null
  float* d_weight;         // [C, W] or null
  float* d_bias;           // [C] or null
  float* part;             // [groups, W + 1, channels] of either, sums of the weights' gradients
  int sums;                // d_weight or d_bias is wanted
};

cudaError_t launch_conv(const ConvArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_conv_step(const ConvArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvArgs& a, bool f32, cudaStream_t st);
cudaError_t launch_conv_bwd_sums(const ConvArgs& a, bool f32, cudaStream_t st);

}  // namespace gdn
