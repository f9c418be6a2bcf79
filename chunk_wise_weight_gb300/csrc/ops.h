// ops.h -- launchers of the operators around the layer: embedding lookup,
// layer norm, the gated delta rule, and their gradients.  The entry points in
// ops_api.cu validate arguments and call these.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace ittt {

// Rows of `d` contiguous elements: row r of [B, T, d] starts at element
// (r / T) * stride_b + (r % T) * stride_t.
struct RowView {
  const void* data;
  int64_t stride_b, stride_t;
  int64_t T;
  bool fp32;
#ifdef __CUDACC__
  __device__ __forceinline__ int64_t offset(int64_t r) const {
    if (r < T) return r * stride_t;  // always so when the rows are evenly spaced
    const uint32_t b = uint32_t(r) / uint32_t(T);
    return int64_t(b) * stride_b + (r - int64_t(b) * T) * stride_t;
  }
#endif
};

// ------------------------------------------------------------------ embedding
struct EmbedArgs {
  const void* ids;
  bool ids64;
  int64_t N, V, d;
  const void* table;
  bool table_fp32;
  float scale;
  void* out;
  bool out_fp32;
};
cudaError_t launch_embed(const LaunchEnv& env, const EmbedArgs& a);

struct EmbedGradArgs {
  const void* ids;
  bool ids64;
  int64_t N, V, d;
  RowView dy;
  float scale;
  void* grad;  // [V, d]
  bool grad_fp32;
  bool accumulate;
  unsigned char* ws;
};
size_t embed_grad_scratch(int64_t N, int64_t d);
cudaError_t launch_embed_grad(const LaunchEnv& env, const EmbedGradArgs& a);

// ----------------------------------------------------------------- layer norm
struct NormArgs {
  int64_t N, d;
  RowView x;
  const void* weight;
  bool w_fp32;
  const void* bias;  // nullptr: none
  bool b_fp32;
  float eps;
  void* out;  // [N, d] dense
  bool out_fp32;
  float* mean;  // [N] or nullptr
  float* rstd;
};
cudaError_t launch_layer_norm(const LaunchEnv& env, const NormArgs& a);

struct NormGradArgs {
  int64_t N, d;
  RowView dy, x;
  const void* weight;
  bool w_fp32;
  const float* mean;
  const float* rstd;
  void* dx;  // [N, d] dense, in x's type
  void* dw;  // [d] or nullptr
  bool dw_fp32;
  void* db;  // [d] or nullptr
  bool db_fp32;
  float* ws;
};
size_t layer_norm_grad_scratch(int64_t N, int64_t d);
cudaError_t launch_layer_norm_grad(const LaunchEnv& env, const NormGradArgs& a);

}  // namespace ittt

namespace ittt {

// ----------------------------------------------------------- gated delta rule
// [B, T, heads, dim] with a contiguous last dimension (strides in elements).
struct HeadView {
  const void* data;
  int64_t sb, st, sh;
  bool vec;  // every row starts on a 16-byte boundary
};
struct GateView {  // fp32 [B, T, Hv]
  const float* data;
  int64_t sb, st, sh;
};

constexpr int kDeltaChunk = 64;

// The sequences: B of T tokens (cu == nullptr), or `ndocs` documents packed
// in one row, document s the tokens [cu[s], cu[s + 1]) (possibly none), its
// chunks [base[s], base[s + 1]) of all.
struct DeltaMap {
  const int* cu;
  const int* base;
  int ndocs, nchunks;
  int T, n;  // regular: tokens and chunks a sequence
#ifdef __CUDACC__
  __device__ __forceinline__ int row(int s) const { return cu ? 0 : s; }
  __device__ __forceinline__ int start(int s) const { return cu ? __ldg(cu + s) : 0; }
  __device__ __forceinline__ int len(int s) const {
    return cu ? __ldg(cu + s + 1) - __ldg(cu + s) : T;
  }
  __device__ __forceinline__ int chunk0(int s) const { return cu ? __ldg(base + s) : s * n; }
  // sequence of chunk g: the last s with base[s] <= g (empty ones own none)
  __device__ __forceinline__ int doc_of(int g) const {
    if (!cu) return g / n;
    int lo = 0, hi = ndocs - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) / 2;
      if (__ldg(base + m) <= g) lo = m; else hi = m - 1;
    }
    return lo;
  }
#endif
};

struct DeltaArgs {
  HeadView q, k, v;
  GateView g, beta;
  bool fp32;  // type of q, k, v
  int B, T, Hk, Hv, dk, dv;
  DeltaMap map;
  float scale;
  const float* state_in;  // [ndocs, Hv, dv, dk] or nullptr (zero)
  float* state_out;       // or nullptr
  void* out;              // [B, T, Hv, dv] dense, or nullptr
  bool out_fp32;
  const void* slots;  // one token a sequence: its row of the state pool, or nullptr
  bool slots64;
  int64_t pool;       // rows of the state pool
  unsigned char* ws;
};

// Scratch and launch of the chunked form (bf16 q, k, v; dk 64 or 128).
size_t delta_scratch(int64_t nchunks, int Hv);
cudaError_t launch_delta_chunked(const LaunchEnv& env, const DeltaArgs& a);
// Gradients of the chunked form.
struct DeltaGradArgs {
  DeltaArgs f;    // the forward call (state_in; no output)
  HeadView dout;  // bf16
  const float* dstate_out;  // [ndocs, Hv, dv, dk] or nullptr (zero)
  float* dstate_in;         // or nullptr
  void *dq, *dk, *dv;       // dense bf16
  float *dg, *dbeta;        // dense fp32 [B, T, Hv]
};
size_t delta_grad_scratch(int64_t nchunks, int Hv, int dk, int dv);
cudaError_t launch_delta_grad(const LaunchEnv& env, const DeltaGradArgs& a);

// Token by token, one warp a few rows of the state: any type; no scratch.
cudaError_t launch_delta_recurrent(const LaunchEnv& env, const DeltaArgs& a);

}  // namespace ittt
