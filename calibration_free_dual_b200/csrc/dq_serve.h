// dq_serve.h — launch descriptors of the 8-bit serving path: row quantizer, INT8 product, paged
// cache append and paged attention.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "dq.h"

namespace dq {

constexpr int SERVE_SMS = 148;          // SMs of the part the launches are planned for
constexpr unsigned ERRBIT_BADARG = 4u;  // error word: an index or length on the device out of its range

// per-device error word (dq_api.cu); false when the device or the symbol cannot be had
bool error_word(unsigned** out);

struct RowsArgs {
  const void* X;
  int64_t rows, n, ldx;
  const float* c;
  int8_t* codes;
  float* scales;
  unsigned* err_word;
};
cudaError_t launch_row_quant(const RowsArgs& A, int esize, cudaStream_t s);

// y[T, N] = x[T, K] w[N, K]^T * xs * ws
struct Gemm8Args {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int64_t T, N, K, ldy;
  int y_bf16;
  unsigned* err_word;
  int after_rows;         // the stream's previous launch is the row quantizer that writes x, xs
};
size_t gemm8_workspace_bytes(int64_t T, int64_t N, int64_t K);
cudaError_t launch_gemm8(const Gemm8Args& A, void* workspace, cudaStream_t s);

struct AppendArgs {
  dq_kv_cache cache;
  int64_t tokens;
  const void* k;
  const void* v;
  const void* q;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  const int64_t* slots;
  dq_rotary rot;          // dim = 0: no rotation
  int q_heads;            // 0: no queries
  void* q_out;
  unsigned* err_word;
};
cudaError_t launch_append(const AppendArgs& A, int esize, cudaStream_t s);

struct AttnArgs {
  dq_kv_cache cache;
  dq_attention a;
  int group;              // query heads per key head
  unsigned* err_word;
};
size_t attn_workspace_bytes(const AttnArgs& A);
cudaError_t launch_attention(const AttnArgs& A, void* workspace, cudaStream_t s);

}  // namespace dq
